// Attention of a few new tokens per sequence (one, or a tree of drafted ones) over a paged cache.
//
// For a sequence with context L and n tokens, the rows of a key/value head are its n * G (token,
// query head) pairs. s = scale q k^T over the positions seen, out = softmax(s) v, in one pass over
// the positions with a running maximum m and sum l per row:
//     p_j = 2^(s_j log2 e - m),  l = sum p_j,  o = sum p_j v_j;   a larger m scales l and o down.
//
// A workgroup's waves lie R side by side over rows, MT tiles of 16 each, and T over positions. Keys and
// values go from memory straight to LDS, 16 bytes a lane, without passing registers:
//   * S^T = K Q^T with v_mfma_f32_16x16x32: keys lie in LDS as the A operand, in the order of the lanes
//     that fetched them. The result leaves lane (row, j) with the positions 4 j .. 4 j + 3 of both
//     16-position halves of a tile.
//   * O^T = V^T P^T: those eight weights, packed to 16 bits, are the B operand as they are, if the
//     operand's k index counts positions in that order. For A, transposing LDS reads give lane (dim, j)
//     the same eight positions of its dim; value rows lie with their 16-byte columns exchanged by XOR so
//     that these reads spread over the banks. 8-bit values are read so too and widened on the way; 8-bit
//     keys are widened as well, or (bf16 queries, 128 dims or more) multiplied as they are by queries in
//     two 8-bit parts, which costs the matrix cores the same and the vector unit nothing: 4 trees of 64 tokens
//     over 30K to 65K positions (512 rows of a head) 520 -> 455 us.
//   * m is not followed exactly: o is scaled only when a score passes m by more than 2^8 (a wave-uniform
//     branch that long contexts take a few times), so the usual step has no cross-lane work at all, l is
//     kept per lane, and fp16 weights p = 2^((s - m) log2 e + 7) stay below 2^15, inside fp16, while those down
//     to 2^-21 of the largest are normal numbers (bf16 ones have fp32's range and no shift). m is kept as a score
//     and -m is what the product K Q^T starts from, so that s - m costs nothing and is right at any size of s
//     (s log2 e - m in one fused step, m rounded, is off by the rounding of m: at |s| = 10^8 the largest weight
//     would be 2^(7 +- 4)). Waves and pieces are joined by differences of these maxima too, and as means of
//     values, which never pass the largest value.
// Descriptors cover 16 rows; one of size 0 stands for rows that are not needed or on no valid page, so
// every step issues the same transfers, their count is waited for exactly, and no table entry is ever
// trusted. Few rows (R = 1): each wave has tiles of its own and no barrier; with one tile, its keys make
// room for the next ones while its values are used (two workgroups a CU with 128 dims in 16 bits, 8 decode
// steps in flight; two tiles each, one workgroup a CU: 337 against 253 us for 1.3 GB). More rows: R waves
// share each step, double-buffered, one barrier a step of 64 positions.
// Nothing in the loop is a vector load the compiler knows of (the block table is read by the scalar
// unit, the queries are waited for before): it would wait for it, and so for all transfers under way
// (1.0 GB at 128 rows: 226 us with such waits, 170 without). No instance spills vector registers with the flags
// of the build (packed fp32 off), so no scratch access is among the loop's loads either.
//
// Split over workgroups: the pieces (sequence, head, row block, run of positions) are cut on the
// device from the lengths, of equal size, and taken by a grid of resident workgroups; a piece that is not
// a whole sequence leaves o / l, m, l in the workspace and k_join weighs them in order. Few rows take about
// three pieces a workgroup where each is long enough (64 ragged sequences, with the join: 236 against 272 us),
// many rows one (their sums are large: 8 trees of 16 tokens 185 against 220 us).
//
// Bound: HBM up to about 64 rows (5.0 to 5.8 TB/s of keys and values over long contexts, where a plain
// streaming read of this card reaches 6.4); beyond, the vector unit beside the matrix cores (1.0 PFLOP/s
// at 512 rows of 128 dims in 8 bits); short contexts, a chain of a dozen memory latencies (7 to 8 us).
#include "cache_internal.h"

namespace ubw {
namespace cache {
namespace {

using h16 = _Float16;
using b16 = __bf16;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t Rsrc;

template <typename T>
struct Half;
template <>
struct Half<h16> {
    typedef h16 x2 __attribute__((ext_vector_type(2)));
    typedef h16 x8 __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExp = 0x7c00;
    static constexpr bool kSplits = false;
    static constexpr float kShift = 7.f;  // of weights: see above
    static __device__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
    static __device__ uint32_t from8(uint32_t w, bool high) {
        return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true)
                                                 : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false));
    }
};
template <>
struct Half<b16> {
    typedef b16 x2 __attribute__((ext_vector_type(2)));
    typedef b16 x8 __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExp = 0x7f80;
    static constexpr bool kSplits = true;
    static constexpr float kShift = 0.f;
    static __device__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
    static __device__ uint32_t from8(uint32_t w, bool high) {
        return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true)
                                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
    }
};
// What sums under the maximum m (a score; -INFINITY: of nothing) are multiplied by under the maximum `to`: a
// difference of scores first, so that it is as exact for large scores as for small ones.
__device__ inline float weight(float m, float to, float cc) {
    return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - to) * cc);
}
// bf16 queries are multiplied by 2^lower(scale) before the product with the keys, so that what is left of the
// scale is 4 or more: a finite score is then below 2^126 there, and neither it nor a difference of two passes
// fp32's range. Down to 2^-32 only, so that elements above 2^-94 lose nothing. (fp16 products stay below 2^41.)
template <typename T>
__device__ inline int lower(float scale) {
    return Half<T>::kSplits ? min(max(__builtin_amdgcn_frexp_expf(scale) - 3, -32), 0) : 0;
}
template <typename T>
__device__ inline uint32_t pack(float a, float b) {  // rounded to nearest even
    typename Half<T>::x2 v;
    v.x = (T)a;
    v.y = (T)b;
    return __builtin_bit_cast(uint32_t, v);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLow = -3.402823466e38f;  // lim of a row that has seen nothing
constexpr float kSlack = 8.f;
constexpr int kCus = 256;
constexpr int kNoLds = 0xf;  // a scheduling barrier for all but arithmetic
// Words that no kernel running beside this one writes, read by the scalar unit. (As vector loads they
// would be waited for behind all transfers under way.)
typedef const __attribute__((address_space(4))) int32_t ScalarWord;
__device__ inline ScalarWord* scalar_words(const int32_t* p) { return (ScalarWord*)(uintptr_t)p; }

// ---- what a piece is
struct Seq {
    int ctx, n, q0;  // context, tokens, first row of q
};
__device__ inline Seq seq_of(const AttnArgs& a, int b) {
    Seq s;
    const int q0 = min(max(a.q_start[b], 0), a.tokens), q1 = min(max(a.q_start[b + 1], q0), a.tokens);
    s.q0 = q0;
    s.n = min(q1 - q0, a.max_tree);
    s.ctx = max(a.ctx_len[b], 0);
    return s;
}
__device__ inline Seq seq_at(const AttnArgs& a, int b) {  // the same for a wave-uniform b
    Seq s;
    const ScalarWord* start = scalar_words(a.q_start) + b;
    const int q0 = min(max((int)start[0], 0), a.tokens), q1 = min(max((int)start[1], q0), a.tokens);
    s.q0 = q0;
    s.n = min(q1 - q0, a.max_tree);
    s.ctx = max((int)scalar_words(a.ctx_len)[b], 0);
    return s;
}
// positions there are: the table ends them
__device__ inline int positions(const AttnArgs& a, const Seq& s) {
    const int64_t most = (int64_t)a.table_cols << a.c.lps;
    return (int)min((int64_t)s.ctx + s.n, most);
}
struct Plan {
    int units, blocks, splits;
};
__device__ inline Plan plan_of(const AttnArgs& a, const Seq& s, int rb, int chunk) {
    Plan p;
    p.blocks = s.n > 0 ? (s.n * a.group + rb - 1) / rb : 0;
    p.units = s.n > 0 ? max(1, (int)(((int64_t)positions(a, s) + kAttnUnit - 1) / kAttnUnit)) : 0;
    p.splits = chunk > 0 ? attn_splits(p.units, chunk) : min(p.units, 1);
    return p;
}

// Which of the four positions behind ctx + d (d may be negative: context, all seen) a token with this
// mask sees. No branches: bit x of (mask << 4 | 15) is position ctx + x - 4.
__device__ inline uint32_t four_seen(uint64_t mask, int d) {
    const int x = min(max(d, -4), 64) + 4;
    const uint64_t low = ((mask << 4) | 15) >> (x & 3), high = mask >> ((x - 4) & 63);
    const uint64_t b = x < 4 ? low : high;
    return x > 67 ? 0u : (uint32_t)b & 15u;
}

// Sum over the workgroup's NT threads (every thread gets it). `lds`: 4 words.
template <int NT>
__device__ inline int64_t wg_sum(int64_t x, int64_t* lds) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor((long long)x, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    int64_t sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) sum += lds[w];
    return sum;
}

// Cuts the batch: units per piece (the least for which the pieces do not pass the target by more than
// the sequences that cannot be joined make them), and in pre[b] the pieces of the sequences before b.
template <int NT>
__device__ inline int cut_batch(const AttnArgs& a, int rb, bool one_row_wave, int* pre, int64_t* lds) {
    const int tid = threadIdx.x;
    const int per = (a.batch + NT - 1) / NT;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    int64_t units = 0;
    // a thread's first sequence, most often its only one, is loaded once
    const Seq s0 = b0 < b1 ? seq_of(a, b0) : Seq{0, 0, 0};
    const auto seq = [&](int b) { return b == b0 ? s0 : seq_of(a, b); };
    for (int b = b0; b < b1; ++b) {
        const Plan p = plan_of(a, seq(b), rb, 0);
        units += (int64_t)p.units * p.blocks;
    }
    const int64_t total = wg_sum<NT>(units, lds) * a.c.heads;
    const int target = attn_aim(total, a.target, one_row_wave);
    int chunk = attn_chunk(total, target);
    int mine = 0;
    for (int step = 0;; ++step) {
        mine = 0;
        for (int b = b0; b < b1; ++b) {
            const Plan p = plan_of(a, seq(b), rb, chunk);
            mine += p.splits * p.blocks * a.c.heads;
        }
        const int64_t pieces = wg_sum<NT>(mine, lds);
        if (step == 4 || pieces <= target) break;
        chunk = attn_larger_chunk(chunk, pieces, target);
    }
    int y = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int z = __shfl_up(y, d);
        if ((tid & 63) >= d) y += z;
    }
    int* sums = reinterpret_cast<int*>(lds);
    __syncthreads();
    if ((tid & 63) == 63) sums[tid >> 6] = y;
    __syncthreads();
    int first = y - mine;
    for (int w = 0; w < (tid >> 6); ++w) first += sums[w];
    for (int b = b0; b < b1; ++b) {
        const Plan p = plan_of(a, seq(b), rb, chunk);
        pre[b] = first;
        first += p.splits * p.blocks * a.c.heads;
    }
    if (tid == NT - 1) pre[a.batch] = first;
    __syncthreads();
    return chunk;
}

// Workspace: pieces' rows of D means, then (m, l) of each row.
__device__ inline float* piece_rows(const AttnArgs& a, int item, int rb, int d) { return a.ws + (int64_t)item * rb * (d + 2); }

__device__ inline Rsrc rows16(const char* p, uint32_t bytes) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
                       ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), (short)0, (int)__builtin_amdgcn_readfirstlane(bytes),
                                             0x00020000);
}

// ---- a tile in LDS: 32 positions of one key/value head, as 1 KiB pieces of 64 lanes x 16 bytes
template <bool FP8, int D>
struct Layout {
    static constexpr int kElem = FP8 ? 1 : 2, kRowB = D * kElem;
    static constexpr int KL = kRowB / 64;            // pieces of 16 key rows
    static constexpr int P = kRowB / 16;             // 16-byte columns of a value row
    static constexpr int RP = 64 / P;                // value rows in a piece
    static constexpr int CK = 2 * KL, CV = 32 / RP;  // pieces of keys, of values
    static constexpr int kBytes = 64 * kRowB;
    // Keys lie as the A operand of S^T = K Q^T takes them: piece (half, s), lane (c, j) = row c, bytes
    // 64 s + 16 j .. Values lie row by row, the 16-byte columns of row t exchanged by XOR with this, so
    // that the 16 or 32 rows a transposing read touches spread over all banks.
    static __device__ constexpr int mix(int t) { return (P >= 16 ? t : P == 8 ? t >> 1 : t >> 2) & (P >= 16 ? 15 : P - 1); }
};

// 16 bytes a lane from memory straight to LDS at `lds` + 16 lane. The compiler does not see the
// transfer: waits are placed by hand (m0 it sets itself wherever it uses it). ONCE: nobody else reads these
// bytes (keys and values under one row block), they need not stay in the L2 (1.3 GB in 64 ragged sequences:
// 229 us, 249 without; 0.85 GB under one block of 128 rows 161, 169 without; under four row blocks they are
// read again: 638 us without, 648 with).
template <bool ONCE>
__device__ inline void to_lds(Rsrc r, uint32_t off, uint32_t lds) {
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(lds), "v"(off), "s"(r) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r) : "memory");
}
template <int N>
__device__ inline void wait_loads() {  // all but the newest N transfers have arrived
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ inline void wait_and_meet() {  // LDS reads done, then the workgroup's barrier
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
template <typename T>
__device__ inline T* lds_at(uint32_t at) {
    return (T*)(__attribute__((address_space(3))) T*)(uintptr_t)at;
}

// The elements of a word that are infinite or NaN (e4m3: NaN), as a mask.
template <typename TQ, bool FP8>
__device__ inline uint32_t not_finite(uint32_t w) {
    if constexpr (FP8) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 32; k += 8) m |= ((w >> k) & 0x7f) == 0x7f ? 0xffu << k : 0u;
        return m;
    } else {
        constexpr uint32_t e = Half<TQ>::kExp;
        return ((w & e) == e ? 0xffffu : 0u) | (((w >> 16) & e) == e ? 0xffff0000u : 0u);
    }
}

// 128 bf16 values of a row (32 of this lane, in q[0 .. 3], the others in the row's other three lanes) as two
// e4m3 parts each, x = 2^u hi + 2^(u - 5) lo: hi is x rounded to 4 bits, what is left of 8 bits fits lo's 4.
// Values below 2^-13 of the row's largest are off by up to 2^-22 of it (less than the fp32 sums of a score
// lose). q[0 .. 1] get hi, q[2 .. 3] lo; returns the parts' powers of two as biased bytes 0 and 1 (one
// power for the row: the product applies those of its four lanes to 32 of the 128 dims each, and these are
// not the lanes that hold them; rows below 2^-115 - low count as of that size, so that it fits). Infinities become NaN, which scores with them end in anyway.
typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr int kOne8 = 0x7f;  // the power 2^0
__device__ inline i32x8 joined(u32x4 a, u32x4 b) {
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
// Returns them times 2^low.
__device__ inline int split_query(u32x4* q, int low) {
    uint32_t top = 0;  // exponent of the largest, in place
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t w = q[i >> 2][i & 3];
        const uint32_t a = w & 0x7f80u, b = (w >> 16) & 0x7f80u;
        top = max(top, max(a == 0x7f80u ? 0u : a, b == 0x7f80u ? 0u : b));
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    const int e = max((int)(top >> 7), 12 - low);
    const float up = __builtin_bit_cast(float, (uint32_t)(261 - e) << 23);  // 2^(134 - e): the largest comes to [128, 256)
    u32x4 hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[2] = {q[i >> 1][2 * (i & 1)], q[i >> 1][2 * (i & 1) + 1]};
        int h = 0, r = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x = __builtin_bit_cast(float, w[k] << 16), y = __builtin_bit_cast(float, w[k] & 0xffff0000u);
            x = __builtin_isfinite(x) ? x * up : __builtin_nanf("");
            y = __builtin_isfinite(y) ? y * up : __builtin_nanf("");
            h = k ? __builtin_amdgcn_cvt_pk_fp8_f32(x, y, h, true) : __builtin_amdgcn_cvt_pk_fp8_f32(x, y, h, false);
            const f32x2 z = k ? __builtin_amdgcn_cvt_pk_f32_fp8(h, true) : __builtin_amdgcn_cvt_pk_f32_fp8(h, false);
            x = (x - z.x) * 32.f;
            y = (y - z.y) * 32.f;
            r = k ? __builtin_amdgcn_cvt_pk_fp8_f32(x, y, r, true) : __builtin_amdgcn_cvt_pk_fp8_f32(x, y, r, false);
        }
        hi[i >> 2][i & 3] = (uint32_t)h;
        lo[i >> 2][i & 3] = (uint32_t)r;
    }
    q[0] = hi[0];
    q[1] = hi[1];
    q[2] = lo[0];
    q[3] = lo[1];
    return (e - 7 + low) | (e - 12 + low) << 8;
}

// MT row tiles a wave, R waves side by side over rows, T over positions, NS tiles of 32 positions a
// step, NB steps in LDS for each of the T.
template <bool FP8, int D, int MT, int R, int T, int NS, int NB>
struct Cfg {
    static constexpr int kThreads = 64 * R * T, RB = 16 * MT * R;
    static constexpr int kTiles = T * NB * NS * Layout<FP8, D>::kBytes;
    static constexpr int kJoin = (T - 1) * RB * (D + 4) * 4;  // laid over the tiles
    static constexpr int kLds = kTiles > kJoin ? kTiles : kJoin;
    // workgroups per CU: by LDS, and waves per SIMD by registers (with three waves the largest tiles spill: 8 bits,
    // 8 tokens of 8 sequences over 16K positions, 64 heads over 8 of 128 dims: 111 us, with two 68)
    static constexpr int kFit = (160 * 1024 - 512) / (kLds + 8 * T * RB + 1024);
    static constexpr int kWaves = D * MT == 256 ? 2 : 3;
    static constexpr int kMost = kWaves * 256 / kThreads;
    static constexpr int kPerCu = kFit < kMost ? kFit : kMost;
    static constexpr int kSimd = kPerCu * kThreads / 256 < 1 ? 1 : kPerCu * kThreads / 256;
};

template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, bool ONCE>
__global__ __launch_bounds__((Cfg<FP8, D, MT, R, T, NS, NB>::kThreads), (Cfg<FP8, D, MT, R, T, NS, NB>::kSimd)) void k_attn(AttnArgs a) {
    using H = Half<TQ>;
    using L = Layout<FP8, D>;
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    constexpr int NE = D / 16, KS = D / 32, RB = C::RB, U = kAttnUnit, STEP = 32 * NS * T;
    constexpr int NC = (L::CK + L::CV) / R;  // transfers of a wave per tile
    constexpr int NP = 2 * NS;  // pages of a wave's part of a step
    constexpr int kRow = D + 4;              // LDS row of o, in floats
    static_assert((L::CK + L::CV) % R == 0, "pieces of a tile are shared out evenly");
    static_assert(R > 1 ? NB == 2 : NS == 1, "shared steps are double-buffered, private ones have one tile");
    extern __shared__ int pre[];  // [batch + 1], with a split
    __shared__ int64_t lds64[4];
    __shared__ float ml[T][RB][2];
    // Of each wave: it met values of the tree that are not finite in this piece. A wave clears and sets its own
    // word only, so both come in its own order; the others read it behind a barrier of the piece's end, and
    // the piece's last barrier stands before the next clearing.
    __shared__ int odd[R * T];
    __shared__ __align__(1024) char buf[C::kLds];
    const uint32_t buf0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)buf;
    float* o_lds = reinterpret_cast<float*>(buf);

    // bf16 queries over 8-bit keys of 128 dims or more: queries as two e4m3 parts (split_query)
    constexpr bool kSplit = FP8 && D >= 128 && Half<TQ>::kSplits;
    constexpr int NG = kSplit ? D / 128 : 1;

    // bf16 values reach as far as the fp32 sums do. A piece whose sums did not stay finite is gone through once
    // more, with the maxima that it ended at and weights so much smaller that the sums do (unless a value is
    // not finite itself). To look costs a piece 0.2 to 0.3 us (one token over 37 positions 7.2 -> 7.5 us, 24 ragged
    // trees of 64 dims 25.6 -> 26.6, 64 ragged single tokens 234); values scaled down beforehand would cost
    // the loop more, and smaller weights at once the smallest ones.
    constexpr bool kWide = !FP8 && H::kExp == Half<b16>::kExp;
    __shared__ int beyond[kWide ? R * T : 1];  // of each wave
    bool again = false;
    float ms[MT], lim[MT], shift = H::kShift;

    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % R, tw = wave / R;

    int chunk = 0, items;
    const int blocks_max = (a.max_tree * a.group + RB - 1) / RB;
    if (a.target > 0) {
        chunk = cut_batch<C::kThreads>(a, RB, R == 1, pre, lds64);
        items = __builtin_amdgcn_readfirstlane(pre[a.batch]);
        if (blockIdx.x == 0) {  // for k_join
            int* head = reinterpret_cast<int*>(a.ws + a.max_items * RB * (D + 2));
            for (int b = threadIdx.x; b < a.batch; b += C::kThreads) head[1 + b] = pre[b];
            if (threadIdx.x == 0) head[0] = chunk;
        }
    } else {
        items = a.batch * a.c.heads * blocks_max;
    }

    // this lane's part of the transfers and reads, in bytes
    const uint32_t tile0 = buf0 + tw * (NB * NS * L::kBytes);
    const uint32_t koff = c * a.c.k_row + j * 16;
    const int vt = lane / L::P, vp = lane % L::P;           // row and column of a value piece
    const int q4 = c >> 2, q2 = c >> 1;                     // a transposing read: rows by fours, by eights
    const int vrow = FP8 ? 4 * j + (q2 & 3) + (q2 & 4) * 4 : 4 * j + q4;
    const uint32_t vread = L::CK * 1024 + vrow * L::kRowB +
                           (FP8 ? L::mix(vrow) * 16 + (c & 1) * 8
                                : (((c >> 1) & 1) ^ (L::mix(vrow) & 1)) * 16 + (c & 1) * 8 + (L::mix(vrow) & ~1) * 16);

    // Workgroups go to the eight XCDs in turn; each XCD takes a contiguous eighth of the pieces, so that
    // the row blocks over the same keys and values, neighbours in the list, meet in one L2.
    const int eighth = (items + 7) >> 3;
    for (int it = blockIdx.x; it < 8 * eighth; it += gridDim.x) {
        const int item = (it & 7) * eighth + (it >> 3);
        if (item >= items) continue;
        int b, h, blk, split;
        Seq s;
        Plan p;
        if (a.target > 0) {
            int lo = 0, hi = a.batch;  // the last b with pre[b] <= item
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid] <= item) lo = mid; else hi = mid;
            }
            b = __builtin_amdgcn_readfirstlane(lo);
            s = seq_at(a, b);
            p = plan_of(a, s, RB, chunk);
            int r = item - __builtin_amdgcn_readfirstlane(pre[b]);
            blk = r % p.blocks;
            r /= p.blocks;
            split = r % p.splits;
            h = r / p.splits;
        } else {
            blk = item % blocks_max;
            const int r = item / blocks_max;
            h = r % a.c.heads;
            b = r / a.c.heads;
            s = seq_at(a, b);
            p = plan_of(a, s, RB, 0);
            split = 0;
            if (blk >= p.blocks) continue;
        }
        if (lane == 0) odd[wave] = 0;
        const int rows = s.n * a.group, len = positions(a, s);
        int u0, u1;
        attn_range(p.units, p.splits, split, &u0, &u1);
        const int r0 = blk * RB + rw * 16 * MT + c;  // this lane's row of tile 0

        const char* kb = a.c.k + h * a.c.k_head;
        const char* vb = a.c.v + h * a.c.v_head;
        const auto* table = scalar_words(a.table + b * a.ld_table);
        const int lps = a.c.lps, pmask = (1 << lps) - 1;
        const int t_end = min(u1 * U, len);
        const auto page_at = [&](int t) -> int {  // page of position t, -1: none
            if (t >= t_end) return -1;
            const int pg = table[t >> lps];
            return (uint32_t)pg < (uint32_t)a.c.pages ? pg : -1;
        };
        struct Pg {  // pages of the positions of this wave's tiles, sixteen at a time
            int p[NP];
        };
        const auto pages_at = [&](int t) {
            Pg g;
#pragma unroll
            for (int i = 0; i < NP; ++i) g.p[i] = page_at(t + 16 * i);
            return g;
        };
        // The transfers of this wave for the step at t, those from first to last of each tile; rows behind the
        // end or on no page arrive as zeros.
        const auto fetch = [&](int t, const Pg& pg, uint32_t at, int first, int last) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int ch = i * R + rw;
                    const uint32_t to = at + n * L::kBytes + ch * 1024;
                    if (i < first || i >= last) continue;
                    if (ch < L::CK) {
                        const int sub = ch / L::KL, piece = ch % L::KL;
                        const int page = sub ? pg.p[2 * n + 1] : pg.p[2 * n], x = t + 32 * n + 16 * sub;
                        to_lds<ONCE>(rows16(kb + (page < 0 ? 0 : page) * a.c.k_page + (int64_t)(x & pmask) * a.c.k_row + piece * 64,
                                         page < 0 ? 0u : min(16, t_end - x) * a.c.k_row - piece * 64), koff, to);
                    } else {
                        const int row = (ch - L::CK) * L::RP, sub = row >> 4;  // of the tile
                        const int page = sub ? pg.p[2 * n + 1] : pg.p[2 * n], x = t + 32 * n + row;
                        const uint32_t off = (uint32_t)vt * a.c.v_row + (uint32_t)((vp ^ L::mix((row + vt) & 15)) * 16);
                        to_lds<ONCE>(rows16(vb + (page < 0 ? 0 : page) * a.c.v_page + (int64_t)(x & pmask) * a.c.v_row,
                                         page < 0 ? 0u : min(L::RP, max(t_end - x, 0)) * a.c.v_row), off, to);
                    }
                }
        };
        int t0 = u0 * U + 32 * NS * tw;
        const int base = R > 1 ? u0 * U : t0;
        Pg pa = pages_at(t0), pb = pages_at(t0 + STEP), pc = pages_at(t0 + 2 * STEP), pd = pages_at(t0 + 3 * STEP);
        fetch(t0, pa, tile0, 0, NC);
        if constexpr (R == 1 && NB == 2) fetch(t0 + STEP, pb, tile0 + L::kBytes, 0, NC);

        uint64_t mask[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = min(r0 + 16 * m, rows - 1) / a.group;
            mask[m] = a.masks ? a.masks[s.q0 + t] : (2ull << t) - 1;
        }
        // queries: the B operand of S^T (8-bit keys come 16 dims a lane, so 32-dim steps take the dims
        // 64 s + 16 j + 8 half ..)
        u32x4 q[MT][KS];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = r0 + 16 * m;
            const int t = r / a.group, g = r - t * a.group;
            const char* at = static_cast<const char*>(a.q) + ((int64_t)(s.q0 + t) * a.ldq + (int64_t)(h * a.group + g) * D) * 2;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int d = FP8 ? (ks >> 1) * 64 + j * 16 + (ks & 1) * 8 : ks * 32 + j * 8;
                q[m][ks] = r < rows ? *reinterpret_cast<const u32x4*>(at + d * 2) : u32x4{0, 0, 0, 0};
            }
        }
        float ks_scale = 1.f, vs_scale = 1.f;
        if constexpr (FP8) {
            if (a.c.k_scale) ks_scale = a.c.k_scale[h];
            if (a.c.v_scale) vs_scale = a.c.v_scale[h];
        }
        // What the products leave is a score over `unit`, and so are the maxima.
        const int low = lower<TQ>(a.scale * ks_scale);
        const float unit = __builtin_bit_cast(
            float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, ldexpf(a.scale * ks_scale, -low))));
        const float cc = unit * kLog2e;
        int qscale[MT][NG];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if constexpr (kSplit) {
#pragma unroll
                for (int g = 0; g < NG; ++g) qscale[m][g] = split_query(&q[m][4 * g], low);
            } else if constexpr (Half<TQ>::kSplits) {
                const float f = ldexpf(1.f, low);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[m][ks][i] = pack<TQ>(__builtin_bit_cast(float, q[m][ks][i] << 16) * f,
                                               __builtin_bit_cast(float, q[m][ks][i] & 0xffff0000u) * f);
            }
        }

        // The compiler waits for queries and masks here, once, instead of at their first use in the loop, where it
        // would wait for all transfers under way as well.
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            asm volatile("" : "+v"(mask[m]));
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) asm volatile("" : "+v"(q[m][ks]));
        }

        f32x4 o[MT][NE];
        float l[MT];
        f32x4 less[MT];  // -ms
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (!kWide || !again) {
                ms[m] = 0.f;
                lim[m] = kLow;
            }
            l[m] = 0.f;
            less[m] = f32x4{-ms[m], -ms[m], -ms[m], -ms[m]};
#pragma unroll
            for (int e = 0; e < NE; ++e) o[m][e] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // The values of 16 dims turned: lane (c, j) gets dim 16 e + c of the positions 4 j .. of both halves; as
        // they lie, and as operand.
        struct Values {
            u32x2 lo, hi;
        };
        const auto turned = [&](uint32_t at, int e) {
            Values r{};
            if constexpr (FP8) {
                r.lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) i32x2*)(uintptr_t)(at + (vread ^ (uint32_t)(e * 16)))));
            } else {
                const uint32_t x = at + (vread ^ (uint32_t)(e * 32));
                r.lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4*)(uintptr_t)x));
                r.hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4*)(uintptr_t)(x + 16 * L::kRowB)));
            }
            return r;
        };
        const auto operand = [&](const Values& r) -> u32x4 {
            if constexpr (FP8)
                return u32x4{H::from8(r.lo.x, false), H::from8(r.lo.x, true), H::from8(r.lo.y, false), H::from8(r.lo.y, true)};
            else
                return u32x4{r.lo.x, r.lo.y, r.hi.x, r.hi.y};
        };
        // Keys of 16 positions: as many of their dims as one product (two, of widened 8-bit keys) takes.
        constexpr int KU = kSplit ? NG : FP8 ? KS / 2 : KS, NK = 2 * NS * KU;
        struct Keys {
            u32x4 a, b;
        };
        const auto keys = [&](uint32_t at, int i) {
            const int sub = i / KU, u = i % KU;
            const uint32_t from = at + (sub >> 1) * L::kBytes + ((sub & 1) * L::KL + (kSplit ? 2 : 1) * u) * 1024 + lane * 16;
            Keys r{};
            r.a = *lds_at<const u32x4>(from);
            if constexpr (kSplit) r.b = *lds_at<const u32x4>(from + 1024);
            return r;
        };
        const auto scores = [&](uint32_t at, f32x4 (&sc)[MT][2 * NS]) {
            // read ahead of the products, as the values below (with both: eight trees of 64 tokens over 12K
            // positions, 64 heads over 8 of 128 dims, fp16 queries over 8-bit keys 253 -> 235 us)
            constexpr int AHEAD = kSplit || NK < 4 ? 2 : 4;
            static_assert(AHEAD <= NK, "reads stay inside the step");
            Keys raw[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) raw[i] = keys(at, i);
            __builtin_amdgcn_sched_barrier(kNoLds);
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int sub = i / KU, u = i % KU;
                const Keys w = raw[i % AHEAD];
                if (i + AHEAD < NK) raw[i % AHEAD] = keys(at, i + AHEAD);
                __builtin_amdgcn_sched_barrier(kNoLds);
                if (u == 0)
#pragma unroll
                    for (int m = 0; m < MT; ++m) sc[m][sub] = less[m];
                if constexpr (kSplit) {
                    const i32x8 kk = joined(w.a, w.b);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        sc[m][sub] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            kk, joined(q[m][4 * u], q[m][4 * u + 1]), sc[m][sub], 0, 0, 0, kOne8, 0, qscale[m][u]);
                        sc[m][sub] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            kk, joined(q[m][4 * u + 2], q[m][4 * u + 3]), sc[m][sub], 0, 0, 0, kOne8, 1, qscale[m][u]);
                    }
                } else if constexpr (FP8) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t lo = x ? w.a.z : w.a.x, hi = x ? w.a.w : w.a.y;
                        const u32x4 kk = {H::from8(lo, false), H::from8(lo, true), H::from8(hi, false), H::from8(hi, true)};
#pragma unroll
                        for (int m = 0; m < MT; ++m) sc[m][sub] = H::mfma(kk, q[m][2 * u + x], sc[m][sub]);
                    }
                } else {
#pragma unroll
                    for (int m = 0; m < MT; ++m) sc[m][sub] = H::mfma(w.a, q[m][u], sc[m][sub]);
                }
            }
        };
        // Hides from row tile m the positions of the step at t0 that it does not see.
        const auto hide = [&](int m, f32x4 (&sc)[2 * NS]) {
#pragma unroll
            for (int sub = 0; sub < 2 * NS; ++sub) {
                const int x = t0 + 16 * sub + 4 * j;
                const uint32_t there = pa.p[sub] < 0 ? 0u : (1u << min(max(t_end - x, 0), 4)) - 1;
                const uint32_t sees = four_seen(mask[m], x - s.ctx) & there;
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[sub][k] = (sees >> k) & 1 ? sc[sub][k] : -INFINITY;
            }
        };
        // Values of the tree that are not finite become zeros in LDS, so that they do not reach the rows that do
        // not see them as 0 * NaN; `odd` asks for them at the end. (Rows behind the end or on no page are zeros.)
        const auto clean = [&](uint32_t at) {
            bool found = false;
            const int first = max(s.ctx - t0, 0), last = min(t_end - t0, 32 * NS);
            for (int n = first * L::P + rw * 64 + lane; n < last * L::P; n += 64 * R) {
                u32x4* w = lds_at<u32x4>(at + (n / (32 * L::P)) * L::kBytes + L::CK * 1024 + (n % (32 * L::P)) * 16);
                u32x4 y = *w, nf;
#pragma unroll
                for (int k = 0; k < 4; ++k) nf[k] = not_finite<TQ, FP8>(y[k]);
                if (nf[0] | nf[1] | nf[2] | nf[3]) {
                    found = true;
                    *w = y & ~nf;
                }
            }
            if (found) odd[wave] = 1;
        };
        // A tile at LDS address `at`.
        const auto step = [&](uint32_t at, bool whole) {
            f32x4 sc[MT][2 * NS];
            scores(at, sc);
            if constexpr (NB == 1) {  // one tile: its keys make room for the next ones, then its values
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                fetch(t0 + STEP, pb, at, 0, NC / 2);
                wait_loads<NC / 2>();
            }
            if (!whole) {
#pragma unroll
                for (int m = 0; m < MT; ++m) hide(m, sc[m]);
                if (R == 1 && t0 + 32 * NS > s.ctx) clean(at);
            }
            float top[MT];
            bool passed = false;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                top[m] = sc[m][0][0];
#pragma unroll
                for (int k = 1; k < 8 * NS; ++k) top[m] = fmaxf(top[m], sc[m][k >> 2][k & 3]);
                passed |= top[m] > lim[m];
            }
            if (__any(passed)) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    float x = fmaxf(top[m], __shfl_xor(top[m], 16));
                    x = fmaxf(x, __shfl_xor(x, 32));
                    const bool first = lim[m] == kLow;  // the row has seen nothing yet: o and l are 0
                    if (!(first ? x > -INFINITY : x > 0.f)) x = 0.f;
                    else lim[m] = kSlack / cc;
                    const float f = first ? 1.f : __builtin_amdgcn_exp2f(-x * cc);
                    ms[m] += x;
                    less[m] = f32x4{-ms[m], -ms[m], -ms[m], -ms[m]};
                    l[m] *= f;
#pragma unroll
                    for (int e = 0; e < NE; ++e) o[m][e] *= f;
#pragma unroll
                    for (int k = 0; k < 8 * NS; ++k) sc[m][k >> 2][k & 3] -= x;
                }
            }
            // The reads of the first values go out before the weights are computed, each of the others four
            // products ahead (left to itself the compiler waits for every read behind its request: trees of 64
            // tokens over 12K positions, 64 heads over 8, in 8 bits: four of 256 dims 317 us, 258 so; eight of 128
            // dims 238 and 231).
            constexpr int AHEAD = 4, NV = NS * NE;
            static_assert(AHEAD <= NV, "reads stay inside the step");
            Values raw[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) raw[i] = turned(at + i / NE * L::kBytes, i % NE);
            __builtin_amdgcn_sched_barrier(kNoLds);
            u32x4 pf[MT][NS];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    float pr[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        pr[k] = __builtin_amdgcn_exp2f(fmaf(sc[m][2 * n + (k >> 2)][k & 3], cc, kWide ? shift : H::kShift));
                        l[m] += pr[k];
                    }
                    pf[m][n] = u32x4{pack<TQ>(pr[0], pr[1]), pack<TQ>(pr[2], pr[3]), pack<TQ>(pr[4], pr[5]), pack<TQ>(pr[6], pr[7])};
                }
            // This wave goes first while it feeds the matrix cores and the other wave of its SIMD computes
            // weights: 128 rows of 8 bits 626 -> 590 us, of 16 bits 171 -> 163, few rows unchanged.
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const u32x4 v = operand(raw[i % AHEAD]);
                if (i + AHEAD < NV) raw[i % AHEAD] = turned(at + (i + AHEAD) / NE * L::kBytes, (i + AHEAD) % NE);
                __builtin_amdgcn_sched_barrier(kNoLds);
#pragma unroll
                for (int m = 0; m < MT; ++m) o[m][i % NE] = H::mfma(v, pf[m][i / NE], o[m][i % NE]);
            }
            __builtin_amdgcn_s_setprio(0);
        };
        uint32_t at = tile0;
        for (int tb = base; tb < t_end; tb += STEP) {
            const bool whole = t0 + 32 * NS <= s.ctx && t0 + 32 * NS <= t_end && [&] {
                bool all = true;
#pragma unroll
                for (int k = 0; k < 2 * NS; ++k) all &= pa.p[k] >= 0;
                return all;
            }();
            if constexpr (R > 1) {
                // The row waves share their steps and go through the same number of them: when all have met, this
                // step has arrived and the one before it is read, so its place takes the next one.
                wait_loads<0>();
                wait_and_meet();
                const uint32_t next = at == tile0 ? at + NS * L::kBytes : tile0;
                fetch(t0 + STEP, pb, next, 0, NC);
                if (tb + STEP > s.ctx) {  // alike in all waves
                    clean(at);            // each wave a share of its tiles, before any of them is read
                    wait_and_meet();
                }
                if (t0 < t_end) step(at, whole);
                at = next;
            } else {
                wait_loads<(NB > 1 ? NC : NC / 2)>();  // of two tiles under way the older one (one tile: its keys)
                step(at, whole);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if constexpr (NB == 1) {
                    fetch(t0 + STEP, pb, at, NC / 2, NC);
                } else {
                    fetch(t0 + 2 * STEP, pc, at, 0, NC);
                    at = at == tile0 ? at + L::kBytes : tile0;
                }
            }
            t0 += STEP;
            pa = pb;
            pb = pc;
            pc = pd;
            pd = pages_at(t0 + 3 * STEP);  // asked for steps before the transfers need it
        }
        wait_loads<0>();  // what was fetched beyond the end

#pragma unroll
        for (int m = 0; m < MT; ++m) {
            l[m] += __shfl_xor(l[m], 16);
            l[m] += __shfl_xor(l[m], 32);
        }
        // l becomes the sum of 2^((s - mx) log2 e). mx: -INFINITY where nothing was seen.
        float mx[MT];
        const int up = -(int)(kWide ? shift : H::kShift);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            mx[m] = lim[m] == kLow ? -INFINITY : ms[m];
            l[m] = ldexpf(l[m], up);
            if (T > 1 && j == 0) {
                ml[tw][(rw * MT + m) * 16 + c][0] = mx[m];
                ml[tw][(rw * MT + m) * 16 + c][1] = l[m];
            }
        }
        if (kWide && !again) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f};  // NaN where a sum is not finite
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < NE; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = fmaf(o[m][e][i], 0.f, x[i]);
            const float y = (x[0] + x[1]) + (x[2] + x[3]);
            const bool found = __any(y != y);
            if (lane == 0) beyond[wave] = found;
        }
        if (T > 1 || (kWide && !again)) __syncthreads();  // all tiles are read, all transfers done
        if constexpr (kWide) {
            int any = 0;
#pragma unroll
            for (int w = 0; w < R * T; ++w) any |= beyond[w];
            if (any && !again) {
                int e = 1;
#pragma unroll
                for (int m = 0; m < MT; ++m) e = max(e, __builtin_amdgcn_frexp_expf(l[m]));
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) e = max(e, __shfl_xor(e, d));
                // l 2^shift < 1/2: sums stay below half of the largest value
                shift = (float)(-1 - __builtin_amdgcn_readfirstlane(e));
                again = true;
                it -= (int)gridDim.x;
                continue;
            }
            again = false;
            shift = H::kShift;
        }

        // The T waves of each row are brought to the common maximum, the first adds them up, weighted so that all
        // weights' sum is 1 (fold; one wave does that at the store). Lane (c, j) has row c, dims 16 e + 4 j .. + 3.
        float fold[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = (rw * MT + m) * 16 + c;
            float f = 1.f;
            if constexpr (T > 1) {
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < T; ++w) top = fmaxf(top, ml[w][r][0]);
#pragma unroll
                for (int w = 0; w < T; ++w) sum += ml[w][r][1] * weight(ml[w][r][0], top, cc);
                f = weight(mx[m], top, cc);
                mx[m] = top;
                l[m] = sum;
            }
            fold[m] = l[m] > 0.f || l[m] != l[m] ? ldexpf(f, up) / l[m] : 0.f;
            if constexpr (T > 1) {
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    o[m][e] *= fold[m];
                    if (tw > 0) *reinterpret_cast<f32x4*>(o_lds + ((tw - 1) * RB + r) * kRow + 16 * e + 4 * j) = o[m][e];
                }
                fold[m] = 1.f;
            }
        }
        if constexpr (T > 1) __syncthreads();
        if (tw == 0) {
            int odds = 0;
#pragma unroll
            for (int w = 0; w < R * T; ++w) odds |= odd[w];
            odds = __builtin_amdgcn_readfirstlane(odds);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                int rl = (rw * MT + m) * 16 + c;
                asm volatile("" : "+v"(rl));  // addresses from it are not kept through the loops (two instances would spill)
                const int r = blk * RB + rl;
                if (r >= rows) continue;
#pragma unroll
                for (int w = 0; w < T - 1; ++w)
#pragma unroll
                    for (int e = 0; e < NE; ++e) o[m][e] += *reinterpret_cast<const f32x4*>(o_lds + (w * RB + rl) * kRow + 16 * e + 4 * j);
                const int t = r / a.group, hq = h * a.group + (r - t * a.group);
                if (odds) {  // what clean() took out: infinite or NaN for the rows that see it
                    const uint64_t mask = a.masks ? a.masks[s.q0 + t] : (2ull << t) - 1;
                    for (int x = max(s.ctx, u0 * U); x < t_end; ++x) {
                        const int page = page_at(x);
                        if (page < 0 || !((mask >> (x - s.ctx)) & 1)) continue;
                        const char* v = vb + page * a.c.v_page + (int64_t)(x & pmask) * a.c.v_row + 4 * j * L::kElem;
#pragma unroll
                        for (int e = 0; e < NE; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t w;
                                if constexpr (FP8)
                                    w = H::from8(reinterpret_cast<const uint8_t*>(v)[16 * e + i], false) & 0xffffu;
                                else
                                    w = reinterpret_cast<const uint16_t*>(v)[16 * e + i];
                                o[m][e][i] += (w & H::kExp) == H::kExp ? (float)__builtin_bit_cast(TQ, (uint16_t)w) : 0.f;
                            }
                    }
                }
                if (p.splits > 1) {
                    float* to = piece_rows(a, item, RB, D);
#pragma unroll
                    for (int e = 0; e < NE; ++e) *reinterpret_cast<f32x4*>(to + rl * D + 16 * e + 4 * j) = o[m][e] * fold[m];
                    if (j == 0) {
                        to[RB * D + 2 * rl] = mx[m];
                        to[RB * D + 2 * rl + 1] = l[m];
                    }
                    continue;
                }
                TQ* out = static_cast<TQ*>(a.out) + (int64_t)(s.q0 + t) * a.ldo + (int64_t)hq * D + 4 * j;
                const float f = fold[m] * vs_scale;
#pragma unroll
                for (int e = 0; e < NE; ++e)
                    *reinterpret_cast<u32x2*>(out + 16 * e) =
                        u32x2{pack<TQ>(o[m][e][0] * f, o[m][e][1] * f), pack<TQ>(o[m][e][2] * f, o[m][e][3] * f)};
                if (a.lse && j == 0)
                    a.lse[(int64_t)(s.q0 + t) * a.heads + hq] =
                        l[m] == 0.f ? -INFINITY : fmaf(mx[m], unit, __builtin_amdgcn_logf(l[m]) * kLn2);
            }
        }
        __syncthreads();  // the tiles, ml, odd and o_lds are written again by the next piece
    }
}

// Joins the pieces of the sequences that were split: WAVES waves per (token, query head) of a sequence
// and key/value head, in an order that does not depend on timing. Lane s of a wave takes the maximum
// and sum of piece s, so that all pieces' rows are requested at once.
template <typename TQ, int D, int WAVES>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, int rb) {
    constexpr int N = D / 64;
    __shared__ float part[4][D + 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int b = blockIdx.x / a.c.heads, h = blockIdx.x - b * a.c.heads;
    const int r = WAVES == 4 ? (int)blockIdx.y : (int)blockIdx.y * 4 + wave;
    const ScalarWord* head = scalar_words(reinterpret_cast<const int*>(a.ws + a.max_items * rb * (D + 2)));
    const int chunk = head[0], before = head[1 + b];
    const Seq s = seq_at(a, b);
    const Plan p = plan_of(a, s, rb, chunk);
    if (p.splits <= 1 || r >= s.n * a.group) return;
    const int blk = r / rb, rl = r - blk * rb;
    const int first = before + h * p.splits * p.blocks + blk;
    const int s0 = WAVES == 4 ? wave : 0;
    const float scale = a.scale * (a.c.k_scale ? a.c.k_scale[h] : 1.f);
    const float unit = ldexpf(scale, -lower<TQ>(scale)), cc = unit * kLog2e;  // as in k_attn
    float m = -INFINITY, l = 0.f, o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
    for (int k0 = s0; k0 < p.splits; k0 += 64 * WAVES) {
        const int mine = k0 + lane * WAVES, count = min(64, (p.splits - k0 + WAVES - 1) / WAVES);
        float y[8][N];
        const auto request = [&](int k) {  // eight rows
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float* from = piece_rows(a, first + (k0 + min(k + i, count - 1) * WAVES) * p.blocks, rb, D) + rl * D + lane * N;
#pragma unroll
                for (int e = 0; e < N; ++e) y[i][e] = from[e];
            }
        };
        // beside the maxima and sums, not behind them (both launches over 500 positions 13.9 -> 13.6 us, over
        // 4000 positions of 8 trees of 16 tokens 47.6 -> 46.8)
        request(0);
        float mk = -INFINITY, lk = 0.f;
        if (lane < count) {
            const float2 x = *reinterpret_cast<const float2*>(piece_rows(a, first + mine * p.blocks, rb, D) + rb * D + 2 * rl);
            mk = x.x;
            lk = x.y;
        }
        float to = mk;
#pragma unroll
        for (int d = 32; d; d >>= 1) to = fmaxf(to, __shfl_xor(to, d));
        to = fmaxf(to, m);
        // the rows are means, weighted so that the weights' sum is 1: nothing passes the largest of them
        float g = lk * weight(mk, to, cc), sum = g;
#pragma unroll
        for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
        const float was = l * weight(m, to, cc);
        m = to;
        l = was + sum;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        g *= inv;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] *= was * inv;
        for (int k = 0; k < count; k += 8) {
            if (k) request(k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = __shfl(g, (k + i) & 63);
#pragma unroll
                for (int e = 0; e < N; ++e) o[e] = k + i < count ? fmaf(y[i][e], w, o[e]) : o[e];
            }
        }
    }
    if constexpr (WAVES == 4) {
#pragma unroll
        for (int e = 0; e < N; ++e) part[wave][lane * N + e] = o[e];
        if (lane == 0) {
            part[wave][D] = m;
            part[wave][D + 1] = l;
        }
        __syncthreads();
        if (wave != 0) return;
        float top = -INFINITY;
        for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][D]);
        l = 0.f;
        m = top;
        for (int w = 0; w < 4; ++w) l += part[w][D + 1] * weight(part[w][D], top, cc);
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = 0.f;
        for (int w = 0; w < 4; ++w) {
            const float f = part[w][D + 1] * weight(part[w][D], top, cc) * inv;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = fmaf(part[w][lane * N + e], f, o[e]);
        }
    }
    const int t = r / a.group, hq = h * a.group + (r - t * a.group);
    const float vs_scale = a.c.v_scale ? a.c.v_scale[h] : 1.f;
    TQ* out = static_cast<TQ*>(a.out) + (int64_t)(s.q0 + t) * a.ldo + (int64_t)hq * D + lane * N;
#pragma unroll
    for (int e = 0; e < N; ++e) out[e] = (TQ)(o[e] * vs_scale);
    if (a.lse && lane == 0)
        a.lse[(int64_t)(s.q0 + t) * a.heads + hq] = l == 0.f ? -INFINITY : fmaf(m, unit, __builtin_amdgcn_logf(l) * kLn2);
}

template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, bool ONCE>
hipError_t launch(const AttnArgs& a, AttnTile t, hipStream_t s) {
    if (t.tiles != MT || t.row_waves != R) return hipErrorInvalidValue;  // the workspace is cut for this tile
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    const int64_t rows = (int64_t)a.max_tree * a.group, pairs = (int64_t)a.batch * a.c.heads;
    const int64_t most = a.target > 0 ? a.max_items : pairs * cdiv(rows, C::RB);
    const int64_t wgs = most < kCus * C::kPerCu ? cdiv(most, 8) * 8 : kCus * C::kPerCu;
    const unsigned lds = a.target > 0 ? (unsigned)(a.batch + 1) * 4 : 0;
    k_attn<TQ, FP8, D, MT, R, T, NS, NB, ONCE><<<(unsigned)wgs, C::kThreads, lds, s>>>(a);
    if (a.target > 0) {
        // Few rows: many pieces each, four waves share them. Both launches with one wave and with four, 64 heads over
        // 8 of 128 dims: one token over 32K positions 36.7 and 35.1 us, 16 tokens (1024 rows) 49.7 and 49.0, over 2000
        // 20.0 and 20.7; two trees of 16 over 8000 36.9 and 37.3, eight over 1500 36.2 and 46.9. Of 64 and 256 dims alike.
        if (rows * pairs <= 1024)
            k_join<TQ, D, 4><<<dim3((unsigned)pairs, (unsigned)rows), 256, 0, s>>>(a, C::RB);
        else
            k_join<TQ, D, 1><<<dim3((unsigned)pairs, (unsigned)cdiv(rows, 4)), 256, 0, s>>>(a, C::RB);
    }
    return hipGetLastError();
}
template <typename TQ, bool FP8, int D>
hipError_t launch_t(const AttnArgs& a, AttnTile t, hipStream_t s) {
    const bool one_block = a.max_tree * a.group <= attn_rows(t);
    if constexpr (D == 256) {
        // 16 bits: 8 sequences of 16K positions, 4 key/value heads, with NB = 1 96 us, with 2 (one workgroup a CU) 132
        if (t.row_waves == 1) return launch<TQ, FP8, D, 1, 1, 2, 1, FP8 ? 2 : 1, true>(a, t, s);
        return one_block ? launch<TQ, FP8, D, 1, 4, 1, 1, 2, true>(a, t, s) : launch<TQ, FP8, D, 1, 4, 1, 1, 2, false>(a, t, s);
    } else {
        constexpr int NB = FP8 || D == 64 ? 2 : 1;
        if (t.tiles == 1) return launch<TQ, FP8, D, 1, 1, 4, 1, NB, true>(a, t, s);
        if (t.row_waves == 1) return launch<TQ, FP8, D, 2, 1, 4, 1, NB, true>(a, t, s);
        if (t.row_waves == 2) return launch<TQ, FP8, D, 2, 2, 2, 1, 2, true>(a, t, s);
        return one_block ? launch<TQ, FP8, D, 2, 4, 1, 2, 2, true>(a, t, s) : launch<TQ, FP8, D, 2, 4, 1, 2, 2, false>(a, t, s);
    }
}
template <typename TQ, bool FP8>
hipError_t launch_d(const AttnArgs& a, int d, AttnTile t, hipStream_t s) {
    return d == 64    ? launch_t<TQ, FP8, 64>(a, t, s)
           : d == 128 ? launch_t<TQ, FP8, 128>(a, t, s)
                      : launch_t<TQ, FP8, 256>(a, t, s);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, int cache_dtype, int q_dtype, int head_dim, AttnTile t, hipStream_t s) {
    if (q_dtype == UBW_F16)
        return cache_dtype == UBW_E4M3 ? launch_d<h16, true>(a, head_dim, t, s) : launch_d<h16, false>(a, head_dim, t, s);
    return cache_dtype == UBW_E4M3 ? launch_d<b16, true>(a, head_dim, t, s) : launch_d<b16, false>(a, head_dim, t, s);
}

}  // namespace cache
}  // namespace ubw

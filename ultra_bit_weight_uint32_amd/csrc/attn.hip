// Attention of a few new tokens per sequence (one, or a tree of drafted ones) over a paged cache.
//
// For a sequence with context L and n tokens, the rows of a key/value head are its n * G (token,
// query head) pairs. s = scale q k^T over the positions seen, out = softmax(s) v, in one pass over
// the positions with a running maximum m and sum l per row:
//     p_j = 2^(s_j log2 e - m),  l = sum p_j,  o = sum p_j v_j;   a larger m scales l and o down.
//
// A wave takes 32 positions at a time for 16 * MT rows, keys and values straight from memory into
// registers (no LDS, no barrier in the loop):
//   * S^T = K Q^T with v_mfma_f32_16x16x32: a lane loads 16-byte pieces of one key row, which are the
//     A operand as they come; the result leaves lane (row, j) with the positions 4 j .. 4 j + 3 of both
//     16-position halves.
//   * O^T = V^T P^T: those eight weights, packed to 16 bits, are the B operand as they are, if the
//     operand's k index counts positions in that order. For A, lane (c, j) loads D / 16 consecutive
//     dims c D / 16 .. of the same eight positions (16 lanes read a whole row) and eight v_perm per
//     two dims turn the block: product e of a tile then has dim c D / 16 + e in its row c.
//   * m is not followed exactly: o is scaled only when a score passes m + 15 (a wave-uniform branch
//     that long contexts take a few times), so the usual step has no cross-lane work at all, l is kept
//     per lane, and p stays below 2^15, inside fp16. m starts 7 below the maximum, so that weights down
//     to 2^-21 of the largest are normal fp16 numbers.
// All loads are raw buffer loads through descriptors of 16 rows; a descriptor of size 0 stands for
// rows that are not needed or on no valid page, so the loop loads one tile ahead without branches and
// no table entry is ever trusted.
//
// Split over workgroups: the pieces (sequence, head, row block, run of positions) are cut on the
// device from the lengths, about kAttnItems of equal size, and taken by a grid of resident workgroups;
// a piece that is not a whole sequence leaves o, m, l in the workspace and k_join adds them up in order.
//
// Bound: HBM where G n is small (2 (L + n) D values per head read once against 4 G n D operations per
// position); from about 64 rows on the vector unit (exponentials, the turning of V, packing) beside
// the matrix cores.
#include "cache_internal.h"

namespace ubw {
namespace cache {
namespace {

using h16 = _Float16;
using b16 = __bf16;
typedef float f32x4 __attribute__((ext_vector_type(4)));
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
    static __device__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
    static __device__ uint32_t from8(uint32_t w, bool high) {
        return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true)
                                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
    }
};
template <typename T>
__device__ inline uint32_t pack(float a, float b) {  // rounded to nearest even
    typename Half<T>::x2 v;
    v.x = (T)a;
    v.y = (T)b;
    return __builtin_bit_cast(uint32_t, v);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLow = -1e30f;     // m of a row that has seen nothing: 2^(-inf - kLow) = 0
constexpr float kShift = 7.f, kSlack = 8.f;

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
// positions there are: the table ends them
__device__ inline int positions(const AttnArgs& a, const Seq& s) {
    const int64_t most = (int64_t)a.table_cols << a.c.lps;
    return (int)min((int64_t)s.ctx + s.n, most);
}
struct Plan {
    int units, blocks, splits;
};
template <int RB, int U>
__device__ inline Plan plan_of(const AttnArgs& a, const Seq& s, int chunk) {
    Plan p;
    p.blocks = s.n > 0 ? (s.n * a.group + RB - 1) / RB : 0;
    p.units = s.n > 0 ? max(1, (int)(((int64_t)positions(a, s) + U - 1) / U)) : 0;
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

// Sum over the workgroup's 256 threads (every thread gets it). `lds`: 4 words.
__device__ inline int64_t wg_sum(int64_t x, int64_t* lds) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor((long long)x, d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0] + lds[1] + lds[2] + lds[3];
    __syncthreads();
    return x;
}

// Cuts the batch: units per piece, and in pre[b] the number of pieces of the sequences before b.
template <int RB, int U>
__device__ inline int cut_batch(const AttnArgs& a, int* pre, int64_t* lds) {
    const int tid = threadIdx.x;
    const int per = (a.batch + 255) >> 8;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    int64_t units = 0;
    for (int b = b0; b < b1; ++b) {
        const Plan p = plan_of<RB, U>(a, seq_of(a, b), 0);
        units += (int64_t)p.units * p.blocks;
    }
    const int chunk = attn_chunk(wg_sum(units, lds) * a.c.heads, a.target);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const Plan p = plan_of<RB, U>(a, seq_of(a, b), chunk);
        mine += p.splits * p.blocks * a.c.heads;
    }
    int y = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int z = __shfl_up(y, d);
        if ((tid & 63) >= d) y += z;
    }
    int* sums = reinterpret_cast<int*>(lds);
    if ((tid & 63) == 63) sums[tid >> 6] = y;
    __syncthreads();
    int first = y - mine;
    for (int w = 0; w < (tid >> 6); ++w) first += sums[w];
    for (int b = b0; b < b1; ++b) {
        const Plan p = plan_of<RB, U>(a, seq_of(a, b), chunk);
        pre[b] = first;
        first += p.splits * p.blocks * a.c.heads;
    }
    if (tid == 255) pre[a.batch] = first;
    __syncthreads();
    return chunk;
}

// Workspace: pieces' rows of D sums, then (m, l) of each row.
__device__ inline float* piece_rows(const AttnArgs& a, int item, int rb, int d) { return a.ws + (int64_t)item * rb * (d + 2); }

__device__ inline Rsrc rows16(const char* p, uint32_t bytes) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
                       ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), (short)0, (int)__builtin_amdgcn_readfirstlane(bytes),
                                             0x00020000);
}

// One tile's keys and values in registers, as loaded.
template <bool FP8, int D>
struct Tile {
    static constexpr int NV = D / 16;                  // dims a lane has of a value row
    static constexpr int KL = FP8 ? D / 64 : D / 32;   // 16-byte pieces of a key row per lane
    static constexpr int VB = FP8 ? NV : 2 * NV;       // bytes of a value row per lane
    static constexpr int VW = VB / 4;
    u32x4 k[2][KL];
    uint32_t v[8][VW];
    __device__ void load_k(int sub, Rsrc r, uint32_t off) {  // off: the lane's row and 16-byte column
#pragma unroll
        for (int s = 0; s < KL; ++s) {
            const auto x = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(off + s * 64), 0, 0);
            k[sub][s] = __builtin_bit_cast(u32x4, x);
        }
    }
    __device__ void load_v(int sub, Rsrc r, uint32_t off, uint32_t row) {  // off: row 4 j, dims of c
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = off + i * row;
            uint32_t(&w)[VW] = v[sub * 4 + i];
            if constexpr (VB == 4) {
                w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)o, 0, 0);
            } else if constexpr (VB == 8) {
                const auto x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)o, 0, 0));
                w[0] = x.x;
                w[1] = x.y;
            } else {
#pragma unroll
                for (int q = 0; q < VB / 16; ++q) {
                    const auto x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(o + q * 16), 0, 0));
                    w[4 * q] = x.x;
                    w[4 * q + 1] = x.y;
                    w[4 * q + 2] = x.z;
                    w[4 * q + 3] = x.w;
                }
            }
        }
    }
};

template <typename TQ, bool FP8, int D, int MT, int RW>
__global__ __launch_bounds__(256) void k_attn(AttnArgs a) {
    using H = Half<TQ>;
    using T = Tile<FP8, D>;
    constexpr int NV = D / 16, KS = D / 32, TW = 4 / RW, RB = 16 * MT * RW, U = 32 * TW;
    constexpr int kRow = D + 4;  // LDS row of o, in floats
    extern __shared__ char lds_raw[];
    __shared__ int64_t lds64[4];
    __shared__ float ml[TW][RB][2];
    float* o_lds = reinterpret_cast<float*>(lds_raw);                             // [TW - 1][RB][kRow]
    int* pre = reinterpret_cast<int*>(lds_raw + (size_t)(TW - 1) * RB * kRow * 4);  // [batch + 1], with a split

    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % RW, tw = wave / RW;
    const float c2 = a.scale * kLog2e;

    int chunk = 0, items;
    const int blocks_max = (a.max_tree * a.group + RB - 1) / RB;
    if (a.target > 0) {
        chunk = cut_batch<RB, U>(a, pre, lds64);
        items = pre[a.batch];
        if (blockIdx.x == 0) {  // for k_join
            int* head = reinterpret_cast<int*>(a.ws + a.max_items * RB * (D + 2));
            for (int b = threadIdx.x; b < a.batch; b += 256) head[1 + b] = pre[b];
            if (threadIdx.x == 0) head[0] = chunk;
        }
    } else {
        items = a.batch * a.c.heads * blocks_max;
    }

    for (int item = blockIdx.x; item < items; item += gridDim.x) {
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
            s = seq_of(a, b);
            p = plan_of<RB, U>(a, s, chunk);
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
            s = seq_of(a, b);
            p = plan_of<RB, U>(a, s, 0);
            split = 0;
            if (blk >= p.blocks) continue;
        }
        const int rows = s.n * a.group, len = positions(a, s);
        int u0, u1;
        attn_range(p.units, p.splits, split, &u0, &u1);
        const int r0 = blk * RB + rw * 16 * MT + c;  // this lane's row of tile 0

        // queries: the B operand of S^T = K Q^T (8-bit keys come 16 dims a lane, so 32-dim steps take
        // the dims 64 s + 16 j + 8 half ..)
        u32x4 q[MT][KS];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = r0 + 16 * m;
            const int t = r / a.group, g = r - t * a.group;
            const char* at = static_cast<const char*>(a.q) +
                             ((int64_t)(s.q0 + t) * a.ldq + (int64_t)(h * a.group + g) * D) * 2;
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
        const float cc = c2 * ks_scale;

        const char* kb = a.c.k + h * a.c.k_head;
        const char* vb = a.c.v + h * a.c.v_head;
        const int32_t* table = a.table + b * a.ld_table;
        const uint32_t koff = c * a.c.k_row + j * 16;
        const uint32_t voff = 4 * j * a.c.v_row + c * T::VB;
        const int lps = a.c.lps, pmask = (1 << lps) - 1;
        const int t_end = min(u1 * U, len);
        const auto page_at = [&](int t) -> int {  // page of position t, -1: none
            if (t >= t_end) return -1;
            const int pg = table[t >> lps];
            return (uint32_t)pg < (uint32_t)a.c.pages ? pg : -1;
        };
        T x;
        const auto load_k = [&](int t, const int (&pg)[2]) {
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
                x.load_k(sub, rows16(kb + (pg[sub] < 0 ? 0 : pg[sub]) * a.c.k_page + (int64_t)((t + 16 * sub) & pmask) * a.c.k_row,
                                     pg[sub] < 0 ? 0u : 16 * a.c.k_row), koff);
        };
        const auto load_v = [&](int t, const int (&pg)[2]) {
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
                x.load_v(sub, rows16(vb + (pg[sub] < 0 ? 0 : pg[sub]) * a.c.v_page + (int64_t)((t + 16 * sub) & pmask) * a.c.v_row,
                                     pg[sub] < 0 ? 0u : 16 * a.c.v_row), voff, a.c.v_row);
        };

        f32x4 o[MT][NV];
        float mx[MT], l[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            mx[m] = kLow;
            l[m] = 0.f;
#pragma unroll
            for (int e = 0; e < NV; ++e) o[m][e] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        int t0 = u0 * U + 32 * tw;
        int pg[2] = {page_at(t0), page_at(t0 + 16)};
        load_k(t0, pg);
        load_v(t0, pg);
        int pn[2] = {page_at(t0 + U), page_at(t0 + U + 16)};
        for (; t0 < t_end; t0 += U) {
            // scores of 32 positions
            f32x4 sc[MT][2];
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
                for (int m = 0; m < MT; ++m) sc[m][sub] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    u32x4 kk;
                    if constexpr (FP8) {
                        const u32x4 w = x.k[sub][ks >> 1];
                        const uint32_t lo = (ks & 1) ? w.z : w.x, hi = (ks & 1) ? w.w : w.y;
                        kk = u32x4{H::from8(lo, false), H::from8(lo, true), H::from8(hi, false), H::from8(hi, true)};
                    } else {
                        kk = x.k[sub][ks];
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) sc[m][sub] = H::mfma(kk, q[m][ks], sc[m][sub]);
                }
            }
            load_k(t0 + U, pn);

            const bool whole = t0 + 32 <= s.ctx && t0 + 32 <= t_end && pg[0] >= 0 && pg[1] >= 0;
            uint32_t sees[MT];  // bit 4 sub + i: position t0 + 16 sub + 4 j + i (only where !whole)
            if (!whole) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int r = r0 + 16 * m;
                    const int t = min(r, rows - 1) / a.group;
                    const uint64_t mask = a.masks ? a.masks[s.q0 + t] : (2ull << t) - 1;
                    sees[m] = 0;
#pragma unroll
                    for (int sub = 0; sub < 2; ++sub) {
                        const int at = t0 + 16 * sub + 4 * j;
                        const uint32_t there = pg[sub] < 0 ? 0u : (1u << min(max(t_end - at, 0), 4)) - 1;
                        sees[m] |= (four_seen(mask, at - s.ctx) & there) << (4 * sub);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) sc[m][k >> 2][k & 3] = (sees[m] >> k) & 1 ? sc[m][k >> 2][k & 3] : -INFINITY;
                }
            }

            // weights
            bool passed = false;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float top = sc[m][0][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[m][i >> 2][i & 3]);
                passed |= fmaf(top, cc, -mx[m]) > kShift + kSlack;
            }
            if (__any(passed)) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    float top = sc[m][0][0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[m][i >> 2][i & 3]);
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float to = fmaxf(mx[m], fmaf(top, cc, -kShift));
                    const float f = __builtin_amdgcn_exp2f(mx[m] - to);
                    mx[m] = to;
                    l[m] *= f;
#pragma unroll
                    for (int e = 0; e < NV; ++e) o[m][e] *= f;
                }
            }
            u32x4 pf[MT];
            float pr[MT][8];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    pr[m][i] = __builtin_amdgcn_exp2f(fmaf(sc[m][i >> 2][i & 3], cc, -mx[m]));
                    l[m] += pr[m][i];
                }
                pf[m] = u32x4{pack<TQ>(pr[m][0], pr[m][1]), pack<TQ>(pr[m][2], pr[m][3]), pack<TQ>(pr[m][4], pr[m][5]),
                              pack<TQ>(pr[m][6], pr[m][7])};
            }

            // values in 16 bits: w[position][dim pair]
            uint32_t w[8][NV / 2];
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < NV / 2; ++e) {
                    if constexpr (FP8)
                        w[k][e] = H::from8(x.v[k][e >> 1], e & 1);
                    else
                        w[k][e] = x.v[k][e];
                }
            if (!whole) {
                // Rows behind the sequence must not reach the sums even as 0 * NaN. Values of the tree
                // that are not finite are taken out of the product and added by hand to the rows that see
                // them, so that the others stay clean.
                bool odd = false;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int at = t0 + 16 * (k >> 2) + 4 * j + (k & 3);
                    const bool none = at >= t_end, tree = at >= s.ctx;
#pragma unroll
                    for (int e = 0; e < NV / 2; ++e) {
                        w[k][e] = none ? 0u : w[k][e];
                        const bool lo = tree && (w[k][e] & H::kExp) == H::kExp;
                        const bool hi = tree && ((w[k][e] >> 16) & H::kExp) == H::kExp;
                        odd |= lo || hi;
                        w[k][e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                    }
                }
                if (__any(odd)) {
                    for (int k = 0; k < 32; ++k) {  // position t0 + k
                        const int at = t0 + k, sub = k >> 4, slot = 4 * sub + (k & 3), from = ((k >> 2) & 3) * 16 + c;
                        if (at < s.ctx || at >= t_end || pg[sub] < 0) continue;
                        const char* row = vb + (int64_t)pg[sub] * a.c.v_page + (int64_t)(at & pmask) * a.c.v_row;
                        float pk[MT];
                        bool see[MT];
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            float v = pr[m][0];
#pragma unroll
                            for (int i = 1; i < 8; ++i) v = slot == i ? pr[m][i] : v;
                            pk[m] = __shfl(v, from);
                            see[m] = (__shfl((int)sees[m], from) >> slot) & 1;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < NV; ++e) {
                                const int d = (4 * j + i) * NV + e;
                                uint32_t bits;
                                if constexpr (FP8) {
                                    bits = H::from8(*reinterpret_cast<const uint8_t*>(row + d), false) & 0xffffu;
                                } else {
                                    bits = *reinterpret_cast<const uint16_t*>(row + 2 * d);
                                }
                                const float v = (float)__builtin_bit_cast(TQ, (uint16_t)bits);
                                const bool nf = (bits & H::kExp) == H::kExp;
#pragma unroll
                                for (int m = 0; m < MT; ++m) o[m][e][i] = nf && see[m] ? fmaf(pk[m], v, o[m][e][i]) : o[m][e][i];
                            }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;  // high or low halves of two positions
                u32x4 vt;
#pragma unroll
                for (int k = 0; k < 4; ++k) vt[k] = __builtin_amdgcn_perm(w[2 * k + 1][e >> 1], w[2 * k][e >> 1], sel);
#pragma unroll
                for (int m = 0; m < MT; ++m) o[m][e] = H::mfma(vt, pf[m], o[m][e]);
            }
            load_v(t0 + U, pn);
            pg[0] = pn[0];
            pg[1] = pn[1];
            pn[0] = page_at(t0 + 2 * U);
            pn[1] = page_at(t0 + 2 * U + 16);
        }

        // join the position waves, then write: lane (c, j) has row c, dims 4 j NV .. + 4 NV of each tile
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            l[m] += __shfl_xor(l[m], 16);
            l[m] += __shfl_xor(l[m], 32);
        }
        if constexpr (TW > 1) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (j == 0) {
                    ml[tw][(rw * MT + m) * 16 + c][0] = mx[m];
                    ml[tw][(rw * MT + m) * 16 + c][1] = l[m];
                }
            __syncthreads();
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = (rw * MT + m) * 16 + c;
                float top = kLow, sum = 0.f;
#pragma unroll
                for (int w = 0; w < TW; ++w) top = fmaxf(top, ml[w][r][0]);
#pragma unroll
                for (int w = 0; w < TW; ++w) sum += ml[w][r][1] * __builtin_amdgcn_exp2f(ml[w][r][0] - top);
                const float f = __builtin_amdgcn_exp2f(mx[m] - top);
                mx[m] = top;
                l[m] = sum;
#pragma unroll
                for (int e = 0; e < NV; ++e) o[m][e] *= f;
                if (tw > 0) {
                    float* to = o_lds + ((tw - 1) * RB + r) * kRow + 4 * j * NV;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < NV; e += 4)
                            *reinterpret_cast<f32x4*>(to + i * NV + e) = f32x4{o[m][e][i], o[m][e + 1][i], o[m][e + 2][i], o[m][e + 3][i]};
                }
            }
            __syncthreads();
        }
        if (tw == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int rl = (rw * MT + m) * 16 + c, r = blk * RB + rl;
                if (r >= rows) continue;
                if constexpr (TW > 1) {
#pragma unroll
                    for (int w = 0; w < TW - 1; ++w) {
                        const float* from = o_lds + (w * RB + rl) * kRow + 4 * j * NV;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < NV; e += 4) {
                                const f32x4 y = *reinterpret_cast<const f32x4*>(from + i * NV + e);
                                o[m][e][i] += y.x;
                                o[m][e + 1][i] += y.y;
                                o[m][e + 2][i] += y.z;
                                o[m][e + 3][i] += y.w;
                            }
                    }
                }
                if (p.splits > 1) {
                    float* to = piece_rows(a, item, RB, D);
                    float* row = to + rl * D + 4 * j * NV;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < NV; e += 4)
                            *reinterpret_cast<f32x4*>(row + i * NV + e) = f32x4{o[m][e][i], o[m][e + 1][i], o[m][e + 2][i], o[m][e + 3][i]};
                    if (j == 0) {
                        to[RB * D + 2 * rl] = mx[m];
                        to[RB * D + 2 * rl + 1] = l[m];
                    }
                    continue;
                }
                const int t = r / a.group, hq = h * a.group + (r - t * a.group);
                const float inv = l[m] > 0.f || l[m] != l[m] ? vs_scale / l[m] : 0.f;
                TQ* out = static_cast<TQ*>(a.out) + (int64_t)(s.q0 + t) * a.ldo + (int64_t)hq * D + 4 * j * NV;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t y[NV / 2];
#pragma unroll
                    for (int e = 0; e < NV; e += 2) y[e / 2] = pack<TQ>(o[m][e][i] * inv, o[m][e + 1][i] * inv);
#pragma unroll
                    for (int e = 0; e < NV / 2; e += 2)
                        *reinterpret_cast<u32x2*>(out + i * NV + 2 * e) = u32x2{y[e], y[e + 1]};
                }
                if (a.lse && j == 0)
                    a.lse[(int64_t)(s.q0 + t) * a.heads + hq] =
                        l[m] > 0.f || l[m] != l[m] ? (mx[m] + __builtin_amdgcn_logf(l[m])) * kLn2 : -INFINITY;
            }
        }
        if constexpr (TW > 1) __syncthreads();  // ml and o_lds are written again by the next piece
    }
}

// Joins the pieces of the sequences that were split: a workgroup per (token, query head), its waves
// taking every fourth piece, in an order that does not depend on timing.
template <typename TQ, int D>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, int rb, int unit) {
    constexpr int N = D / 64;
    __shared__ float part[4][D + 2];
    const int t = blockIdx.x, hq = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int lo = 0, hi = a.batch;  // the last b with q_start[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = lo;
    const Seq s = seq_of(a, b);
    const int i = t - s.q0;
    if (i < 0 || i >= s.n) return;
    const int* head = reinterpret_cast<const int*>(a.ws + a.max_items * rb * (D + 2));
    const int units = max(1, (int)(((int64_t)positions(a, s) + unit - 1) / unit));
    const int splits = attn_splits(units, head[0]), blocks = (s.n * a.group + rb - 1) / rb;
    if (splits <= 1) return;
    const int h = hq / a.group, r = i * a.group + hq - h * a.group;
    const int blk = r / rb, rl = r - blk * rb;
    const int first = head[1 + b] + h * splits * blocks + blk;
    float m = kLow, l = 0.f, o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int k = wave; k < splits; k += 4) {
        const float* p = piece_rows(a, first + k * blocks, rb, D);
        const float mk = p[rb * D + 2 * rl], lk = p[rb * D + 2 * rl + 1];
        float y[N];
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] = p[rl * D + lane * N + e];
        const float to = fmaxf(m, mk), f = __builtin_amdgcn_exp2f(m - to), g = __builtin_amdgcn_exp2f(mk - to);
        m = to;
        l = l * f + lk * g;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = o[e] * f + y[e] * g;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) part[wave][lane * N + e] = o[e];
    if (lane == 0) {
        part[wave][D] = m;
        part[wave][D + 1] = l;
    }
    __syncthreads();
    if (wave != 0) return;
    float top = kLow;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][D]);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
    for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(part[w][D] - top);
        sum += part[w][D + 1] * f;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += part[w][lane * N + e] * f;
    }
    const bool any = sum > 0.f || sum != sum;
    const float inv = any ? (a.c.v_scale ? a.c.v_scale[h] : 1.f) / sum : 0.f;
    TQ* out = static_cast<TQ*>(a.out) + (int64_t)t * a.ldo + (int64_t)hq * D + lane * N;
#pragma unroll
    for (int e = 0; e < N; ++e) out[e] = (TQ)(o[e] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t)t * a.heads + hq] = any ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
}

template <typename TQ, bool FP8, int D, int MT, int RW>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    constexpr int TW = 4 / RW, RB = 16 * MT * RW;
    const size_t lds = (size_t)(TW - 1) * RB * (D + 4) * 4 + (a.target > 0 ? ((size_t)a.batch + 1) * 4 : 0);
    int64_t wgs = a.target > 0 ? a.max_items
                               : (int64_t)a.batch * a.c.heads * ((a.max_tree * a.group + RB - 1) / RB);
    if (wgs > 2048) wgs = 2048;
    k_attn<TQ, FP8, D, MT, RW><<<(unsigned)wgs, 256, lds, s>>>(a);
    if (a.target > 0) k_join<TQ, D><<<dim3(a.tokens, a.heads), 256, 0, s>>>(a, RB, 32 * TW);
    return hipGetLastError();
}
template <typename TQ, bool FP8, int D>
hipError_t launch_t(const AttnArgs& a, AttnTile t, hipStream_t s) {
    if constexpr (D == 256) {
        return t.row_waves == 1 ? launch<TQ, FP8, D, 1, 1>(a, s) : t.row_waves == 2 ? launch<TQ, FP8, D, 1, 2>(a, s)
                                                                                    : launch<TQ, FP8, D, 1, 4>(a, s);
    } else {
        if (t.tiles == 1) return launch<TQ, FP8, D, 1, 1>(a, s);
        return t.row_waves == 1 ? launch<TQ, FP8, D, 2, 1>(a, s) : t.row_waves == 2 ? launch<TQ, FP8, D, 2, 2>(a, s)
                                                                                    : launch<TQ, FP8, D, 2, 4>(a, s);
    }
}
template <typename TQ, bool FP8>
hipError_t launch_d(const AttnArgs& a, int d, AttnTile t, hipStream_t s) {
    return d == 64 ? launch_t<TQ, FP8, 64>(a, t, s) : d == 128 ? launch_t<TQ, FP8, 128>(a, t, s) : launch_t<TQ, FP8, 256>(a, t, s);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, int cache_dtype, int q_dtype, int head_dim, AttnTile t, hipStream_t s) {
    if (q_dtype == UBW_F16)
        return cache_dtype == UBW_E4M3 ? launch_d<h16, true>(a, head_dim, t, s) : launch_d<h16, false>(a, head_dim, t, s);
    return cache_dtype == UBW_E4M3 ? launch_d<b16, true>(a, head_dim, t, s) : launch_d<b16, false>(a, head_dim, t, s);
}

}  // namespace cache
}  // namespace ubw

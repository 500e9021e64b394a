// Which blocks (pages) of its context a query attends to.
//
// k_bounds: for every dim the smallest and the largest element of a page's keys, lo and hi, in the cache's type (they
// are elements of it, so nothing is rounded).
// k_scores, k_scores_tree: for a token t and key/value head h the score of a block,
//     sum over h's query heads g and dims d of max(q_gd lo_d, q_gd hi_d) = sum_d hi_d up_d + lo_d down_d,
//     up_d = sum_g max(q_gd, 0),  down_d = sum_g min(q_gd, 0),
// which no sum over g of q_g k for a key k of the block passes. The right side costs 2 D products a block, however
// many query heads there are. Sums are 64 bits wide: in 32 bits the order of summing would decide between blocks next to
// the border, in 64 only between those whose scores agree in all but their last bits (sums of queries and products with
// bounds of 16 bits can span more than 53; the order is one for single tokens and another for trees); equal bounds give
// equal scores within a call. The vector unit does them at the rate of 32 bits. Where lo or hi is infinite and its factor 0 the right side is no number, though the left one may be:
// scores that are NaN are taken again without the products with 0.
// k_select, k_select_few: the blocks of the largest scores, ties to the lowest index, by a search on the scores' bits.
#include "cache_internal.h"

namespace ubw {
namespace cache {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) int32_t ScalarWord;
__device__ inline int scalar_word(const int32_t* p, int64_t i) { return ((ScalarWord*)(uintptr_t)p)[i]; }

// 16 bytes of a type as numbers.
template <int DT>
struct Elems;
template <>
struct Elems<UBW_F16> {
    static constexpr int N = 8, kSize = 2;
    static __device__ void read(u32x4 w, float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    }
    static __device__ u32x4 write(const float (&x)[N]) {  // of values of the type
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i]) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]) << 16;
        return w;
    }
};
template <>
struct Elems<UBW_BF16> {
    static constexpr int N = 8, kSize = 2;
    static __device__ void read(u32x4 w, float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        }
    }
    static __device__ u32x4 write(const float (&x)[N]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_bit_cast(uint32_t, x[2 * i]) >> 16 | (__builtin_bit_cast(uint32_t, x[2 * i + 1]) & 0xffff0000u);
        return w;
    }
};
template <>
struct Elems<UBW_E4M3> {
    static constexpr int N = 16, kSize = 1;
    static __device__ void read(u32x4 w, float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
            x[4 * i] = a.x;
            x[4 * i + 1] = a.y;
            x[4 * i + 2] = b.x;
            x[4 * i + 3] = b.y;
        }
    }
    static __device__ u32x4 write(const float (&x)[N]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int y = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
            w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], y, true);
        }
        return w;
    }
};

// ---- bounds
// The smallest and the largest of each of a lane's 16 bytes of elements. A NaN stays one.
template <int DT>
struct Range {
    using E = Elems<DT>;
    float lo[E::N], hi[E::N];
    __device__ void add(u32x4 w, bool first) {
        float x[E::N];
        E::read(w, x);
#pragma unroll
        for (int e = 0; e < E::N; ++e) {
            lo[e] = first ? x[e] : __builtin_elementwise_minimum(lo[e], x[e]);
            hi[e] = first ? x[e] : __builtin_elementwise_maximum(hi[e], x[e]);
        }
    }
    __device__ void write(char* to, int apart) const {
        *reinterpret_cast<u32x4*>(to) = E::write(lo);
        *reinterpret_cast<u32x4*>(to + apart) = E::write(hi);
    }
};
// 8 bits, as whole numbers: with the other seven bits turned where the sign is set they ascend as the numbers do, the
// NaN below and above all others. Bytes are compared in the upper halves of 16 bits, the even ones moved there: 8
// instructions for four, where numbers of 32 bits take 10 (new pages of 36 sequences, 32 heads, 28 layers: 147 MB of 128
// dims 30 us instead of 31, of 256 dims 58 instead of 63).
template <>
struct Range<UBW_E4M3> {
    s16x2 lo[8], hi[8];
    static __device__ uint32_t turned(uint32_t w) {
        return w ^ (__builtin_amdgcn_perm(w, w << 8, 0x0b090a08u) & 0x7f7f7f7fu);  // (the signs, over their bytes)
    }
    static __device__ uint32_t zero_bytes(uint32_t w) { return ~(((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w | 0x7f7f7f7fu); }
    __device__ void add(u32x4 w, bool first) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t t = turned(w[i]);
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                const s16x2 x = __builtin_bit_cast(s16x2, odd ? t : t << 8);
                lo[2 * i + odd] = first ? x : __builtin_elementwise_min(lo[2 * i + odd], x);
                hi[2 * i + odd] = first ? x : __builtin_elementwise_max(hi[2 * i + odd], x);
            }
        }
    }
    static __device__ uint32_t joined(s16x2 even, s16x2 odd) {
        return (__builtin_bit_cast(uint32_t, even) >> 8 & 0x00ff00ffu) | (__builtin_bit_cast(uint32_t, odd) & 0xff00ff00u);
    }
    __device__ void write(char* to, int apart) const {
        u32x4 l, h;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = joined(lo[2 * i], lo[2 * i + 1]), y = joined(hi[2 * i], hi[2 * i + 1]);
            const uint32_t nan = ((zero_bytes(x ^ 0x80808080u) | zero_bytes(y ^ 0x7f7f7f7fu)) >> 7) * 0xffu;
            l[i] = (turned(x) & ~nan) | (nan & 0x7f7f7f7fu);
            h[i] = (turned(y) & ~nan) | (nan & 0x7f7f7f7fu);
        }
        *reinterpret_cast<u32x4*>(to) = l;
        *reinterpret_cast<u32x4*>(to + apart) = h;
    }
};

// As many lanes as a row has 16 bytes go through a page of one head together, each with its own dims, several rows
// requested at once: no lane needs another's. Bound: HBM (pages that 64 sequences filled in 80 layers, 97 MB: 18.2 us, 5.3
// TB/s; a prompt of 50K positions, 435 MB: 78 us, 5.6 TB/s; before rows were requested ahead of the ones in use 91; the same in 8 bits, 218 MB: 44).
template <int DT, int D>
__global__ __launch_bounds__(256) void k_bounds(BoundsArgs a) {
    using E = Elems<DT>;
    constexpr int P = D * E::kSize / 16, kGroups = 256 / P, AHEAD = 8;
    const int b = blockIdx.y, lps = a.c.lps, rows = 1 << lps;
    const int lane = threadIdx.x % P, group = blockIdx.x * kGroups + threadIdx.x / P;
    const int first = max(scalar_word(a.start, b), 0) >> lps, end = min(max(scalar_word(a.stop, b), 0) >> lps, a.table_cols);
    const int each = a.layers * a.c.heads;
    const int64_t all = (int64_t)max(end - first, 0) * each;
    for (int64_t it = group; it < all; it += (int64_t)gridDim.x * kGroups) {
        const int64_t col = it / each;
        const int r = (int)(it - col * each), layer = r / a.c.heads, h = r - layer * a.c.heads;
        const int page = a.table[b * a.ld_table + first + col];
        if ((uint32_t)page >= (uint32_t)a.c.pages) continue;
        const char* k = a.c.k + layer * a.c.k_layer + page * a.c.k_page + h * a.c.k_head + lane * 16;
        Range<DT> range;
        u32x4 w[2 * AHEAD];
#pragma unroll
        for (int i = 0; i < 2 * AHEAD; ++i) w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(k + (int64_t)i * a.c.k_row));
        for (int r0 = 0; r0 < rows; r0 += AHEAD) {
            u32x4 now[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                now[i] = w[i];
                w[i] = w[AHEAD + i];
            }
            if (r0 + 2 * AHEAD < rows) {  // requested before these are looked at
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    w[AHEAD + i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(k + (int64_t)(r0 + 2 * AHEAD + i) * a.c.k_row));
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) range.add(now[i], r0 + i == 0);
        }
        char* to = static_cast<char*>(a.bounds) + (((int64_t)layer * a.c.pages + page) * a.c.heads + h) * (2 * D * E::kSize) + lane * 16;
        range.write(to, D * E::kSize);
    }
}

// ---- scores
struct Rows {
    int q0, n, whole;  // first token, tokens, whole blocks of the context
};
__device__ inline Rows rows_of(const SelectArgs& a, int b) {
    Rows r;
    r.q0 = min(max(scalar_word(a.q_start, b), 0), a.tokens);
    r.n = min(min(max(scalar_word(a.q_start, b + 1), r.q0), a.tokens) - r.q0, a.max_tree);
    r.whole = min(max(scalar_word(a.ctx_len, b), 0) >> a.lps, a.stride);
    return r;
}
template <typename TQ>
__device__ inline float number(uint16_t w) {
    if constexpr (__is_same(TQ, _Float16)) return (float)__builtin_bit_cast(_Float16, w);
    else return __builtin_bit_cast(float, (uint32_t)w << 16);
}
// up and down of one dim of a token and key/value head
template <typename TQ>
__device__ inline void up_down(const SelectArgs& a, int token, int h, int d, int dims, double* up, double* down) {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)token * a.ldq + (int64_t)h * a.group * dims + d;
    double u = 0, v = 0;
#pragma unroll 8
    for (int g = 0; g < a.group; ++g) {
        const float x = number<TQ>(q[(int64_t)g * dims]);
        u += __builtin_elementwise_maximum(x, 0.0f);  // (a NaN in both)
        v += __builtin_elementwise_minimum(x, 0.0f);
    }
    *up = u;
    *down = v;
}
// The same of eight dims; N heads' rows are requested together, those behind the last are zeros.
template <typename TQ, int N>
__device__ inline void add_heads(const uint16_t* q, int heads, int dims, double (&up)[8], double (&down)[8]) {
    u32x4 w[N];
#pragma unroll
    for (int g = 0; g < N; ++g) w[g] = *reinterpret_cast<const u32x4*>(q + (int64_t)min(g, heads - 1) * dims);
#pragma unroll
    for (int g = 0; g < N; ++g) {
        if (g >= heads) w[g] = u32x4{};  // (without a branch, which would keep the loads apart)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = number<TQ>((uint16_t)(w[g][e >> 1] >> (16 * (e & 1))));
            up[e] += __builtin_elementwise_maximum(x, 0.0f);  // (a NaN in both)
            down[e] += __builtin_elementwise_minimum(x, 0.0f);
        }
    }
}
template <typename TQ>
__device__ inline void up_down8(const SelectArgs& a, int token, int h, int d, int dims, double (&up)[8], double (&down)[8]) {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)token * a.ldq + (int64_t)h * a.group * dims + d;
    if (a.group == 1) return add_heads<TQ, 1>(q, 1, dims, up, down);
    for (int g = 0; g < a.group; g += 8) {
        if (a.group - g > 4) add_heads<TQ, 8>(q + (int64_t)g * dims, a.group - g, dims, up, down);
        else add_heads<TQ, 4>(q + (int64_t)g * dims, a.group - g, dims, up, down);
    }
}
// Scores as whole numbers of the same order: a NaN is the largest, both zeros are one, 0 is below all.
__device__ inline uint64_t key_of(double x) {
    const uint64_t w = __builtin_bit_cast(uint64_t, x + 0.0);
    return x != x ? ~0ull : w >> 63 ? ~w : w | 1ull << 63;
}
// A block's score by one lane, without the products whose factor is 0. (Kept out of the loops, whose registers it
// would cost.)
template <int DT, int D, typename F>
__device__ inline double without_zeros(const SelectArgs& a, int64_t page, int h, const F& factor) {
    using E = Elems<DT>;
    const char* at = static_cast<const char*>(a.bounds) + (page * a.kv + h) * (2 * D * E::kSize);
    double sum = 0;
#pragma unroll 1
    for (int i = 0; i < 2 * D; i += E::N) {
        float y[E::N];
        E::read(*reinterpret_cast<const u32x4*>(at + i * E::kSize), y);
#pragma unroll
        for (int e = 0; e < E::N; ++e) {
            const double t = factor(i / D, i % D + e);
            if (t != 0) sum = fma((double)y[e], t, sum);
        }
    }
    return sum;
}
template <int CTRL>
__device__ inline double moved(double x) {
    const uint64_t w = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, 0xf, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over groups of P neighbouring lanes.
template <int P>
__device__ inline double group_sum(double x) {
    x += moved<0xb1>(x);                  // of pairs (quad_perm 1 0 3 2)
    x += moved<0x4e>(x);                  // of fours (2 3 0 1)
    if (P >= 8) x += moved<0x141>(x);     // of eights (mirrored)
    if (P >= 16) x += moved<0x140>(x);    // of sixteens (mirrored)
    if (P >= 32) x += __shfl_xor(x, 16);
    return x;
}

// One token a sequence: a workgroup takes kScoreBlocks blocks of a sequence and head. Bound: HBM or the Infinity Cache,
// with the vector unit busy 61% of the cycles (64 ragged contexts, 251 MB of bounds: 40 us out of the latter, 52 out of memory; workgroups that stay and request ahead,
// or all heads of a block on one XCD, 54 and 58).
template <int DT, typename TQ, int D>
__global__ __launch_bounds__(256) void k_scores(SelectArgs a) {
    using E = Elems<DT>;
    constexpr int P = D * E::kSize / 16, B = 64 / P, STEPS = kScoreBlocks / (4 * B);
    __shared__ double up[D], down[D];
    const int b = blockIdx.y, h = blockIdx.x % a.kv, c0 = blockIdx.x / a.kv * kScoreBlocks;
    const Rows s = rows_of(a, b);
    if (s.n <= 0 || c0 >= s.whole || s.whole <= a.count) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, part = lane % P;
    int page[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int c = c0 + (i * 4 + wave) * B + lane / P;
        page[i] = c < s.whole ? a.table[b * a.ld_table + c] : -1;
    }
    u32x4 lo[STEPS], hi[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t pg = (uint32_t)page[i] < (uint32_t)a.pages ? page[i] : 0;
        const char* at = static_cast<const char*>(a.bounds) + (pg * a.kv + h) * (2 * D * E::kSize) + part * 16;
        lo[i] = *reinterpret_cast<const u32x4*>(at);
        hi[i] = *reinterpret_cast<const u32x4*>(at + D * E::kSize);
    }
    if (threadIdx.x < D) up_down<TQ>(a, s.q0, h, threadIdx.x, D, &up[threadIdx.x], &down[threadIdx.x]);
    __syncthreads();
    double u[E::N], v[E::N];
#pragma unroll
    for (int e = 0; e < E::N; ++e) {
        u[e] = up[part * E::N + e];
        v[e] = down[part * E::N + e];
    }
    double sum[STEPS];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        float x[E::N], y[E::N];
        E::read(lo[i], x);
        E::read(hi[i], y);
        sum[i] = 0;
#pragma unroll
        for (int e = 0; e < E::N; ++e) sum[i] = fma((double)y[e], u[e], fma((double)x[e], v[e], sum[i]));
        sum[i] = group_sum<P>(sum[i]);
        odd = odd || sum[i] != sum[i];
    }
    if (part != 0) return;
    uint64_t* keys = a.keys + ((int64_t)s.q0 * a.kv + h) * a.stride;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int c = c0 + (i * 4 + wave) * B + lane / P;
        const bool ok = (uint32_t)page[i] < (uint32_t)a.pages;
        if (odd && ok) {
            const double again = without_zeros<DT, D>(a, page[i], h, [&](int half, int d) { return half ? up[d] : down[d]; });
            if (sum[i] != sum[i]) sum[i] = again;
        }
        if (c < s.whole) keys[c] = ok ? key_of(sum[i]) : 0;
    }
}

// Trees: 16 blocks x 16 tokens a product of the matrix cores, in 64 bits. A workgroup takes kScoreBlocksTree blocks of
// 16 tokens, its waves two times 16 blocks in turn.
// Lane (c, j) holds of block c the 16-byte pieces j, j + 4, ..; the tokens' sums lie in LDS in the order of the
// products' lanes. Bound: the 64-bit products (8 trees of 16 tokens over 40K to 130K positions, 8 heads, 1.4 GFLOP of
// 78 TFLOP/s: 18 us of 40, the matrix cores busy 56% of them; 3 workgroups on most CUs, 6 us to sum up the queries).
template <int DT, typename TQ, int D>
__global__ __launch_bounds__(256, D == 256 ? 2 : 1) void k_scores_tree(SelectArgs a) {
    using E = Elems<DT>;
    constexpr int S = D / (4 * E::N), TILES = kScoreBlocksTree / 64;
    __shared__ double q[2][S * E::N][64];
    const int b = blockIdx.y, h = blockIdx.x % a.kv, c0 = blockIdx.x / a.kv * kScoreBlocksTree, t0 = blockIdx.z * 16;
    const Rows s = rows_of(a, b);
    if (t0 >= s.n || c0 >= s.whole || s.whole <= a.count) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    for (int i = threadIdx.x; i < 2 * D; i += 256) {  // eight dims of a token
        const int t = i / (D / 8), d = i % (D / 8) * 8, piece = d / E::N;
        double u[8] = {}, v[8] = {};
        if (t0 + t < s.n) up_down8<TQ>(a, s.q0 + t0 + t, h, d, D, u, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = piece / 4 * E::N + (d + e) % E::N, to = piece % 4 * 16 + t;
            q[0][at][to] = v[e];
            q[1][at][to] = u[e];
        }
    }
    __syncthreads();
    const auto put = [&](f64x4 score, int page, int first) {
        const uint64_t all = __ballot(page >= 0);
        if (t0 + c >= s.n) return;
        uint64_t* keys = a.keys + ((int64_t)(s.q0 + t0 + c) * a.kv + h) * a.stride + first;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int x = 4 * r + j;
            double y = score[r];
            if (first + x >= s.whole) continue;
            if (y != y && (all >> x) & 1)
                y = without_zeros<DT, D>(a, a.table[b * a.ld_table + first + x], h, [&](int half, int d) {
                    return q[half][d / E::N / 4 * E::N + d % E::N][d / E::N % 4 * 16 + c];
                });
            keys[x] = (all >> x) & 1 ? key_of(y) : 0;
        }
    };
#pragma unroll 1
    for (int i = 0; i < TILES; i += 2) {  // two tiles at a time share the tokens' sums
        const int first = c0 + (4 * i + 2 * wave) * 16;
        if (first >= s.whole) break;
        int page[2];
        const char* at[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int x = first + 16 * k + c;
            page[k] = x < s.whole ? a.table[b * a.ld_table + x] : -1;
            if ((uint32_t)page[k] >= (uint32_t)a.pages) page[k] = -1;
            at[k] = static_cast<const char*>(a.bounds) + ((int64_t)max(page[k], 0) * a.kv + h) * (2 * D * E::kSize) + j * 16;
        }
        f64x4 sum[2][2] = {};  // of each tile, lower and upper bounds
        u32x4 w[2][2][S];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int n = 0; n < S; ++n) w[k][x][n] = *reinterpret_cast<const u32x4*>(at[k] + x * D * E::kSize + n * 64);
#pragma unroll
        for (int n = 0; n < S; ++n) {
            float y[2][2][E::N];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x) E::read(w[k][x][n], y[k][x]);
#pragma unroll
            for (int e = 0; e < E::N; ++e)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const double t = q[x][n * E::N + e][lane];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        sum[k][x] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)y[k][x][e], t, sum[k][x], 0, 0, 0);
                }
        }
        // lane (t, j) has the blocks j, j + 4, .. of token t
        put(sum[0][0] + sum[0][1], page[0], first);
        put(sum[1][0] + sum[1][1], page[1], first + 16);
    }
}

// ---- the choice
constexpr int kSelThreads = 256, kSelEach = 16, kSelWaves = kSelThreads / 64, kBuckets = 2048;
struct Chosen {
    uint64_t key;
    int at;  // the last block that is in: larger keys are, and this one up to here
};
struct SelectLds {
    int hist[kBuckets];
    uint64_t key[kSelThreads];
    int at[kSelThreads];
    uint64_t ends[2][kSelWaves];
    int sums[kSelEach][kSelWaves];
    int bucket, above, count, listed;
    Chosen last;
};
__device__ inline int wave_before(int x) {  // sum of the lanes before this one
    int y = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int z = __shfl_up(y, d);
        if ((int)(threadIdx.x & 63) >= d) y += z;
    }
    return y - x;
}

// The need-th of the keys keys[0 .. m - 1], m > need > 0, the largest first and of equal ones the lowest index. IN: m
// is at most kSelThreads * kSelEach and a thread keeps its keys.
template <bool IN, typename F>
__device__ inline void each_key(const uint64_t* keys, const uint64_t (&mine)[kSelEach], int m, const F& f) {
    if constexpr (IN) {
#pragma unroll
        for (int r = 0; r < kSelEach; ++r) {
            const int i = r * kSelThreads + threadIdx.x;
            if (i < m) f(i, mine[r]);
        }
    } else {
        for (int i = threadIdx.x; i < m; i += kSelThreads) f(i, keys[i]);
    }
}
template <bool IN>
__device__ inline Chosen find(const uint64_t* keys, const uint64_t (&mine)[kSelEach], int m, int need, SelectLds& l) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t lo = ~0ull, hi = 0;
    each_key<IN>(keys, mine, m, [&](int, uint64_t k) {
        lo = k < lo ? k : lo;
        hi = k > hi ? k : hi;
    });
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t x = __shfl_xor((unsigned long long)lo, d), y = __shfl_xor((unsigned long long)hi, d);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
    }
    if (lane == 0) {
        l.ends[0][wave] = lo;
        l.ends[1][wave] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWaves; ++w) {
        lo = l.ends[0][w] < lo ? l.ends[0][w] : lo;
        hi = l.ends[1][w] > hi ? l.ends[1][w] : hi;
    }
    // Every round looks at the keys in [lo, hi], by 2048 buckets of equal width, and goes on with the bucket that the
    // need-th is in; a last one of up to kSelThreads keys is ranked pair by pair.
    for (;;) {
        const int bits = 64 - __builtin_clzll(hi - lo | 1), shift = bits > 11 ? bits - 11 : 0;
        for (int i = tid; i < kBuckets; i += kSelThreads) l.hist[i] = 0;
        if (tid == 0) l.listed = 0;
        __syncthreads();
        each_key<IN>(keys, mine, m, [&](int, uint64_t k) {
            if (k >= lo && k <= hi) atomicAdd(&l.hist[(int)((k - lo) >> shift)], 1);
        });
        __syncthreads();
        constexpr int PER = kBuckets / kSelThreads;
        int h[PER], sum = 0;  // this thread's buckets, the highest first
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            h[i] = l.hist[kBuckets - 1 - (tid * PER + i)];
            sum += h[i];
        }
        int before = wave_before(sum);
        if (lane == 63) l.sums[0][wave] = before + sum;
        __syncthreads();
        for (int w = 0; w < wave; ++w) before += l.sums[0][w];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < need && need <= before + h[i]) {
                l.bucket = kBuckets - 1 - (tid * PER + i);
                l.above = before;
                l.count = h[i];
            }
            before += h[i];
        }
        __syncthreads();
        const int count = l.count;
        need -= l.above;
        lo += (uint64_t)l.bucket << shift;
        if ((1ull << shift) - 1 < hi - lo) hi = lo + ((1ull << shift) - 1);
        if (count == need) return Chosen{lo, 0x7fffffff};  // all of the bucket
        if (count <= kSelThreads) {
            each_key<IN>(keys, mine, m, [&](int i, uint64_t k) {
                if (k >= lo && k <= hi) {
                    const int x = atomicAdd(&l.listed, 1);
                    l.key[x] = k;
                    l.at[x] = i;
                }
            });
            __syncthreads();
            if (tid < count) {
                const uint64_t k = l.key[tid];
                const int at = l.at[tid];
                int rank = 0;
                for (int i = 0; i < count; ++i) rank += l.key[i] > k || (l.key[i] == k && l.at[i] < at);
                if (rank == need - 1) l.last = Chosen{k, at};
            }
            __syncthreads();
            return l.last;
        }
        if (lo == hi) break;
        __syncthreads();
    }
    // more than kSelThreads equal ones: the need-th by index
    int seen = 0;
    for (int i0 = 0;; i0 += kSelThreads) {  // (m - 1 is reached: there are more than need)
        const int i = i0 + tid;
        const bool is = i < m && keys[i] == lo;
        int before = wave_before(is);
        __syncthreads();
        if (lane == 63) l.sums[0][wave] = before + is;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kSelWaves; ++w) {
            if (w < wave) before += l.sums[0][w];
            all += l.sums[0][w];
        }
        if (is && seen + before == need - 1) l.last = Chosen{lo, i};
        seen += all;
        if (seen >= need || i0 + kSelThreads >= m) break;
    }
    __syncthreads();
    return l.last;
}

// Writes the indices of the keys that are in, ascending.
template <bool IN>
__device__ inline void write_chosen(const uint64_t* keys, const uint64_t (&mine)[kSelEach], int m, Chosen last, int first, int32_t* out,
                                    SelectLds& l) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const auto in = [&](int i, uint64_t k) { return i < m && (k > last.key || (k == last.key && i <= last.at)); };
    if constexpr (IN) {
        int at[kSelEach];
#pragma unroll
        for (int r = 0; r < kSelEach; ++r) {
            const uint64_t b = __ballot(in(r * kSelThreads + tid, mine[r]));
            at[r] = __popcll(b & ((1ull << lane) - 1));
            if (lane == 0) l.sums[r][wave] = __popcll(b);
        }
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int r = 0; r < kSelEach; ++r)
            for (int w = 0; w < kSelWaves; ++w) {
                if (w == wave) at[r] += before;
                before += l.sums[r][w];
            }
#pragma unroll
        for (int r = 0; r < kSelEach; ++r) {
            const int i = r * kSelThreads + tid;
            if (in(i, mine[r])) out[at[r]] = first + i;
        }
    } else {
        int before = 0;
        for (int i0 = 0; i0 < m; i0 += kSelThreads) {
            const int i = i0 + tid;
            const bool is = in(i, i < m ? keys[i] : 0);
            const uint64_t b = __ballot(is);
            __syncthreads();
            if (lane == 0) l.sums[0][wave] = __popcll(b);
            __syncthreads();
            int at = before + __popcll(b & ((1ull << lane) - 1));
            for (int w = 0; w < kSelWaves; ++w) {
                if (w < wave) at += l.sums[0][w];
                before += l.sums[0][w];
            }
            if (is) out[at] = first + i;
        }
    }
}

__global__ __launch_bounds__(kSelThreads) void k_select(SelectArgs a) {
    __shared__ SelectLds l;
    const int tid = threadIdx.x, b = blockIdx.y, h = blockIdx.x % a.kv, i = blockIdx.x / a.kv;
    const Rows s = rows_of(a, b);
    if (i >= s.n) return;
    const int64_t row = (int64_t)(s.q0 + i) * a.kv + h;
    int32_t* out = a.blocks + row * a.count;
    if (s.whole <= a.count) {
        for (int x = tid; x < a.count; x += kSelThreads) out[x] = x < s.whole ? x : -1;
        return;
    }
    for (int x = tid; x < a.first; x += kSelThreads) out[x] = x;
    for (int x = tid; x < a.last; x += kSelThreads) out[a.count - a.last + x] = s.whole - a.last + x;
    const int m = s.whole - a.first - a.last, need = a.count - a.first - a.last;
    if (need <= 0) return;
    const uint64_t* keys = a.keys + row * a.stride + a.first;
    uint64_t mine[kSelEach] = {};
    if (m <= kSelThreads * kSelEach) {
#pragma unroll
        for (int r = 0; r < kSelEach; ++r) {
            const int x = r * kSelThreads + tid;
            if (x < m) mine[r] = keys[x];
        }
        const Chosen last = find<true>(keys, mine, m, need, l);
        __syncthreads();
        write_chosen<true>(keys, mine, m, last, a.first, out + a.first, l);
    } else {
        const Chosen last = find<false>(keys, mine, m, need, l);
        __syncthreads();
        write_chosen<false>(keys, mine, m, last, a.first, out + a.first, l);
    }
}

// Up to 64 R blocks: a wave has a token and head to itself, and finds the need-th key bit by bit, without a barrier. With
// the scores, in us, by this / by k_select; 8 heads, one token, 64 tokens and 64 trees of 16:
//   60 blocks 6.9 / 10.1, 8.7 / 12.3, 27 / 70; 250 blocks 7.9 / 10.3, 19.2 / 21.9, 43 / 83
//   500 blocks 9.6 / 10.3, 30.3 / 30.9, 68 / 104; 1000 blocks 12.7 / 10.5, 52.5 / 50.0, 128 / 157
// so that more than kFewBlocks take it only if there are kManyRows (token, head).
constexpr int kFewBlocks = 512, kManyBlocks = 1024, kManyRows = 4096;
template <int R>
__global__ __launch_bounds__(256) void k_select_few(SelectArgs a) {
    const int lane = threadIdx.x & 63, b = blockIdx.y, x = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const int i = x / a.kv, h = x - i * a.kv;
    const Rows s = rows_of(a, b);
    if (i >= s.n) return;
    const int64_t row = (int64_t)(s.q0 + i) * a.kv + h;
    int32_t* out = a.blocks + row * a.count;
    if (s.whole <= a.count) {
        for (int k = lane; k < a.count; k += 64) out[k] = k < s.whole ? k : -1;
        return;
    }
    for (int k = lane; k < a.first; k += 64) out[k] = k;
    for (int k = lane; k < a.last; k += 64) out[a.count - a.last + k] = s.whole - a.last + k;
    const int m = s.whole - a.first - a.last, need = a.count - a.first - a.last;
    const uint64_t* keys = a.keys + row * a.stride + a.first;
    if (need <= 0) return;
    uint64_t mine[R];
#pragma unroll
    for (int r = 0; r < R; ++r) mine[r] = r * 64 + lane < m ? keys[r * 64 + lane] : 0;
    uint64_t last = 0;  // the largest number that `need` keys reach
    for (int bit = 63; bit >= 0; --bit) {
        const uint64_t k = last | 1ull << bit;
        int count = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) count += __popcll(__ballot(mine[r] >= k));
        if (count >= need) last = k;
        if (count == need) break;  // these are they
    }
    int equal = need;  // of those with this key: the first ones
#pragma unroll
    for (int r = 0; r < R; ++r) equal -= __popcll(__ballot(mine[r] > last));
    const uint64_t below = (1ull << lane) - 1;
    int before = a.first, seen = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool is = r * 64 + lane < m && mine[r] == last;
        const uint64_t same = __ballot(is);
        const bool in = mine[r] > last || (is && seen + __popcll(same & below) < equal);
        const uint64_t all = __ballot(in);
        if (in) out[before + __popcll(all & below)] = a.first + r * 64 + lane;
        seen += __popcll(same);
        before += __popcll(all);
    }
}

template <int DT, int D>
hipError_t bounds_d(const BoundsArgs& a, int64_t pages, hipStream_t s) {
    constexpr int kGroups = 256 / (D * Elems<DT>::kSize / 16);
    k_bounds<DT, D><<<dim3((unsigned)cdiv(bounds_groups(a.layers, a.c.heads, a.batch, pages), kGroups), (unsigned)a.batch), 256, 0, s>>>(a);
    return hipGetLastError();
}
template <int DT>
hipError_t bounds_t(const BoundsArgs& a, int d, int64_t pages, hipStream_t s) {
    return d == 64 ? bounds_d<DT, 64>(a, pages, s) : d == 128 ? bounds_d<DT, 128>(a, pages, s) : bounds_d<DT, 256>(a, pages, s);
}

template <int DT, typename TQ, int D>
hipError_t select_d(const SelectArgs& a, hipStream_t s) {
    if (a.max_tree == 1)
        k_scores<DT, TQ, D><<<dim3((unsigned)(cdiv(a.stride, kScoreBlocks) * a.kv), (unsigned)a.batch), 256, 0, s>>>(a);
    else
        k_scores_tree<DT, TQ, D><<<dim3((unsigned)(cdiv(a.stride, kScoreBlocksTree) * a.kv), (unsigned)a.batch, (unsigned)cdiv(a.max_tree, 16)), 256, 0, s>>>(a);
    const int64_t rows = (int64_t)a.max_tree * a.kv;
    const dim3 few((unsigned)cdiv(rows, 4), (unsigned)a.batch);
    if (a.stride <= 128) k_select_few<2><<<few, 256, 0, s>>>(a);
    else if (a.stride <= 256) k_select_few<4><<<few, 256, 0, s>>>(a);
    else if (a.stride <= kFewBlocks) k_select_few<8><<<few, 256, 0, s>>>(a);
    else if (a.stride <= kManyBlocks && rows * a.batch >= kManyRows) k_select_few<16><<<few, 256, 0, s>>>(a);
    else k_select<<<dim3((unsigned)rows, (unsigned)a.batch), kSelThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <int DT, typename TQ>
hipError_t select_t(const SelectArgs& a, int d, hipStream_t s) {
    return d == 64 ? select_d<DT, TQ, 64>(a, s) : d == 128 ? select_d<DT, TQ, 128>(a, s) : select_d<DT, TQ, 256>(a, s);
}

}  // namespace

hipError_t launch_page_bounds(const BoundsArgs& a, int dtype, int head_dim, int64_t pages, hipStream_t s) {
    return dtype == UBW_F16    ? bounds_t<UBW_F16>(a, head_dim, pages, s)
           : dtype == UBW_BF16 ? bounds_t<UBW_BF16>(a, head_dim, pages, s)
                               : bounds_t<UBW_E4M3>(a, head_dim, pages, s);
}

hipError_t launch_block_select(const SelectArgs& a, int dtype, int q_dtype, int head_dim, hipStream_t s) {
    if (dtype == UBW_F16) return select_t<UBW_F16, _Float16>(a, head_dim, s);
    if (dtype == UBW_BF16) return select_t<UBW_BF16, __bf16>(a, head_dim, s);
    return q_dtype == UBW_F16 ? select_t<UBW_E4M3, _Float16>(a, head_dim, s) : select_t<UBW_E4M3, __bf16>(a, head_dim, s);
}

}  // namespace cache
}  // namespace ubw

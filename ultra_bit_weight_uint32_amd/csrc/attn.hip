// Attention of a few new tokens per sequence (one, or a tree of drafted ones) over a paged cache, in the pieces of
// attn_pieces.h.
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
#include "attn_pieces.h"

namespace ubw {
namespace cache {
namespace {

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

template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, bool ONCE>
__global__ __launch_bounds__((Cfg<FP8, D, MT, R, T, NS, NB>::kThreads), (Cfg<FP8, D, MT, R, T, NS, NB>::kSimd)) void k_attn(AttnArgs a) {
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    constexpr int RB = C::RB;
    extern __shared__ int pre[];  // [batch + 1], with a split
    __shared__ __align__(1024) Shared<C> sh;
    int chunk = 0, items;
    const int blocks_max = (a.max_tree * a.group + RB - 1) / RB;
    if (a.target > 0) {
        chunk = cut_batch<C::kThreads>(a, RB, R == 1, pre, sh.sums);
        items = __builtin_amdgcn_readfirstlane(pre[a.batch]);
        if (blockIdx.x == 0) {  // for k_join
            int* head = reinterpret_cast<int*>(a.ws + a.max_items * RB * (D + 2));
            for (int b = threadIdx.x; b < a.batch; b += C::kThreads) head[1 + b] = pre[b];
            if (threadIdx.x == 0) head[0] = chunk;
        }
    } else {
        items = a.batch * a.c.heads * blocks_max;
    }

    attn_pieces<kTrees, TQ, FP8, D, MT, R, T, NS, NB, ONCE>(a, sh, blockIdx.x, a.ws, [&](int it) { return it < 8 * xcd_share(items); }, [&](int it) { return it + (int)gridDim.x; }, [&](int it, Piece& p) {
        const int item = xcd_item(it, items);
        if (item >= items) return false;
        int b, split;
        Seq s;
        Plan n;
        if (a.target > 0) {
            int lo = 0, hi = a.batch;  // the last b with pre[b] <= item
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid] <= item) lo = mid; else hi = mid;
            }
            b = __builtin_amdgcn_readfirstlane(lo);
            s = seq_at(a, b);
            n = plan_of(a, s, RB, chunk);
            int r = item - __builtin_amdgcn_readfirstlane(pre[b]);
            p.r0 = r % n.blocks * RB;
            r /= n.blocks;
            split = r % n.splits;
            p.h = r / n.splits;
        } else {
            p.r0 = item % blocks_max * RB;
            const int r = item / blocks_max;
            p.h = r % a.c.heads;
            b = r / a.c.heads;
            s = seq_at(a, b);
            n = plan_of(a, s, RB, 0);
            split = 0;
            if (item % blocks_max >= n.blocks) return false;
        }
        attn_range(n.units, n.splits, split, &p.u0, &p.u1);
        p.row = b;
        p.slot = item;
        p.q0 = s.q0;
        p.rows = s.n * a.group;
        p.tree = p.base = 0;
        p.ctx = s.ctx;
        p.len = positions(a, s);
        p.last = n.splits <= 1;
        return true;
    });
}

// Joins the pieces of the sequences that were split: WAVES waves per (token, query head) of a sequence
// and key/value head, in an order that does not depend on timing.
template <typename TQ, int D, int WAVES>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, int rb) {
    __shared__ float part[4][D + 2];
    const int wave = threadIdx.x >> 6;
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
    RowSums<D> x;
    join_row<D, WAVES>(x, piece_rows(a.ws, first, rb, D), (uint32_t)(p.blocks * rb * (D + 2)), p.splits, s0, rb, rl, cc);
    if constexpr (WAVES == 4) {
        if (!join_waves<D, WAVES>(x, part, cc)) return;
    }
    const int t = r / a.group;
    store_row<TQ, D>(a, x, s.q0 + t, h, r - t * a.group, unit);
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

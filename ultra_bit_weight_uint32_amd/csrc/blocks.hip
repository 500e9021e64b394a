// Attention of each token over blocks (pages) of its context that a list names, for every key/value head one: the
// rows of a piece are the head's queries of one token, its positions those of the list's blocks one behind the
// other, then the page where the context ends and the tree behind it, which are always seen. To the loop over
// positions (attn_pieces.h) that is a context like any other; only the page of a position takes two loads.
// A list ends at its first entry that does not ascend or is no whole block of the context, so that no block counts
// twice and no entry is trusted.
//
// Pieces are numbered head by head, then by the run of positions, tokens side by side: those of one tree, which
// share most of their blocks, run at the same time on one XCD and meet in its L2.
//
// Bound: single tokens of a batch the memory (64 ragged contexts, 64 blocks of 32 positions each, bf16: 86 us, 5.9
// TB/s), one token alone the chain list -> table -> keys -> values -> join (9.6 and 4.1 us, 13.1 in a queue), trees the issue of a
// step, whose 16-row tile a token of 8 query heads fills by half (8 trees of 16 over 64 blocks of 64 positions in 8 bits
// 95 us, 11 TB/s out of the L2).
#include "attn_pieces.h"

namespace ubw {
namespace cache {
namespace {

template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, bool ONCE>
__global__ __launch_bounds__((Cfg<FP8, D, MT, R, T, NS, NB>::kThreads), (Cfg<FP8, D, MT, R, T, NS, NB>::kSimd)) void k_blocks(BlockArgs a) {
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    constexpr int RB = C::RB;
    __shared__ __align__(1024) Shared<C> sh;
    const int blocks = (a.group + RB - 1) / RB, lane = threadIdx.x & 63;
    const int items = a.tokens * a.splits * blocks * a.c.heads;
    attn_pieces<kBlocks, TQ, FP8, D, MT, R, T, NS, NB, ONCE>(a, sh, blockIdx.x, a.ws, [&](int it) { return it < 8 * xcd_share(items); }, [&](int it) { return it + (int)gridDim.x; }, [&](int it, Piece& p) {
        const int item = xcd_item(it, items);
        if (item >= items) return false;
        int r = item / a.tokens;
        const int token = item - r * a.tokens;
        const int split = r % a.splits;
        r /= a.splits;
        p.r0 = r % blocks * RB;
        p.h = r / blocks;
        const int b = find_last(a.q_start, a.batch, token);
        const Seq s = seq_at(a, b);
        if (token < s.q0 || token >= s.q0 + s.n) return false;
        p.whole = s.ctx >> a.c.lps;
        p.list = a.blocks + ((int64_t)token * a.c.heads + p.h) * a.count;
        const int most = min(p.whole, a.table_cols);
        p.chosen = a.count;
        for (int i0 = 0; i0 < a.count; i0 += 64) {
            const int i = i0 + lane;
            const int x = i < a.count ? p.list[i] : -1, y = i > 0 && i < a.count ? p.list[i - 1] : -1;
            const uint64_t ends = __ballot(x <= y || x >= most);
            if (ends) {
                p.chosen = i0 + __builtin_ctzll(ends);
                break;
            }
        }
        p.chosen = __builtin_amdgcn_readfirstlane(p.chosen);
        p.row = b;
        p.q0 = token;
        p.rows = a.group;
        p.tree = token - s.q0;
        p.base = 0;
        p.ctx = (p.chosen << a.c.lps) + (s.ctx & ((1 << a.c.lps) - 1));
        p.len = p.ctx + s.n;
        const int units = units_of(p.len);
        const int splits = min(units, a.splits);
        if (a.splits > 1 && split == 0 && p.r0 == 0 && threadIdx.x == 0) a.cut[p.h * a.tokens + token] = splits;
        if (split >= splits) return false;
        attn_range(units, splits, split, &p.u0, &p.u1);
        p.slot = item;
        p.last = splits <= 1;
        return true;
    });
}

template <typename TQ, int D, int WAVES>
__global__ __launch_bounds__(256) void k_join_blocks(BlockArgs a, int rb) {
    __shared__ float part[4][D + 2];
    const int wave = threadIdx.x >> 6;
    const int h = blockIdx.x / a.tokens, token = blockIdx.x - h * a.tokens;
    const int r = WAVES == 4 ? (int)blockIdx.y : (int)blockIdx.y * 4 + wave;
    if (r >= a.group) return;
    const Seq s = seq_at(a, find_last(a.q_start, a.batch, token));
    if (token < s.q0 || token >= s.q0 + s.n) return;
    const int pieces = scalar_words(a.cut)[h * a.tokens + token], blocks = (a.group + rb - 1) / rb;
    if (pieces <= 1) return;
    const float scale = a.scale * (a.c.k_scale ? a.c.k_scale[h] : 1.f);
    const float unit = ldexpf(scale, -lower<TQ>(scale)), cc = unit * kLog2e;  // as in attn_pieces
    RowSums<D> x;
    join_row<D, WAVES>(x, piece_rows(a.ws, ((h * blocks + r / rb) * a.splits) * a.tokens + token, rb, D),
                       (uint32_t)(a.tokens * rb * (D + 2)), pieces, WAVES == 4 ? wave : 0, rb, r % rb, cc);
    if constexpr (WAVES == 4) {
        if (!join_waves<D, WAVES>(x, part, cc)) return;
    }
    store_row<TQ, D>(a, x, token, h, r, unit);
}

template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, bool ONCE>
hipError_t launch(const BlockArgs& a, hipStream_t s) {
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    const int64_t most = (int64_t)a.tokens * a.splits * cdiv(a.group, C::RB) * a.c.heads;
    const int64_t wgs = most < kCus * C::kPerCu ? cdiv(most, 8) * 8 : kCus * C::kPerCu;
    k_blocks<TQ, FP8, D, MT, R, T, NS, NB, ONCE><<<(unsigned)wgs, C::kThreads, 0, s>>>(a);
    if (a.splits > 1) {
        const int64_t pairs = (int64_t)a.tokens * a.c.heads;
        if (a.group * pairs <= 1024)
            k_join_blocks<TQ, D, 4><<<dim3((unsigned)pairs, (unsigned)a.group), 256, 0, s>>>(a, C::RB);
        else
            k_join_blocks<TQ, D, 1><<<dim3((unsigned)pairs, (unsigned)cdiv(a.group, 4)), 256, 0, s>>>(a, C::RB);
    }
    return hipGetLastError();
}
template <typename TQ, bool FP8, int D>
hipError_t launch_t(const BlockArgs& a, hipStream_t s) {
    const bool few = attn_rows(block_tile(a.group, D)) == 16;
    // 16 rows: one tile of keys and values a wave, refilled in place, and so three workgroups a CU (with two tiles and two
    // workgroups eight trees of 16 over 64 blocks of 64 positions in 8 bits take 100 us instead of 95). Where a sequence
    // has one token its blocks are read once, past the L2.
    constexpr int T = D == 256 ? 2 : 4;
    if (few) return a.max_tree == 1 ? launch<TQ, FP8, D, 1, 1, T, 1, 1, true>(a, s) : launch<TQ, FP8, D, 1, 1, T, 1, 1, false>(a, s);
    return launch<TQ, FP8, D, D == 256 ? 1 : 2, 4, 1, D == 256 ? 1 : 2, 2, false>(a, s);
}
template <typename TQ, bool FP8>
hipError_t launch_d(const BlockArgs& a, int d, hipStream_t s) {
    return d == 64 ? launch_t<TQ, FP8, 64>(a, s) : d == 128 ? launch_t<TQ, FP8, 128>(a, s) : launch_t<TQ, FP8, 256>(a, s);
}

}  // namespace

hipError_t launch_block_attn(const BlockArgs& a, int cache_dtype, int q_dtype, int head_dim, hipStream_t s) {
    if (q_dtype == UBW_F16)
        return cache_dtype == UBW_E4M3 ? launch_d<h16, true>(a, head_dim, s) : launch_d<h16, false>(a, head_dim, s);
    return cache_dtype == UBW_E4M3 ? launch_d<b16, true>(a, head_dim, s) : launch_d<b16, false>(a, head_dim, s);
}

}  // namespace cache
}  // namespace ubw

// Attention of each sequence's new tokens over its context, where sequences have the beginning of it in common:
// a group's prefix is gone through once, with the rows of all its sequences side by side, and each sequence's
// own positions behind it as in tree attention. With the sums of both parts, m the maximum and l the sum of
// 2^((s - m) log2 e) over a part's positions, o their weighted mean,
//     out = sum_parts l_i 2^((m_i - m) log2 e) o_i / sum_parts l_i 2^((m_i - m) log2 e),  m = max m_i.
//
// Three launches: k_plan (one workgroup) measures the groups, cuts both lists into pieces (attn_pieces.h) and
// leaves the plan in the workspace; k_prefix goes through them; k_join_parts joins each row's.
//   * A prefix ends at a multiple of 16 positions, so that no tile has positions of both parts; the few behind
//     it are each sequence's own (its own row of the table has them too).
//   * A prefix passes the shortest context of its group nowhere, so that a sequence never sees what is not its own.
#include "attn_pieces.h"

namespace ubw {
namespace cache {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMost = UBW_MAX_SEQS, kEach = kMost / kPlanThreads;

// The plan's arrays. Groups: first piece (and the end of the list), positions, table row, first token, rows, pieces a
// row's positions are cut into. Sequences: first piece (and the end), base, group, pieces.
struct PlanAt {
    int *head, *g_first, *g_len, *g_row, *g_q0, *g_rows, *g_splits, *s_first, *s_base, *s_group, *s_splits;
};
__device__ __host__ inline PlanAt plan_at(int* p, int groups, int batch) {
    PlanAt x;
    x.head = p;
    x.g_first = p + kPlanHead;
    x.g_len = x.g_first + groups + 1;
    x.g_row = x.g_len + groups + 1;
    x.g_q0 = x.g_row + groups + 1;
    x.g_rows = x.g_q0 + groups + 1;
    x.g_splits = x.g_rows + groups + 1;
    x.s_first = x.g_splits + groups + 1;
    x.s_base = x.s_first + batch + 1;
    x.s_group = x.s_base + batch + 1;
    x.s_splits = x.s_group + batch + 1;
    return x;
}

// Sums of two numbers over the workgroup, for every thread.
struct Two {
    int64_t a, b;
};
__device__ inline Two plan_sum(Two x, int64_t (&lds)[2][kPlanThreads / 64]) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        x.a += __shfl_xor((long long)x.a, d);
        x.b += __shfl_xor((long long)x.b, d);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        lds[0][threadIdx.x >> 6] = x.a;
        lds[1][threadIdx.x >> 6] = x.b;
    }
    __syncthreads();
    Two s{0, 0};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        s.a += lds[0][w];
        s.b += lds[1][w];
    }
    return s;
}
// Sums of the threads before this one.
__device__ inline Two plan_before(Two mine, int64_t (&lds)[2][kPlanThreads / 64]) {
    Two y = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t u = __shfl_up((long long)y.a, d), v = __shfl_up((long long)y.b, d);
        if ((int)(threadIdx.x & 63) >= d) {
            y.a += u;
            y.b += v;
        }
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) {
        lds[0][threadIdx.x >> 6] = y.a;
        lds[1][threadIdx.x >> 6] = y.b;
    }
    __syncthreads();
    Two s{y.a - mine.a, y.b - mine.b};
    for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) {
        s.a += lds[0][w];
        s.b += lds[1][w];
    }
    return s;
}
// A thread has the groups and the sequences kEach t .. kEach t + kEach - 1.
__global__ __launch_bounds__(kPlanThreads) void k_plan(PrefixArgs a, bool one_row_wave) {
    __shared__ int start[kMost + 1], len[kMost], lead[kMost], last[kMost];
    __shared__ int64_t lds[2][kPlanThreads / 64];
    const int tid = threadIdx.x, kv = a.c.heads;
    const PlanAt at = plan_at(a.plan, a.groups, a.batch);
    const int per_g = (a.groups + kPlanThreads - 1) / kPlanThreads, per_s = (a.batch + kPlanThreads - 1) / kPlanThreads;
    const int most = (int)min((int64_t)a.table_cols << a.c.lps, (int64_t)1 << 30);
    for (int g = tid; a.groups > 0 && g <= a.groups; g += kPlanThreads) {
        start[g] = min(max(a.group_start[g], 0), a.batch);
        if (g < a.groups) {
            len[g] = min(max(a.prefix_len[g], 0), most);
            lead[g] = kMost;
            last[g] = -1;
        }
    }
    Seq s[kEach];
    int of[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int b = tid * per_s + i;
        s[i] = i < per_s && b < a.batch ? seq_of(a, b) : Seq{0, 0, 0};
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int b = tid * per_s + i;
        of[i] = -1;
        if (s[i].n <= 0 || a.groups == 0) continue;
        int lo = 0, hi = a.groups;  // the last group that begins at b or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= b) lo = mid; else hi = mid;
        }
        if (start[lo] > b || b >= start[lo + 1]) continue;
        of[i] = lo;
        atomicMin(&len[lo], s[i].ctx);
        atomicMin(&lead[lo], b);
        atomicMax(&last[lo], b);
    }
    __syncthreads();

    int g_units[kEach], g_blocks[kEach];
    Two sum{0, 0};  // units, blocks of the groups
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = tid * per_g + i;
        g_units[i] = g_blocks[i] = 0;
        if (i >= per_g || g >= a.groups) continue;
        const int q0 = min(max(a.q_start[start[g]], 0), a.tokens);
        const int q1 = min(max(a.q_start[max(start[g + 1], start[g])], q0), a.tokens);
        const int rows = (q1 - q0) * a.group;
        const int n = last[g] > lead[g] && rows > 0 ? len[g] & ~15 : 0;  // one sequence alone shares nothing
        g_units[i] = units_of(n);
        g_blocks[i] = n > 0 ? (rows + a.z.rb_shared - 1) / a.z.rb_shared : 0;
        len[g] = n;
        at.g_len[g] = n;
        at.g_row[g] = min(lead[g], a.batch - 1);
        at.g_q0[g] = q0;
        at.g_rows[g] = rows;
        sum.a += (int64_t)g_units[i] * g_blocks[i] * kv;
        sum.b += (int64_t)g_blocks[i] * kv;
    }
    sum = plan_sum(sum, lds);  // (its barriers stand before the others read len)
    // q_start does not ascend: the groups would have more rows than there are, nothing is shared
    const bool none = sum.b > a.z.blocks_shared;
    int s_units[kEach], s_blocks[kEach], base[kEach];
    Two units{none ? 0 : sum.a, 0};
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (none) g_units[i] = g_blocks[i] = 0;
        base[i] = of[i] >= 0 && !none ? len[of[i]] : 0;
        s_blocks[i] = s[i].n > 0 ? (s[i].n * a.group + a.z.rb_own - 1) / a.z.rb_own : 0;
        s_units[i] = s[i].n > 0 ? max(1, units_of(positions(a, s[i]) - base[i])) : 0;
        units.b += (int64_t)s_units[i] * s_blocks[i] * kv;
    }
    units.b = plan_sum(Two{0, units.b}, lds).b;
    const int goal_s = a.z.target_shared, goal_o = attn_aim(units.b, a.z.target_own, one_row_wave);
    int chunk_s = attn_chunk(units.a, goal_s), chunk_o = attn_chunk(units.b, goal_o);
    Two mine;
    for (int step = 0;; ++step) {
        mine = Two{0, 0};
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            mine.a += (int64_t)attn_splits(g_units[i], chunk_s) * g_blocks[i] * kv;
            mine.b += (int64_t)attn_splits(s_units[i], chunk_o) * s_blocks[i] * kv;
        }
        const Two all = plan_sum(mine, lds);
        const bool fits_s = all.a <= goal_s, fits_o = all.b <= goal_o;
        if (step == 4 || (fits_s && fits_o)) break;
        if (!fits_s) chunk_s = attn_larger_chunk(chunk_s, all.a, goal_s);
        if (!fits_o) chunk_o = attn_larger_chunk(chunk_o, all.b, goal_o);
    }
    const Two before = plan_before(mine, lds);
    int first = (int)before.a;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = tid * per_g + i;
        if (i >= per_g || g >= a.groups) continue;
        const int splits = attn_splits(g_units[i], chunk_s);
        at.g_first[g] = first;
        at.g_splits[g] = splits;
        first += splits * g_blocks[i] * kv;
    }
    int own = (int)before.b;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int b = tid * per_s + i;
        if (i >= per_s || b >= a.batch) continue;
        const int splits = attn_splits(s_units[i], chunk_o);
        at.s_first[b] = own;
        at.s_splits[b] = splits;
        at.s_base[b] = base[i];
        at.s_group[b] = base[i] > 0 ? of[i] : -1;
        own += splits * s_blocks[i] * kv;
    }
    if (tid == kPlanThreads - 1) {
        at.head[0] = first;
        at.head[1] = own;
    }
}

// PART: 1 the prefixes, 2 what is behind them.
template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, int PART>
__global__ __launch_bounds__((Cfg<FP8, D, MT, R, T, NS, NB>::kThreads), (Cfg<FP8, D, MT, R, T, NS, NB>::kSimd)) void k_prefix(PrefixArgs a) {
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    constexpr int RB = C::RB;
    __shared__ __align__(1024) Shared<C> sh;
    const PlanAt at = plan_at(a.plan, a.groups, a.batch);
    if constexpr (PART == 1)
        attn_pieces<kShared, TQ, FP8, D, MT, R, T, NS, NB, false>(a, sh, scalar_words(at.head)[0], a.ws, [&](int item, Piece& p) {
            const int g = find_last(at.g_first, a.groups, item);
            const int rows = scalar_words(at.g_rows)[g], splits = scalar_words(at.g_splits)[g], blocks = (rows + RB - 1) / RB;
            int r = item - scalar_words(at.g_first)[g];
            p.blk = r % blocks;
            r /= blocks;
            p.h = r / splits;
            p.row = scalar_words(at.g_row)[g];
            p.q0 = scalar_words(at.g_q0)[g];
            p.rows = rows;
            p.splits = splits;
            p.ctx = p.len = scalar_words(at.g_len)[g];
            attn_range(units_of(p.len), splits, r % splits, &p.u0, &p.u1);
            p.tree = p.base = 0;
            p.last = false;
            return true;
        });
    else
        attn_pieces<kOwn, TQ, FP8, D, MT, R, T, NS, NB, (R == 1)>(a, sh, scalar_words(at.head)[1], a.ws + a.own_at, [&](int item, Piece& p) {
            const int b = find_last(at.s_first, a.batch, item);
            const Seq s = seq_at(a, b);
            const int splits = scalar_words(at.s_splits)[b], blocks = (s.n * a.group + RB - 1) / RB;
            int r = item - scalar_words(at.s_first)[b];
            p.blk = r % blocks;
            r /= blocks;
            p.h = r / splits;
            p.row = b;
            p.q0 = s.q0;
            p.rows = s.n * a.group;
            p.splits = splits;
            p.ctx = s.ctx;
            p.len = positions(a, s);
            p.base = scalar_words(at.s_base)[b];
            p.tree = 0;
            attn_range(max(1, units_of(p.len - p.base)), splits, r % splits, &p.u0, &p.u1);
            p.last = splits <= 1 && p.base == 0;
            return true;
        });
}

// Joins the pieces of the prefix and of what is behind it, WAVES waves per (token, query head), in an order that
// does not depend on timing.
template <typename TQ, int D, int WAVES>
__global__ __launch_bounds__(256) void k_join_parts(PrefixArgs a) {
    __shared__ float part[4][D + 2];
    const int wave = threadIdx.x >> 6;
    const int b = blockIdx.x / a.c.heads, h = blockIdx.x - b * a.c.heads;
    const int r = WAVES == 4 ? (int)blockIdx.y : (int)blockIdx.y * 4 + wave;
    const PlanAt at = plan_at(a.plan, a.groups, a.batch);
    const Seq s = seq_at(a, b);
    const int own = scalar_words(at.s_splits)[b], g = scalar_words(at.s_group)[b];
    if ((own <= 1 && g < 0) || r >= s.n * a.group) return;
    const int s0 = WAVES == 4 ? wave : 0;
    const float scale = a.scale * (a.c.k_scale ? a.c.k_scale[h] : 1.f);
    const float unit = ldexpf(scale, -lower<TQ>(scale)), cc = unit * kLog2e;  // as in attn_pieces
    RowSums<D> x;
    if (g >= 0) {
        const int rows = scalar_words(at.g_rows)[g], splits = scalar_words(at.g_splits)[g], rb = a.z.rb_shared;
        const int rp = (s.q0 - scalar_words(at.g_q0)[g]) * a.group + r, blocks = (rows + rb - 1) / rb;
        if (rp >= 0 && rp < rows)
            join_row<D, WAVES>(x, piece_rows(a.ws, scalar_words(at.g_first)[g] + h * splits * blocks + rp / rb, rb, D),
                               (uint32_t)(blocks * rb * (D + 2)), splits, s0, rb, rp % rb, cc);
    }
    const int rb = a.z.rb_own, blocks = (s.n * a.group + rb - 1) / rb;
    join_row<D, WAVES>(x, piece_rows(a.ws + a.own_at, scalar_words(at.s_first)[b] + h * own * blocks + r / rb, rb, D),
                       (uint32_t)(blocks * rb * (D + 2)), own, s0, rb, r % rb, cc);
    if constexpr (WAVES == 4) {
        if (!join_waves<D, WAVES>(x, part, cc)) return;
    }
    const int t = r / a.group;
    store_row<TQ, D>(a, x, s.q0 + t, h, r - t * a.group, unit);
}

template <typename TQ, bool FP8, int D, int MT, int R, int T, int NS, int NB, int PART>
void launch_part(const PrefixArgs& a, int64_t most, hipStream_t s) {
    using C = Cfg<FP8, D, MT, R, T, NS, NB>;
    const int64_t wgs = most < kCus * C::kPerCu ? cdiv(most, 8) * 8 : kCus * C::kPerCu;
    k_prefix<TQ, FP8, D, MT, R, T, NS, NB, PART><<<(unsigned)wgs, C::kThreads, 0, s>>>(a);
}
template <typename TQ, bool FP8, int D>
hipError_t launch_t(const PrefixArgs& a, hipStream_t s) {
    const bool few = a.z.rb_own == 16;
    k_plan<<<1, kPlanThreads, 0, s>>>(a, few);
    if constexpr (D == 256) {
        if (a.groups > 0) launch_part<TQ, FP8, D, 1, 4, 1, 1, 2, 1>(a, a.z.cap_shared, s);
        if (few) launch_part<TQ, FP8, D, 1, 1, 2, 1, FP8 ? 2 : 1, 2>(a, a.z.cap_own, s);
        else launch_part<TQ, FP8, D, 1, 4, 1, 1, 2, 2>(a, a.z.cap_own, s);
    } else {
        if (a.groups > 0) launch_part<TQ, FP8, D, 2, 4, 1, 2, 2, 1>(a, a.z.cap_shared, s);
        if (few) launch_part<TQ, FP8, D, 1, 1, 4, 1, FP8 || D == 64 ? 2 : 1, 2>(a, a.z.cap_own, s);
        else launch_part<TQ, FP8, D, 2, 4, 1, 2, 2, 2>(a, a.z.cap_own, s);
    }
    const int64_t rows = (int64_t)a.max_tree * a.group, pairs = (int64_t)a.batch * a.c.heads;
    if (rows * pairs <= 1024)
        k_join_parts<TQ, D, 4><<<dim3((unsigned)pairs, (unsigned)rows), 256, 0, s>>>(a);
    else
        k_join_parts<TQ, D, 1><<<dim3((unsigned)pairs, (unsigned)cdiv(rows, 4)), 256, 0, s>>>(a);
    return hipGetLastError();
}
template <typename TQ, bool FP8>
hipError_t launch_d(const PrefixArgs& a, int d, hipStream_t s) {
    return d == 64 ? launch_t<TQ, FP8, 64>(a, s) : d == 128 ? launch_t<TQ, FP8, 128>(a, s) : launch_t<TQ, FP8, 256>(a, s);
}

}  // namespace

hipError_t launch_prefix_attn(const PrefixArgs& a, int cache_dtype, int q_dtype, int head_dim, hipStream_t s) {
    if (q_dtype == UBW_F16)
        return cache_dtype == UBW_E4M3 ? launch_d<h16, true>(a, head_dim, s) : launch_d<h16, false>(a, head_dim, s);
    return cache_dtype == UBW_E4M3 ? launch_d<b16, true>(a, head_dim, s) : launch_d<b16, false>(a, head_dim, s);
}

}  // namespace cache
}  // namespace ubw

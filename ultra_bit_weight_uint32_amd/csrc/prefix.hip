// Attention of each sequence's new tokens over its context, where sequences have the beginning of it in common:
// a group's prefix is gone through once, with the rows of all its sequences side by side, and each sequence's
// own positions behind it as in tree attention. With the sums of both parts, m the maximum and l the sum of
// 2^((s - m) log2 e) over a part's positions, o their weighted mean,
//     out = sum_parts l_i 2^((m_i - m) log2 e) o_i / sum_parts l_i 2^((m_i - m) log2 e),  m = max m_i.
//
// Three launches: k_plan (one workgroup) measures the groups, cuts the lists of rows and positions into pieces and
// deals them out (cache_plan.h); k_prefix goes through them (attn_pieces.h); k_join_parts joins each row's.
//   * A prefix ends at a multiple of 16 positions, so that no tile has positions of both parts; the few behind
//     it are each sequence's own (its own row of the table has them too).
//   * A prefix passes the shortest context of its group nowhere, so that a sequence never sees what is not its own.
//   * Prefixes of many rows keep the vector unit and the matrix cores busy, single rows the memory: each XCD has an
//     eighth of the full pieces, in order (row blocks over the same keys and values meet in its L2), and of the rests.
//     Which workgroup has a piece decides nothing but the time.
//
// Bound: behind many rows the loop's issue and latency (a unit of 128 positions takes 4.0 to 4.5 us with 128 rows or
// fewer, 2 workgroups a CU), behind few rows the memory, and 8 to 10 us to begin and end a piece. 64 samples over a prompt of
// 16K positions, 64 heads over 8 of 128 dims, bf16: plan 11, pieces 86 to 89 (matrix cores busy 24% of the cycles, the vector
// unit 34%), join 8 us, 102 to 104 in a queue (tree attention, which reads the prompt 64 times, 697); five groups of trees in
// 8 bits 14, 225 to 239 one launch at a time (39% and 52%), 20 and 234 in a queue (0.68 PFLOP/s; 388); 40 sequences of 32
// heads with keys of their own 11, 85, 5 and 102 (4.2 TB/s; 636). Short contexts are left to tree attention (prefix_alone).
// More than 1024 sequences or groups: k_plan keeps part of its eight owners a thread in scratch (1500 sequences 31 us, 4096 in
// four groups 49, in 4096 groups 61; 512 sequences 11, 1024 15).
#include "attn_pieces.h"

namespace ubw {
namespace cache {
namespace {

constexpr int kPlanThreads = 512;
static_assert(kPlanThreads >= kPrefixWgs, "a thread for every workgroup of rests");
static_assert(kRestBuckets == 64, "a lane for every bucket");

// An owner in the plan. Class 0: whole blocks of rows, class 1: the small one.
struct Owner {
    int row, q0, rows, base;  // row of the table, first token, rows, position where its units begin
    int ctx, len, tree, big;  // ends of the context and of the positions; 0, or -1: no tree; whole blocks
    int full0[2], full[2];    // first full piece, full pieces of a list
    int rest[2];              // units of the rest
    int units, group;         // of a list; a sequence's group, -1: none
};
static_assert(sizeof(Owner) == 4 * kPlanOwner, "owners lie in the plan");
struct Work {
    int owner, index;  // index: class, then (part, head, block) of it; part: the full piece, or behind them the rest
};
struct PlanAt {
    int* head;  // full pieces, long rests
    int* run;   // where each workgroup's run of the other rests begins, and the end
    Owner* owner;
    Work* full;
    Work* rest;
};
__device__ inline PlanAt plan_at(int* p, int owners) {
    PlanAt x;
    x.head = p;
    x.run = p + 8;
    x.owner = reinterpret_cast<Owner*>(p + kPlanHead);
    x.full = reinterpret_cast<Work*>(x.owner + owners);
    x.rest = x.full + kPrefixFull;
    return x;
}

// Two numbers of the threads before this one, added up.
struct Two {
    int a, b;
};
__device__ inline Two plan_before(Two mine, Two (&lds)[kPlanThreads / 64], Two* all) {
    Two y = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(y.a, d), v = __shfl_up(y.b, d);
        if ((int)(threadIdx.x & 63) >= d) {
            y.a += u;
            y.b += v;
        }
    }
    Two x{y.a - mine.a, y.b - mine.b}, t{0, 0};
    if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = y;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        const Two z = lds[w];
        if (w < (int)(threadIdx.x >> 6)) {
            x.a += z.a;
            x.b += z.b;
        }
        t.a += z.a;
        t.b += z.b;
    }
    *all = t;
    return x;
}

// The sum of x over the lanes up to this one.
template <typename N>
__device__ inline N lanes_up_to(N x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const N u = __shfl_up(x, d);
        if ((int)(threadIdx.x & 63) >= d) x += u;
    }
    return x;
}
// Blocks of `rows` rows: whole ones, and a small one. (The tile of 256 dims has no small one.)
struct RowBlocks {
    int big, small;
};
__device__ inline RowBlocks blocks_of(int rows, int lrb) {
    const int whole = rows >> lrb, rest = rows - (whole << lrb);
    return rest == 0 ? RowBlocks{whole, 0} : rest <= kSmallRows && lrb == 7 ? RowBlocks{whole, 1} : RowBlocks{whole + 1, 0};
}

// A thread has the groups and the sequences EACH t .. EACH t + EACH - 1.
template <int EACH>
__global__ __launch_bounds__(kPlanThreads) void k_plan(PrefixArgs a, int lrb, int small_cost) {
    constexpr int kMost = EACH * kPlanThreads;
    __shared__ int start[kMost + 1], len[kMost], lead[kMost], last[kMost];
    __shared__ int bucket[kRestBuckets], bucket0[kRestBuckets + 1];  // rests, and those before
    __shared__ int64_t cost0[kRestBuckets + 1];                      // what those before cost
    __shared__ unsigned long long cost;                              // of all lists
    __shared__ int full0[4 * kMost];  // first full piece of each owner's classes
    __shared__ Two lds[kPlanThreads / 64];
    __shared__ int64_t rooms[kPlanThreads / 64];
    const int tid = threadIdx.x, kv = a.c.heads;
    const PlanAt at = plan_at(a.plan, a.groups + a.batch);
    const int most = (int)min((int64_t)a.table_cols << a.c.lps, (int64_t)1 << 30);
    bool falls = false;
    for (int g = tid; a.groups > 0 && g <= a.groups; g += kPlanThreads) {
        falls |= g > 0 && a.group_start[g] < a.group_start[g - 1];
        start[g] = min(max(a.group_start[g], 0), a.batch);
        if (g < a.groups) {
            len[g] = min(max(a.prefix_len[g], 0), most);
            lead[g] = a.batch;
            last[g] = -1;
        }
    }
    if (tid < kRestBuckets) bucket[tid] = 0;
    if (tid == 0) cost = 0;
    Seq s[EACH];
    int of[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = tid * EACH + i;
        s[i] = b < a.batch ? seq_of(a, b) : Seq{0, 0, 0};
        falls |= b < a.batch && a.q_start[b + 1] < a.q_start[b];
    }
    const bool none = __syncthreads_or(falls);  // these do not ascend: nothing is shared
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = tid * EACH + i;
        of[i] = -1;
        if (s[i].n <= 0 || a.groups == 0 || none) continue;
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

    // Owners 0, 2, ..: this thread's groups, 1, 3, ..: its sequences.
    Owner x[2 * EACH];
    RowBlocks rows[2 * EACH];
    const auto cost_of = [&](const Owner& o, const RowBlocks& r) {
        return (int64_t)kv * (r.big * ((int64_t)o.units * kUnitCost + kPieceCost) + r.small * ((int64_t)o.units * small_cost + kPieceCost));
    };
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int g = tid * EACH + i;
        Owner& o = x[2 * i];
        o = Owner{};
        rows[2 * i] = RowBlocks{0, 0};
        if (g >= a.groups) continue;
        o.q0 = min(max(a.q_start[start[g]], 0), a.tokens);
        o.rows = (min(max(a.q_start[max(start[g + 1], start[g])], o.q0), a.tokens) - o.q0) * a.group;
        const int n = last[g] > lead[g] && o.rows > 0 ? len[g] & ~15 : 0;  // one sequence alone shares nothing
        o.row = min(lead[g], a.batch - 1);
        o.ctx = o.len = n;
        o.tree = o.group = -1;
        o.units = units_of(n);
        if (n > 0) rows[2 * i] = blocks_of(o.rows, lrb);
        o.big = rows[2 * i].big;
        if (n > 0) atomicAdd(&cost, (unsigned long long)cost_of(o, rows[2 * i]));
        len[g] = n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = tid * EACH + i;
        Owner& o = x[2 * i + 1];
        o = Owner{};
        rows[2 * i + 1] = RowBlocks{0, 0};
        if (b >= a.batch) continue;
        o.row = b;
        o.q0 = s[i].q0;
        o.rows = s[i].n * a.group;
        o.base = of[i] >= 0 ? len[of[i]] : 0;
        o.group = o.base > 0 ? of[i] : -1;
        o.ctx = s[i].ctx;
        o.len = positions(a, s[i]);
        if (s[i].n <= 0) continue;
        o.units = max(1, units_of(o.len - o.base));
        rows[2 * i + 1] = blocks_of(o.rows, lrb);
        o.big = rows[2 * i + 1].big;
        atomicAdd(&cost, (unsigned long long)cost_of(o, rows[2 * i + 1]));
    }
    __syncthreads();
    const int64_t goal = prefix_goal((int64_t)cost);
    const float scale = (float)kRestBuckets / (float)goal;
    const int64_t begin = rest_begin_cost(goal);
    Two first, all;          // full pieces of the groups, of the sequences
    int in[2 * EACH][2];     // places in the rests' buckets
    const auto bucket_of = [&](int rest, int c) { return rest_bucket(rest, c ? small_cost : kUnitCost, scale); };
    int64_t full_cost = goal;
    for (int turn = 0;; ++turn) {
        const int length[2] = {prefix_full(full_cost, kUnitCost), prefix_full(full_cost, small_cost)};
        Two count{0, 0};
#pragma unroll
        for (int i = 0; i < 2 * EACH; ++i) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int lists = (c ? rows[i].small : rows[i].big) * kv;
                const PrefixCut cut = prefix_cut(x[i].units, length[c]);
                x[i].full[c] = lists > 0 ? cut.full : 0;
                x[i].rest[c] = lists > 0 ? cut.rest : 0;
                (i & 1 ? count.b : count.a) += x[i].full[c] * lists;
                if (x[i].rest[c] > 0) in[i][c] = atomicAdd(&bucket[bucket_of(x[i].rest[c], c)], lists);
            }
        }
        first = plan_before(count, lds, &all);  // (the buckets are full, too)
        if (tid < kRestBuckets) {
            const int y = lanes_up_to(bucket[tid]);
            const int64_t z = lanes_up_to((int64_t)bucket[tid] * rest_cost(tid, begin));
            bucket0[tid + 1] = y;
            cost0[tid + 1] = z;
            if (tid == 0) bucket0[0] = 0, cost0[0] = 0;
            if (tid == kRestBuckets - 1) at.head[0] = all.a + all.b;
        }
        __syncthreads();
        if (prefix_fits(all.a + all.b, cost0[kRestBuckets], goal, full_cost) || turn == kPrefixTurns - 1) break;
        __syncthreads();
        full_cost = prefix_longer(full_cost);
        if (tid < kRestBuckets) bucket[tid] = 0;
        __syncthreads();
    }
    first.b += all.a;
#pragma unroll
    for (int i = 0; i < 2 * EACH; ++i) {
        const int n = tid * EACH + (i >> 1), id = i & 1 ? a.groups + n : n;
        if (n >= (i & 1 ? a.batch : a.groups)) continue;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int lists = (c ? rows[i].small : rows[i].big) * kv;
            int& k = i & 1 ? first.b : first.a;
            x[i].full0[c] = k;
            const int full = x[i].full[c] * lists;
            full0[2 * id + c] = k;
            k += full;
            if (x[i].rest[c] > 0) {
                Work* to = at.rest + bucket0[bucket_of(x[i].rest[c], c)] + in[i][c];
                for (int j = 0; j < lists; ++j) to[j] = Work{id, c << 30 | (full + j)};
            }
        }
        at.owner[id] = x[i];
    }
    __syncthreads();
    for (int k = tid; k < all.a + all.b; k += kPlanThreads) {
        int lo = 0, hi = 2 * (a.groups + a.batch);  // the last class that begins at k or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (full0[mid] <= k) lo = mid; else hi = mid;
        }
        at.full[k] = Work{lo >> 1, (lo & 1) << 30 | (k - full0[lo])};
    }
    // The rests for the workgroups without a full piece.
    const int bins = rest_bins(all.a + all.b), rests = bucket0[kRestBuckets];
    const int64_t have = cost0[kRestBuckets] / bins;
    const int long_ones = long_buckets(have, begin), longs = bucket0[long_ones];
    const int64_t room = tid < bins ? rest_room(tid, bins, longs, have, bucket0, begin) : 0;
    const int64_t y = lanes_up_to(room);
    if ((tid & 63) == 63) rooms[tid >> 6] = y;
    __syncthreads();
    int64_t before = y - room, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        if (w < (tid >> 6)) before += rooms[w];
        total += rooms[w];
    }
    if (tid < bins) at.run[tid] = rest_run(before, total, bucket0, cost0, long_ones, begin);
    if (tid == 0) at.run[bins] = rests;
    if (tid == 0) at.head[1] = longs;
}

// The tile of whole blocks, and that of small ones.
template <bool FP8, int D>
struct Tiles {
    static constexpr int MT = D == 256 ? 1 : 2, NS = D == 256 ? 1 : 2, NB = FP8 || D == 64 ? 2 : 1;
    using Big = Cfg<FP8, D, MT, 4, 1, NS, 2>;
    using Small = Cfg<FP8, D == 256 ? 64 : D, 2, 1, 4, 1, NB>;  // (256 dims: not used)
};
template <typename C1, typename C2>
union SharedOf {
    Shared<C1> big;
    Shared<C2> small;
};

template <typename TQ, bool FP8, int D>
__global__ __launch_bounds__(256, 2) void k_prefix(PrefixArgs a) {
    using W = Tiles<FP8, D>;
    constexpr int RB = W::Big::RB, ROW = D + 4;
    static_assert(W::Big::kThreads == 256 && W::Small::kThreads == 256 && (D == 256 || W::Small::RB == kSmallRows), "tiles of one workgroup");
    __shared__ __align__(1024) SharedOf<typename W::Big, typename W::Small> sh;
    const PlanAt at = plan_at(a.plan, a.groups + a.batch);
    const int full = scalar_words(at.head)[0];
    const PrefixShare share = prefix_share(blockIdx.x, full, scalar_words(at.head)[1], scalar_words(at.run));
    // Work n of this workgroup, -1 behind the last.
    Work work{0, 0};
    const auto get = [&](int n) {
        const int k = prefix_work(share, n);
        if (k < 0) return -1;
        const ScalarWord* w = scalar_words(reinterpret_cast<const int*>(at.full + k));
        work = Work{w[0], w[1]};
        return n;
    };
    const auto next = [&](int n) { return get(n + 1); };
    const auto piece = [&](int, Piece& p) {
        const ScalarWord* o = scalar_words(reinterpret_cast<const int*>(at.owner + work.owner));
        const int c = work.index >> 30, big = o[7], blocks = c ? 1 : big, units = o[14], cut = o[10 + c], rest = o[12 + c];
        int r = work.index & ((1 << 30) - 1);
        const int part = r / (blocks * a.c.heads);
        r -= part * blocks * a.c.heads;
        p.h = r / blocks;
        p.r0 = (c ? big : r - p.h * blocks) * RB;
        p.row = o[0];
        p.q0 = o[1];
        p.rows = o[2];
        p.base = o[3];
        p.ctx = o[4];
        p.len = o[5];
        p.tree = o[6];
        if (part < cut) attn_range(units - rest, cut, part, &p.u0, &p.u1);
        else p.u0 = units - rest, p.u1 = units;
        p.slot = part < cut ? o[8 + c] + (work.index & ((1 << 30) - 1)) : -1;
        p.last = p.base == 0 && p.tree == 0 && p.u1 - p.u0 == units;
        return true;
    };
    const auto row_of = [&](const Piece& p, int rl, int token, int hq) {
        const int64_t rest = (int64_t)kPrefixFull * RB + ((p.tree < 0 ? a.tokens : 0) + (int64_t)token) * a.heads + hq;
        return a.ws + (p.slot >= 0 ? (int64_t)p.slot * RB + rl : rest) * ROW;
    };
    int n = get(0);
#pragma unroll 1
    while (n >= 0) {
        if (D == 256 || work.index >> 30 == 0) {
            n = attn_pieces<kParts, TQ, FP8, D, W::MT, 4, 1, W::NS, 2, false>(
                a, sh.big, n, a.ws, [&](int n) { return n >= 0 && (D == 256 || work.index >> 30 == 0); }, next, piece, row_of);
        } else if constexpr (D < 256) {
            n = attn_pieces<kParts, TQ, FP8, D, 2, 1, 4, 1, W::NB, true>(
                a, sh.small, n, a.ws, [&](int n) { return n >= 0 && work.index >> 30 != 0; }, next, piece, row_of);
        }
    }
}

// Joins the pieces of the prefix and of what is behind it, WAVES waves per (token, query head), in an order that
// does not depend on timing: the prefix's full pieces and rest, the own ones.
template <typename TQ, int D, int WAVES>
__global__ __launch_bounds__(256) void k_join_parts(PrefixArgs a) {
    constexpr int RB = D == 256 ? 64 : 128, ROW = D + 4;
    __shared__ float part[4][D + 2];
    const int wave = threadIdx.x >> 6;
    const int b = blockIdx.x / a.c.heads, h = blockIdx.x - b * a.c.heads;
    const int r = WAVES == 4 ? (int)blockIdx.y : (int)blockIdx.y * 4 + wave;
    const PlanAt at = plan_at(a.plan, a.groups + a.batch);
    const ScalarWord* o = scalar_words(reinterpret_cast<const int*>(at.owner + a.groups + b));
    if (r >= (int)o[2]) return;
    const int q0 = o[1], g = o[15], t = r / a.group, hq = h * a.group + (r - t * a.group);
    // where the pieces of row x of an owner are
    struct Rows {
        const float *full, *rest;
        uint32_t apart;
        int n, all;
    };
    const auto rows_at = [&](const ScalarWord* o, int x, bool shared) {
        const int big = o[7], blk = x / RB, c = blk >= big, blocks = c ? 1 : big, n = o[10 + c];
        Rows y;
        y.full = a.ws + ((int64_t)(o[8 + c] + h * blocks + (c ? 0 : blk)) * RB + (x - blk * RB)) * ROW;
        y.rest = a.ws + ((int64_t)kPrefixFull * RB + ((shared ? a.tokens : 0) + (int64_t)(q0 + t)) * a.heads + hq) * ROW;
        y.apart = (uint32_t)(a.c.heads * blocks * RB * ROW);
        y.n = n;
        y.all = n + (o[12 + c] > 0);
        return y;
    };
    const Rows own = rows_at(o, r, false);
    if (own.all <= 1 && g < 0) return;
    Rows group{};
    if (g >= 0) {
        const ScalarWord* go = scalar_words(reinterpret_cast<const int*>(at.owner + g));
        const int x = (q0 - (int)go[1]) * a.group + r;
        if (x >= 0 && x < (int)go[2]) group = rows_at(go, x, true);
    }
    const float scale = a.scale * (a.c.k_scale ? a.c.k_scale[h] : 1.f);
    const float unit = ldexpf(scale, -lower<TQ>(scale)), cc = unit * kLog2e;  // as in attn_pieces
    const auto row = [&](int i) {
        const bool mine = i >= group.all;
        const int k = mine ? i - group.all : i, n = mine ? own.n : group.n;
        const float* full = mine ? own.full : group.full;
        return k < n ? full + (uint64_t)(uint32_t)k * (mine ? own.apart : group.apart) : mine ? own.rest : group.rest;
    };
    RowSums<D> x;
    join_row<D, WAVES>(x, group.all + own.all, WAVES == 4 ? wave : 0, cc, row, [&](int i) { return row(i) + D; });
    if constexpr (WAVES == 4) {
        if (!join_waves<D, WAVES>(x, part, cc)) return;
    }
    store_row<TQ, D>(a, x, q0 + t, h, r - t * a.group, unit);
}

template <typename TQ, bool FP8, int D>
hipError_t launch_t(const PrefixArgs& a, hipStream_t s) {
    const int most = a.batch > a.groups ? a.batch : a.groups, lrb = log2_of(prefix_rows(D)), cost = FP8 ? kSmallUnitCost8 : kSmallUnitCost;
    if (most <= kPlanThreads) k_plan<1><<<1, kPlanThreads, 0, s>>>(a, lrb, cost);
    else if (most <= 2 * kPlanThreads) k_plan<2><<<1, kPlanThreads, 0, s>>>(a, lrb, cost);
    else k_plan<8><<<1, kPlanThreads, 0, s>>>(a, lrb, cost);
    k_prefix<TQ, FP8, D><<<kPrefixWgs, 256, 0, s>>>(a);
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

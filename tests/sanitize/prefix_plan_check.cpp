// Host checks of the planning of attention over shared prefixes and over selected blocks (ultra_bit_weight_uint32_amd/
// csrc/cache_plan.h), built with -fsanitize=address,undefined: random and edge shapes. Prints "ok" and exits 0 on success.
#include <cstdio>
#include <random>
#include <vector>

#include "../../ultra_bit_weight_uint32_amd/csrc/cache_plan.h"

using namespace ubw::cache;

static int fails = 0;
#define CHECK(c, ...)                                                     \
    do {                                                                  \
        if (!(c) && fails++ < 20) {                                       \
            std::fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__);     \
            std::fprintf(stderr, __VA_ARGS__);                            \
            std::fprintf(stderr, "\n");                                   \
        }                                                                 \
    } while (0)

typedef std::mt19937_64 Rng;
static int64_t rnd(Rng& r, int64_t lo, int64_t hi) { return lo + (int64_t)(r() % (uint64_t)(hi - lo + 1)); }

// Lists of any units and tiles: every unit in one piece, no more full pieces than the workspace holds, and none much
// longer than what a workgroup is to have.
static void check_cut(Rng& r) {
    for (int it = 0; it < 20000; ++it) {
        const int n = (int)rnd(r, 1, it % 3 ? 30 : 2000);
        const int64_t longest = it % 5 == 0 ? 1 << 23 : it % 2 ? 40 : 2000;
        const int small = it & 1 ? kSmallUnitCost : kSmallUnitCost8;
        std::vector<int> units(n), lists(n), cost(n);
        int64_t total = 0;
        for (int i = 0; i < n; ++i) {
            units[i] = (int)rnd(r, 1, longest);
            lists[i] = (int)rnd(r, 1, it % 7 ? 64 : 4096);
            cost[i] = rnd(r, 0, 1) ? kUnitCost : small;
            total += lists[i] * ((int64_t)units[i] * cost[i] + kPieceCost);
        }
        const int64_t goal = prefix_goal(total);
        int64_t full = 0;
        for (int i = 0; i < n; ++i) {
            const int length = prefix_full(goal, cost[i]);
            CHECK(length >= 1, "length %d", length);
            const PrefixCut c = prefix_cut(units[i], length);
            full += (int64_t)c.full * lists[i];
            CHECK(c.full >= 0 && c.rest >= 0 && (c.full > 0 || c.rest > 0), "cut of %d", units[i]);
            CHECK(c.rest == 0 || (int64_t)c.full * length + c.rest == units[i], "%d + %d of %d", c.full, c.rest, units[i]);
            int at = 0, u0 = 0, u1 = 0;
            for (int k = 0; k < c.full && k < 100; ++k) {
                attn_range(units[i] - c.rest, c.full, k, &u0, &u1);
                CHECK(u0 == at && u1 > u0 && u1 - u0 <= length + length / 8 + 1, "piece %d of %d: %d .. %d", k, c.full, u0, u1);
                at = u1;
            }
            if (c.full > 0 && c.full <= 100) CHECK(at == units[i] - c.rest, "full pieces end at %d of %d", at, units[i]);
            CHECK((int64_t)c.rest * cost[i] <= goal, "rest %d", c.rest);
        }
        CHECK(full <= kPrefixFull, "%lld full pieces", (long long)full);
    }
    CHECK(prefix_goal(0) == kPieceCost && prefix_full(kPieceCost, kUnitCost) == 1, "nothing to do");
    CHECK(prefix_full((int64_t)1 << 60, kUnitCost) == kAttnMostChunk, "as long as lists can be");
}

// Lists of some units and cost, so many of each kind.
struct Kind {
    int units, lists, cost;
};
// The pieces of such lists as the planning kernel cuts and deals them out: what the workgroups go through is every
// piece once, runs ascend, and no workgroup has rests of much more than its share. (Long ones dealt there and back differ
// by the largest at most, and their mean is no more than the share; the others fill what is left up to one of them, a
// quarter of the share or less, and what the shares' rounding down leaves over.)
static void check_dealing(const std::vector<Kind>& kinds, int* most_turns) {
    int64_t total = 0;
    for (const Kind& k : kinds) total += k.lists * ((int64_t)k.units * k.cost + kPieceCost);
    const int64_t goal = prefix_goal(total), begin = rest_begin_cost(goal);
    int64_t full_cost = goal;
    int full = 0, before[kRestBuckets + 1], turn = 0;
    int64_t cost[kRestBuckets + 1];
    for (;; ++turn) {
        int in[kRestBuckets] = {};
        full = 0;
        for (const Kind& k : kinds) {
            const PrefixCut c = prefix_cut(k.units, prefix_full(full_cost, k.cost));
            full += c.full * k.lists;
            if (c.rest > 0) in[rest_bucket(c.rest, k.cost, (float)kRestBuckets / (float)goal)] += k.lists;
        }
        before[0] = 0;
        cost[0] = 0;
        for (int b = 0; b < kRestBuckets; ++b) {
            before[b + 1] = before[b] + in[b];
            cost[b + 1] = cost[b] + in[b] * rest_cost(b, begin);
        }
        if (prefix_fits(full, cost[kRestBuckets], goal, full_cost) || turn == kPrefixTurns - 1) break;
        full_cost = prefix_longer(full_cost);
    }
    if (turn > *most_turns) *most_turns = turn;
    const int rests = before[kRestBuckets], bins = rest_bins(full);
    CHECK(full <= kPrefixFull && bins >= 1 && bins <= kPrefixWgs, "%d full pieces, %d workgroups for %d rests", full, bins, rests);
    const int64_t have = cost[kRestBuckets] / bins;
    const int long_ones = long_buckets(have, begin), longs = before[long_ones];
    for (int b = 0; b < kRestBuckets; ++b)
        CHECK((4 * rest_cost(b, begin) > have) == (b < long_ones) && rest_cost(b, begin) <= 1 << 17, "cost of bucket %d", b);
    std::vector<int64_t> room(bins);
    int64_t rooms = 0;
    for (int w = 0; w < bins; ++w) rooms += room[w] = rest_room(w, bins, longs, have, before, begin);
    std::vector<int> run(bins + 1);
    int64_t sum = 0;
    for (int w = 0; w < bins; ++w) {
        run[w] = rest_run(sum, rooms, before, cost, long_ones, begin);
        sum += room[w];
        CHECK(w == 0 ? run[w] == longs : run[w] >= run[w - 1], "run %d begins at %d", w, run[w]);
    }
    run[bins] = rests;
    CHECK(run[bins - 1] <= rests, "the last run begins at %d of %d", run[bins - 1], rests);
    if (fails) return;
    std::vector<int> done(kPrefixFull + rests, 0);
    int64_t largest = 0;
    for (int b = kRestBuckets - 1; b >= 0; --b) largest = before[b + 1] > before[b] ? rest_cost(b, begin) : largest;
    for (int wg = 0; wg < kPrefixWgs; ++wg) {
        const PrefixShare s = prefix_share(wg, full, longs, run.data());
        int n = 0;
        for (;; ++n) {
            const int k = prefix_work(s, n);
            if (k < 0) break;
            const bool is = k < full || (k >= kPrefixFull && k < kPrefixFull + rests);
            CHECK(is, "workgroup %d has %d", wg, k);
            if (is) ++done[k];
        }
        CHECK(n == s.fulls + s.longs + s.rests, "workgroup %d ends at %d", wg, n);
        int64_t load = 0;
        for (int i = s.fulls; i < n; ++i) {
            const int k = prefix_work(s, i) - kPrefixFull;
            int b = 0;
            while (before[b + 1] <= k) ++b;
            load += rest_cost(b, begin);
        }
        CHECK(load <= have + have / 4 + largest + 2048, "workgroup %d has %lld of %lld", wg, (long long)load, (long long)have);
    }
    int lost = 0, twice = 0;
    for (int k = 0; k < kPrefixFull + rests; ++k) {
        const int want = k < full || k >= kPrefixFull;
        lost += done[k] < want;
        twice += done[k] > want;
    }
    CHECK(!lost && !twice, "of %d full pieces and %d rests %d lost, %d twice", full, rests, lost, twice);
}
static void check_dealings(Rng& r) {
    int turns = 0;
    // ends of neighbouring runs fall together in these (tokens beside key/value heads: heads x sequences lists)
    check_dealing({{39, 320, kUnitCost}, {20, 620, kUnitCost}, {4, 310, kUnitCost}}, &turns);
    check_dealing({{92, 216, kUnitCost}, {36, 256, kUnitCost}, {2, 860, kSmallUnitCost8}}, &turns);
    check_dealing({{47, 440, kUnitCost}, {11, 660, kUnitCost}, {22, 230, kUnitCost}}, &turns);
    check_dealing({{18, 610, kUnitCost}, {60, 370, kUnitCost}, {100, 440, kUnitCost}}, &turns);
    check_dealing({{74, 400, kSmallUnitCost}, {4, 256, kUnitCost}, {18, 444, kUnitCost}}, &turns);
    // nothing; one list; as many, and as long, as there may be
    check_dealing({}, &turns);
    check_dealing({{1, 1, kUnitCost}}, &turns);
    check_dealing({{1 << 23, 1, kSmallUnitCost8}}, &turns);
    check_dealing({{1, (1 << 24) - 1, kUnitCost}}, &turns);
    check_dealing({{1 << 23, (1 << 23), kUnitCost}, {1, (1 << 23) - 1, kSmallUnitCost}}, &turns);
    for (int it = 0; it < 3000; ++it) {
        const int kv = it % 4 ? 1 << rnd(r, 0, 4) : 10, small = it & 1 ? kSmallUnitCost : kSmallUnitCost8;
        std::vector<Kind> kinds(it % 3 == 0 ? rnd(r, 1, 60) : rnd(r, 2, 3));
        const int longest = it % 5 ? 100 : 3000;
        for (Kind& k : kinds) k = Kind{(int)rnd(r, 1, longest), (int)rnd(r, 1, kinds.size() > 3 ? 3 : 150) * kv, rnd(r, 0, 3) ? kUnitCost : small};
        check_dealing(kinds, &turns);
    }
    CHECK(turns > 0, "full pieces were never made longer");
}

// Workspaces: what serves a call serves every smaller one; the plan fits behind the sums.
static void check_sizes(Rng& r) {
    for (int it = 0; it < 3000; ++it) {
        const int dim = 64 << rnd(r, 0, 2), group = (int)rnd(r, 1, it % 5 ? 16 : 300), kv = (int)rnd(r, 1, 9);
        const int batch = (int)rnd(r, 1, it % 3 ? 40 : 4096), groups = (int)rnd(r, 0, batch), tree = (int)rnd(r, 1, UBW_MAX_TREE);
        const int64_t tokens = rnd(r, 0, (int64_t)batch * tree);
        const int64_t have = prefix_workspace_floats(batch, groups, tokens, tree, group, kv, dim);
        const int b2 = (int)rnd(r, 1, batch), g2 = (int)rnd(r, 0, groups < b2 ? groups : b2), t2 = (int)rnd(r, 1, tree);
        const int64_t n2 = rnd(r, 0, tokens);
        const PrefixSizes z = prefix_sizes(b2, g2, n2, (int64_t)t2 * group, group, kv, dim);
        CHECK(z.rows * prefix_row_floats(dim) + z.words <= have, "a smaller call needs more");
        CHECK(z.lists >= (int64_t)b2 * kv && z.rows >= (int64_t)kPrefixFull * prefix_rows(dim), "rows for all");
        CHECK((z.rows * prefix_row_floats(dim)) % 4 == 0, "the plan's words are aligned");
        // blocks: every cut of a row fits
        const int64_t bt = rnd(r, 0, 4096), small = rnd(r, 0, bt);
        const AttnTile tile = block_tile(group, dim);
        const int64_t pairs = block_pairs(small, group, kv, tile);
        const int splits = block_splits(pairs, block_positions((int)rnd(r, 0, 5000), 16 << rnd(r, 0, 6), tree));
        CHECK(splits >= 1, "splits %d", splits);
        CHECK(splits == 1 || pairs * splits <= block_cap(pairs), "%lld pairs x %d", (long long)pairs, splits);
        CHECK(block_workspace_floats(small, group, kv, dim) <= block_workspace_floats(bt, group, kv, dim), "fewer tokens need more");
        CHECK(block_cap(pairs) * attn_rows(tile) * (dim + 2) + small * kv <= block_workspace_floats(bt, group, kv, dim), "blocks' sums");
    }
    CHECK(bounds_groups(80, 8, 64, 2) == 80 * 8 * 2 && bounds_groups(80, 8, 4096, 1 << 24) == 64, "groups of lanes");
}

int main() {
    Rng r(12345);
    check_cut(r);
    check_dealings(r);
    check_sizes(r);
    if (fails) {
        std::fprintf(stderr, "%d checks failed\n", fails);
        return 1;
    }
    std::puts("ok");
    return 0;
}

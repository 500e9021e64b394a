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
    check_sizes(r);
    if (fails) {
        std::fprintf(stderr, "%d checks failed\n", fails);
        return 1;
    }
    std::puts("ok");
    return 0;
}

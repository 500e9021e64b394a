// Host checks of the key/value cache calls' planning and argument validation (ultra_bit_weight_uint32_amd/
// csrc/cache_plan.h), built with -fsanitize=address,undefined: random and edge shapes, each result
// compared with a plain recomputation. Prints "ok" and exits 0 on success.
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

// The pieces of a batch: every unit of every (sequence, head, row block) exactly once, sizes alike, no
// more pieces than the workspace holds.
static void check_cut(Rng& r) {
    for (int it = 0; it < 4000; ++it) {
        const int dim = 64 << rnd(r, 0, 2), group = (int)rnd(r, 1, it % 7 ? 16 : 1024), kv = (int)rnd(r, 1, 9);
        const int tree = (int)rnd(r, 1, UBW_MAX_TREE), batch = (int)rnd(r, 1, it % 5 ? 40 : 600);
        const int64_t max_rows = (int64_t)tree * group;
        const AttnTile t = attn_tile(max_rows, dim);
        const int rb = attn_rows(t);
        CHECK(rb >= 16 && (t.row_waves == 1 || t.row_waves == 2 || t.row_waves == 4), "tile %d x %d", t.tiles, t.row_waves);
        if (dim < 256 && max_rows <= 128) CHECK(rb >= max_rows, "%d rows in blocks of %d", (int)max_rows, rb);
        std::vector<int64_t> units(batch), blocks(batch);
        int64_t total = 0;
        const int64_t longest = it % 3 ? 2000 : 1 << 24;
        for (int b = 0; b < batch; ++b) {
            const int n = (int)rnd(r, 0, tree);
            units[b] = n ? cdiv(rnd(r, 1, longest), kAttnUnit) : 0;
            blocks[b] = cdiv((int64_t)n * group, rb);
            total += units[b] * blocks[b] * kv;
        }
        const int target = attn_aim(total, attn_target(t, dim), t.row_waves == 1);
        CHECK(target >= 256 && target <= attn_target(t, dim), "aim %d", target);
        int chunk = attn_chunk(total, target);
        const auto pieces = [&](int c) {
            int64_t p = 0;
            for (int b = 0; b < batch; ++b) p += (int64_t)attn_splits((int)units[b], c) * blocks[b] * kv;
            return p;
        };
        const int64_t room = attn_max_items(batch, max_rows, kv, dim, t);
        for (int step = 0; step < 5; ++step) {
            const int64_t p = pieces(chunk);
            CHECK(p <= room, "%lld pieces, room for %lld", (long long)p, (long long)room);
            if (p <= target) break;
            const int next = attn_larger_chunk(chunk, p, target);
            CHECK(next > chunk || chunk == kAttnMostChunk, "chunk %d stays", chunk);
            chunk = next;
        }
        for (int b = 0; b < batch && b < 8; ++b) {
            const int u = (int)units[b], s = attn_splits(u, chunk);
            int at = 0;
            for (int i = 0; i < s; ++i) {
                int u0, u1;
                attn_range(u, s, i, &u0, &u1);
                CHECK(u0 == at && u1 > u0 && u1 - u0 <= chunk && u1 - u0 >= u / s, "piece %d of %d: %d..%d", i, s, u0, u1);
                at = u1;
            }
            CHECK(at == u, "%d of %d units", at, u);
        }
        // scratch for smaller trees and batches is never more
        const int64_t need = attn_workspace_floats(batch, tree, group, kv, dim);
        const int smaller = (int)rnd(r, 1, tree), fewer = (int)rnd(r, 1, batch);
        CHECK(attn_workspace_floats(fewer, smaller, group, kv, dim) <= need, "scratch of %d, %d", fewer, smaller);
        CHECK(need >= room * rb * (dim + 2) + batch + 1, "scratch %lld", (long long)need);
    }
}

static ubw_kv_cache good(Rng& r) {
    static char store[64];
    ubw_kv_cache c{};
    c.k = c.v = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(store) + 15) & ~(uintptr_t)15);
    c.dtype = (int)rnd(r, 1, 3);
    c.layers = (int)rnd(r, 1, 80);
    c.pages = (int)rnd(r, 1, 100000);
    c.page_size = 16 << rnd(r, 0, 6);
    c.kv_heads = (int)rnd(r, 1, 64);
    c.head_dim = 64 << rnd(r, 0, 2);
    while ((int64_t)c.pages * c.page_size * c.kv_heads * c.head_dim > (int64_t)1 << 40) c.pages /= 2;
    const int64_t row = c.head_dim, head = row * c.page_size, page = head * c.kv_heads;
    const int64_t st[4] = {page * c.pages, page, head, row};
    for (int i = 0; i < 4; ++i) c.k_stride[i] = c.v_stride[i] = st[i];
    return c;
}

static void check_caches(Rng& r) {
    CHECK(check_cache(nullptr) == UBW_EINVAL, "null");
    for (int it = 0; it < 2000; ++it) {
        const ubw_kv_cache c = good(r);
        CHECK(check_cache(&c) == UBW_OK, "a good cache: %d", check_cache(&c));
        CHECK(1 << log2_of(c.page_size) == c.page_size, "log2");
        const int64_t vecs = (int64_t)c.kv_heads * c.page_size * c.head_dim * type_size(c.dtype) / 16;
        CHECK(copy_grid(c) == cdiv(vecs, 1024) * c.layers, "copy grid");
        ubw_kv_cache d = c;
        const int64_t values[] = {0, -1, 1, INT32_MAX, INT32_MIN, 24, 1 << 20};
        int* fields[] = {&d.dtype, &d.layers, &d.pages, &d.page_size, &d.kv_heads, &d.head_dim};
        *fields[rnd(r, 0, 5)] = (int)values[rnd(r, 0, 6)];
        (void)check_cache(&d);  // whatever it says: no overflow on the way
        d = c;
        const int64_t far[] = {-16, 8, INT64_MAX, INT64_MIN, (int64_t)1 << 41, ((int64_t)1 << 40) - 16};
        d.k_stride[rnd(r, 0, 3)] = far[rnd(r, 0, 5)];
        (void)check_cache(&d);
    }
    ubw_page_pool p{};
    CHECK(check_pool(nullptr) == UBW_EINVAL && check_pool(&p) == UBW_EINVAL, "pool");
    int32_t w[4];
    uint32_t u[4];
    p = ubw_page_pool{w, u, w, w, w, u, 1 << 24, 16, UBW_MAX_SEQS, 1 << 24};
    CHECK(check_pool(&p) == UBW_OK, "the largest pool");
    p.page_size = 1024;
    CHECK(check_pool(&p) == UBW_ERANGE, "lengths past 32 bits");
    p.page_size = 40;
    CHECK(check_pool(&p) == UBW_EUNSUPPORTED, "page size");
    alignas(16) char rows[64];
    CHECK(check_rows(rows, 64, 2, 1, 64, 2) == UBW_OK && check_rows(rows, 63, 2, 1, 64, 2) == UBW_EINVAL, "rows");
    CHECK(check_rows(rows, 0, 1, 1, 64, 2) == UBW_OK && check_rows(rows, 68, 2, 1, 64, 2) == UBW_EALIGN, "rows");
    CHECK(check_rows(rows + 8, 64, 2, 1, 64, 2) == UBW_EALIGN && check_rows(nullptr, 64, 2, 1, 64, 2) == UBW_EINVAL, "rows");
    CHECK(check_rows(rows, INT64_MAX, 2, 1, 64, 2) == UBW_ERANGE, "rows");
}

int main() {
    Rng r(7);
    check_cut(r);
    check_caches(r);
    if (fails) return 1;
    std::puts("ok");
    return 0;
}

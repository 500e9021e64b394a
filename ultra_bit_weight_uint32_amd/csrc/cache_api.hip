// C ABI of the key/value cache calls: argument validation and dispatch. Every check runs on the
// host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>

#include "cache_internal.h"

using namespace ubw::cache;

namespace {

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline int hip_status(hipError_t e) { return e == hipSuccess ? UBW_OK : UBW_EHIP; }
inline bool half_type(int t) { return t == UBW_F16 || t == UBW_BF16; }

// A one-element tensor dimension may come with any stride: the kernels never use it.
ubw_kv_cache with_used_strides(const ubw_kv_cache& c) {
    ubw_kv_cache o = c;
    const int64_t n[4] = {c.layers, c.pages, c.kv_heads, c.page_size};
    for (int i = 0; i < 4; ++i)
        if (n[i] == 1) o.k_stride[i] = o.v_stride[i] = 0;
    return o;
}

int check_table(const int32_t* table, int64_t ld, int cols) {
    if (!table || cols < 1 || ld < cols) return UBW_EINVAL;
    if (!aligned4(table)) return UBW_EALIGN;
    if (cols > (1 << 24) || ld > ((int64_t)1 << 40)) return UBW_ERANGE;
    return UBW_OK;
}

// What the attention calls check alike, and the arguments they share. UBW_OK with a.tokens == 0: nothing to do.
int attn_args(AttnArgs* to, const ubw_kv_cache* cache, const void* q, int q_dtype, int64_t ldq, int64_t tokens, int heads,
              const int32_t* q_start, const int32_t* ctx_len, int batch, const int32_t* table, int64_t ld_table, int table_cols,
              int max_tree, const uint64_t* masks, float scale, void* out, int64_t ldo, float* lse, int* head_dim) {
    if (!cache || tokens < 0 || batch < 0 || heads < 1 || max_tree < 1) return UBW_EINVAL;
    if (!(scale > 0.f) || !std::isfinite(scale)) return UBW_EINVAL;
    const ubw_kv_cache c = with_used_strides(*cache);
    int st = check_cache(&c);
    if (st != UBW_OK) return st;
    *head_dim = c.head_dim;
    if (heads % c.kv_heads != 0) return UBW_EINVAL;
    if (!half_type(q_dtype) || (c.dtype != UBW_E4M3 && c.dtype != q_dtype)) return UBW_EUNSUPPORTED;
    if (batch > UBW_MAX_SEQS || max_tree > UBW_MAX_TREE || tokens > (1 << 24) || heads > 65536 || heads / c.kv_heads > 1024)
        return UBW_ERANGE;
    if (tokens == 0 || batch == 0) return UBW_OK;
    if (!q_start || !ctx_len) return UBW_EINVAL;
    if ((st = check_table(table, ld_table, table_cols)) != UBW_OK) return st;
    if ((int64_t)table_cols * c.page_size > (1 << 30)) return UBW_ERANGE;  // positions stay clear of 2^31
    if ((st = check_rows(q, ldq, tokens, heads, c.head_dim, 2)) != UBW_OK ||
        (st = check_rows(out, ldo, tokens, heads, c.head_dim, 2)) != UBW_OK)
        return st;
    if ((reinterpret_cast<uintptr_t>(masks) & 7) || !aligned4(lse) || !aligned4(q_start) || !aligned4(ctx_len)) return UBW_EALIGN;
    AttnArgs a{};
    a.c = pages_of(c);
    a.q = q;
    a.out = out;
    a.ldq = ldq;
    a.ldo = ldo;
    a.tokens = (int)tokens;
    a.heads = heads;
    a.group = heads / c.kv_heads;
    a.batch = batch;
    a.q_start = q_start;
    a.ctx_len = ctx_len;
    a.table = table;
    a.ld_table = ld_table;
    a.table_cols = table_cols;
    a.max_tree = max_tree;
    a.masks = masks;
    a.scale = scale;
    a.lse = lse;
    *to = a;
    return UBW_OK;
}

// Scratch of `need` bytes: NULL with 0 bytes where it may be left out.
int check_workspace(const void* ws, size_t bytes, size_t need, bool may_lack) {
    if (!ws) return may_lack && bytes == 0 ? UBW_OK : UBW_EINVAL;
    if (!aligned16(ws)) return UBW_EALIGN;
    return bytes < need ? UBW_ESIZE : UBW_OK;
}

}  // namespace

extern "C" {

int ubw_qk_norm_rope(const ubw_kv_cache* cache, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                     int64_t ldv, int in_dtype, int64_t tokens, int heads, const float* q_weight, const float* k_weight,
                     float eps, const float* inv_freq, int rot, int interleaved, const int32_t* positions,
                     const int32_t* slots, void* q_out, int out_dtype, int64_t ldo, void* stream) {
    if (!cache || tokens < 0 || heads < 1 || rot < 0) return UBW_EINVAL;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return UBW_EINVAL;
    const ubw_kv_cache c = with_used_strides(*cache);
    int st = check_cache(&c);
    if (st != UBW_OK) return st;
    if (in_dtype != UBW_F32 && !half_type(in_dtype)) return UBW_EUNSUPPORTED;
    if (!half_type(out_dtype)) return UBW_EUNSUPPORTED;
    const int d = c.head_dim;
    if (rot > d || (rot & 1) || (!interleaved && rot % (d / 8) != 0)) return UBW_EUNSUPPORTED;
    if (tokens > kMaxGrid || heads > 65536) return UBW_ERANGE;
    if (tokens == 0) return UBW_OK;
    if (!positions || !slots || (rot > 0 && !inv_freq)) return UBW_EINVAL;
    const int size = type_size(in_dtype);
    if ((st = check_rows(q, ldq, tokens, heads, d, size)) != UBW_OK ||
        (st = check_rows(k, ldk, tokens, c.kv_heads, d, size)) != UBW_OK ||
        (st = check_rows(v, ldv, tokens, c.kv_heads, d, size)) != UBW_OK ||
        (st = check_rows(q_out, ldo, tokens, heads, d, 2)) != UBW_OK)
        return st;
    if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned4(inv_freq) || !aligned4(positions) || !aligned4(slots))
        return UBW_EALIGN;
    RopeArgs a{};
    a.c = pages_of(c);
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldo = ldo;
    a.tokens = (int)tokens;
    a.heads = heads;
    a.qw = q_weight;
    a.kw = k_weight;
    a.eps = eps;
    a.inv_freq = inv_freq;
    a.rot = rot;
    a.positions = positions;
    a.slots = slots;
    a.out = q_out;
    a.cache_dtype = c.dtype;
    a.out_dtype = out_dtype;
    return hip_status(launch_rope(a, in_dtype, d, interleaved != 0, as_stream(stream)));
}

int ubw_tree_attn_workspace_bytes(int batch, int max_tree, int heads, int kv_heads, int head_dim, size_t* out) {
    if (!out || batch < 0 || max_tree < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0) return UBW_EINVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return UBW_EUNSUPPORTED;
    if (batch > UBW_MAX_SEQS || max_tree > UBW_MAX_TREE || heads > 65536 || kv_heads > 4096 || heads / kv_heads > 1024)
        return UBW_ERANGE;
    *out = (size_t)attn_workspace_floats(batch, max_tree, heads / kv_heads, kv_heads, head_dim) * 4;
    return UBW_OK;
}

namespace {
// Positions that a sequence has at most, as the table or the caller says.
int64_t longest_of(const AttnArgs& a, int64_t max_len) {
    const int64_t room = (int64_t)a.table_cols << a.c.lps;
    return max_len > 0 && max_len < room ? max_len : room;
}
int run_attn(AttnArgs& a, int cache_dtype, int q_dtype, int d, int64_t max_len, void* stream) {
    const int64_t rows = (int64_t)a.max_tree * a.group;
    const AttnTile t = attn_tile(rows, d);
    a.max_items = attn_max_items(a.batch, rows, a.c.heads, d, t);
    if (a.max_items > kMaxGrid) return UBW_ERANGE;
    // short contexts are not split: one launch
    a.target = a.ws && longest_of(a, max_len) > attn_unsplit(t, d, (int64_t)a.batch * a.c.heads) ? attn_target(t, d) : 0;
    return hip_status(launch_attn(a, cache_dtype, q_dtype, d, t, as_stream(stream)));
}
}  // namespace

int ubw_tree_attn(const ubw_kv_cache* cache, const void* q, int q_dtype, int64_t ldq, int64_t tokens, int heads,
                  const int32_t* q_start, const int32_t* ctx_len, int batch, const int32_t* table, int64_t ld_table,
                  int table_cols, int max_tree, int64_t max_len, const uint64_t* masks, float scale, void* out,
                  int64_t ldo, float* lse, void* workspace, size_t ws_bytes, void* stream) {
    if (max_len < 0) return UBW_EINVAL;
    AttnArgs a{};
    int d = 0, st = attn_args(&a, cache, q, q_dtype, ldq, tokens, heads, q_start, ctx_len, batch, table, ld_table, table_cols,
                              max_tree, masks, scale, out, ldo, lse, &d);
    if (st != UBW_OK || a.tokens == 0) return st;
    size_t need = 0;
    if ((st = ubw_tree_attn_workspace_bytes(batch, max_tree, heads, a.c.heads, d, &need)) != UBW_OK ||
        (st = check_workspace(workspace, ws_bytes, need, true)) != UBW_OK)
        return st;
    a.ws = static_cast<float*>(workspace);
    return run_attn(a, cache->dtype, q_dtype, d, max_len, stream);
}

int ubw_prefix_attn_workspace_bytes(int batch, int groups, int64_t tokens, int max_tree, int heads, int kv_heads,
                                    int head_dim, size_t* out) {
    if (!out || batch < 0 || groups < 0 || tokens < 0 || max_tree < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
        return UBW_EINVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return UBW_EUNSUPPORTED;
    if (batch > UBW_MAX_SEQS || groups > UBW_MAX_SEQS || max_tree > UBW_MAX_TREE || tokens > (1 << 24) || heads > 65536 ||
        kv_heads > 4096 || heads / kv_heads > 1024 || tokens * (heads / kv_heads) > (1 << 30))
        return UBW_ERANGE;
    *out = (size_t)prefix_workspace_floats(batch, groups, tokens, max_tree, heads / kv_heads, kv_heads, head_dim) * 4;
    return UBW_OK;
}

int ubw_prefix_attn(const ubw_kv_cache* cache, const void* q, int q_dtype, int64_t ldq, int64_t tokens, int heads,
                    const int32_t* q_start, const int32_t* ctx_len, int batch, const int32_t* table, int64_t ld_table,
                    int table_cols, const int32_t* group_start, const int32_t* prefix_len, int groups, int max_tree,
                    int64_t max_len, const uint64_t* masks, float scale, void* out, int64_t ldo, float* lse, void* workspace,
                    size_t ws_bytes, void* stream) {
    if (max_len < 0 || groups < 0) return UBW_EINVAL;
    PrefixArgs a{};
    int d = 0, st = attn_args(&a, cache, q, q_dtype, ldq, tokens, heads, q_start, ctx_len, batch, table, ld_table, table_cols,
                              max_tree, masks, scale, out, ldo, lse, &d);
    if (st != UBW_OK || a.tokens == 0) return st;
    if (groups > 0 && (!group_start || !prefix_len)) return UBW_EINVAL;
    if (!aligned4(group_start) || !aligned4(prefix_len)) return UBW_EALIGN;
    size_t need = 0;
    if ((st = ubw_prefix_attn_workspace_bytes(batch, groups, tokens, max_tree, heads, a.c.heads, d, &need)) != UBW_OK ||
        (st = check_workspace(workspace, ws_bytes, need, false)) != UBW_OK)
        return st;
    a.ws = static_cast<float*>(workspace);
    const int64_t position_bytes = 2 * (int64_t)a.c.heads * d * type_size(cache->dtype);
    if (prefix_alone(batch, longest_of(a, max_len), position_bytes)) return run_attn(a, cache->dtype, q_dtype, d, max_len, stream);
    const PrefixSizes z = prefix_sizes(batch, groups, tokens, (int64_t)max_tree * a.group, a.group, a.c.heads, d);
    if (z.lists > kMaxGrid) return UBW_ERANGE;
    a.group_start = group_start;
    a.prefix_len = prefix_len;
    a.groups = groups;
    a.plan = reinterpret_cast<int*>(a.ws + z.rows * prefix_row_floats(d));
    return hip_status(launch_prefix_attn(a, cache->dtype, q_dtype, d, as_stream(stream)));
}

int ubw_page_bounds(const ubw_kv_cache* cache, void* bounds, const int32_t* table, int64_t ld_table, int table_cols,
                    const int32_t* start, const int32_t* stop, int batch, int64_t max_new, void* stream) {
    if (!cache || batch < 0 || max_new < 0) return UBW_EINVAL;
    const ubw_kv_cache c = with_used_strides(*cache);
    int st = check_cache(&c);
    if (st != UBW_OK) return st;
    if (batch > UBW_MAX_SEQS) return UBW_ERANGE;
    if (batch == 0) return UBW_OK;
    if (!bounds || !start || !stop) return UBW_EINVAL;
    if ((st = check_table(table, ld_table, table_cols)) != UBW_OK) return st;
    if (!aligned16(bounds) || !aligned4(start) || !aligned4(stop)) return UBW_EALIGN;
    BoundsArgs a{};
    a.c = pages_of(c);
    a.bounds = bounds;
    a.table = table;
    a.start = start;
    a.stop = stop;
    a.ld_table = ld_table;
    a.table_cols = table_cols;
    a.batch = batch;
    a.layers = c.layers;
    // pages that max_new positions fill at most
    const int64_t pages = max_new > 0 && cdiv(max_new, c.page_size) < table_cols ? cdiv(max_new, c.page_size) : table_cols;
    return hip_status(launch_page_bounds(a, c.dtype, c.head_dim, pages, as_stream(stream)));
}

int ubw_block_select_workspace_bytes(int64_t tokens, int kv_heads, int64_t max_blocks, size_t* out) {
    if (!out || tokens < 0 || kv_heads < 1 || max_blocks < 1) return UBW_EINVAL;
    if (tokens > (1 << 24) || kv_heads > 4096 || max_blocks > (1 << 24)) return UBW_ERANGE;
    *out = (size_t)tokens * kv_heads * max_blocks * 8;
    return UBW_OK;
}

int ubw_block_select(const void* bounds, int dtype, int pages, int page_size, int kv_heads, int head_dim, const void* q,
                     int q_dtype, int64_t ldq, int64_t tokens, int heads, const int32_t* q_start, const int32_t* ctx_len,
                     int batch, const int32_t* table, int64_t ld_table, int table_cols, int max_tree, int64_t max_len, int count,
                     int first, int last, int32_t* blocks, void* workspace, size_t ws_bytes, void* stream) {
    if (pages < 1 || kv_heads < 1 || tokens < 0 || heads < 1 || batch < 0 || max_tree < 1 || max_len < 0 || count < 1 || first < 0 ||
        last < 0 || first > count - last || heads % kv_heads != 0)
        return UBW_EINVAL;
    if (dtype != UBW_F16 && dtype != UBW_BF16 && dtype != UBW_E4M3) return UBW_EUNSUPPORTED;
    if (!half_type(q_dtype) || (dtype != UBW_E4M3 && dtype != q_dtype)) return UBW_EUNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return UBW_EUNSUPPORTED;
    if (!page_size_ok(page_size)) return UBW_EUNSUPPORTED;
    if (pages > (1 << 24) || (int64_t)pages * page_size > 0x7fffffff || kv_heads > 4096 || batch > UBW_MAX_SEQS ||
        max_tree > UBW_MAX_TREE || tokens > (1 << 24) || heads > 65536 || heads / kv_heads > 1024 || count > (1 << 20))
        return UBW_ERANGE;
    if (tokens == 0 || batch == 0) return UBW_OK;
    if (!bounds || !q_start || !ctx_len || !blocks) return UBW_EINVAL;
    int st = check_table(table, ld_table, table_cols);
    if (st != UBW_OK || (st = check_rows(q, ldq, tokens, heads, head_dim, 2)) != UBW_OK) return st;
    if ((int64_t)table_cols * page_size > (1 << 30)) return UBW_ERANGE;
    if (!aligned16(bounds) || !aligned4(q_start) || !aligned4(ctx_len) || !aligned4(blocks)) return UBW_EALIGN;
    // blocks there can be
    const int64_t most = max_len > 0 && max_len / page_size + 1 < table_cols ? max_len / page_size + 1 : table_cols;
    size_t need = 0;
    if ((st = ubw_block_select_workspace_bytes(tokens, kv_heads, most, &need)) != UBW_OK ||
        (st = check_workspace(workspace, ws_bytes, need, false)) != UBW_OK)
        return st;
    if (select_grid(kv_heads, most, max_tree) > kMaxGrid) return UBW_ERANGE;
    SelectArgs a{};
    a.bounds = bounds;
    a.q = q;
    a.ldq = ldq;
    a.tokens = (int)tokens;
    a.heads = heads;
    a.group = heads / kv_heads;
    a.kv = kv_heads;
    a.batch = batch;
    a.pages = pages;
    a.lps = log2_of(page_size);
    a.q_start = q_start;
    a.ctx_len = ctx_len;
    a.table = table;
    a.ld_table = ld_table;
    a.table_cols = table_cols;
    a.max_tree = max_tree;
    a.count = count;
    a.first = first;
    a.last = last;
    a.blocks = blocks;
    a.keys = static_cast<uint64_t*>(workspace);
    a.stride = (int)most;
    return hip_status(launch_block_select(a, dtype, q_dtype, head_dim, as_stream(stream)));
}

int ubw_block_attn_workspace_bytes(int64_t tokens, int heads, int kv_heads, int head_dim, size_t* out) {
    if (!out || tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0) return UBW_EINVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return UBW_EUNSUPPORTED;
    if (tokens > (1 << 24) || heads > 65536 || kv_heads > 4096 || heads / kv_heads > 1024) return UBW_ERANGE;
    *out = (size_t)block_workspace_floats(tokens, heads / kv_heads, kv_heads, head_dim) * 4;
    return UBW_OK;
}

int ubw_block_attn(const ubw_kv_cache* cache, const void* q, int q_dtype, int64_t ldq, int64_t tokens, int heads,
                   const int32_t* q_start, const int32_t* ctx_len, int batch, const int32_t* table, int64_t ld_table,
                   int table_cols, const int32_t* blocks, int count, int max_tree, const uint64_t* masks, float scale, void* out,
                   int64_t ldo, float* lse, void* workspace, size_t ws_bytes, void* stream) {
    if (count < 0) return UBW_EINVAL;
    BlockArgs a{};
    int d = 0, st = attn_args(&a, cache, q, q_dtype, ldq, tokens, heads, q_start, ctx_len, batch, table, ld_table, table_cols,
                              max_tree, masks, scale, out, ldo, lse, &d);
    if (st != UBW_OK || a.tokens == 0) return st;
    if (count > 0 && !blocks) return UBW_EINVAL;
    if (!aligned4(blocks)) return UBW_EALIGN;
    if (count > (1 << 20) || block_positions(count, cache->page_size, max_tree) > (1 << 30)) return UBW_ERANGE;
    size_t need = 0;
    if ((st = ubw_block_attn_workspace_bytes(tokens, heads, a.c.heads, d, &need)) != UBW_OK ||
        (st = check_workspace(workspace, ws_bytes, need, true)) != UBW_OK)
        return st;
    const int64_t pairs = block_pairs(tokens, a.group, a.c.heads, block_tile(a.group, d));
    a.splits = workspace ? block_splits(pairs, block_positions(count, cache->page_size, max_tree)) : 1;
    if (block_cap(pairs) > kMaxGrid) return UBW_ERANGE;
    a.blocks = blocks;
    a.count = count;
    a.ws = static_cast<float*>(workspace);
    a.cut = workspace ? reinterpret_cast<int*>(a.ws + block_floats(tokens, a.group, a.c.heads, d)) : nullptr;
    return hip_status(launch_block_attn(a, cache->dtype, q_dtype, d, as_stream(stream)));
}

int ubw_cache_copy_pages(const ubw_kv_cache* cache, const int32_t* pairs, int64_t count, void* stream) {
    if (!cache || count < 0) return UBW_EINVAL;
    const ubw_kv_cache c = with_used_strides(*cache);
    int st = check_cache(&c);
    if (st != UBW_OK) return st;
    if (count > (1 << 20) || copy_grid(c) > kMaxGrid) return UBW_ERANGE;
    if (count == 0) return UBW_OK;
    if (!pairs) return UBW_EINVAL;
    if (!aligned4(pairs)) return UBW_EALIGN;
    return hip_status(launch_copy_pages(pages_of(c), c.layers, c.page_size, c.head_dim * type_size(c.dtype), pairs,
                                        (int)count, as_stream(stream)));
}

int ubw_cache_compact(const ubw_kv_cache* cache, const int32_t* table, int64_t ld_table, int table_cols,
                      const int32_t* ctx_len, const int32_t* keep, int width, int batch, void* stream) {
    if (!cache || width < 0 || batch < 0) return UBW_EINVAL;
    const ubw_kv_cache c = with_used_strides(*cache);
    int st = check_cache(&c);
    if (st != UBW_OK) return st;
    if (batch > UBW_MAX_SEQS || width > 1024 || compact_grid(c) > kMaxGrid) return UBW_ERANGE;
    if (batch == 0 || width == 0) return UBW_OK;
    if (!ctx_len || !keep) return UBW_EINVAL;
    if (!aligned4(ctx_len) || !aligned4(keep)) return UBW_EALIGN;
    if ((st = check_table(table, ld_table, table_cols)) != UBW_OK) return st;
    return hip_status(launch_compact(pages_of(c), c.layers, c.head_dim * type_size(c.dtype), table, ld_table, table_cols,
                                     ctx_len, keep, width, batch, as_stream(stream)));
}

int ubw_pages_init(const ubw_page_pool* pool, void* stream) {
    const int st = check_pool(pool);
    return st != UBW_OK ? st : hip_status(launch_pages_init(*pool, as_stream(stream)));
}

int ubw_pages_trim(const ubw_page_pool* pool, const int32_t* new_len, void* stream) {
    const int st = check_pool(pool);
    if (st != UBW_OK) return st;
    if (!new_len) return UBW_EINVAL;
    if (!aligned4(new_len)) return UBW_EALIGN;
    return hip_status(launch_pages_trim(*pool, new_len, as_stream(stream)));
}

int ubw_pages_fork(const ubw_page_pool* pool, const int32_t* parents, void* stream) {
    const int st = check_pool(pool);
    if (st != UBW_OK) return st;
    if (!parents) return UBW_EINVAL;
    if (!aligned4(parents)) return UBW_EALIGN;
    return hip_status(launch_pages_fork(*pool, parents, as_stream(stream)));
}

int ubw_pages_reserve(const ubw_page_pool* pool, const int32_t* room, int32_t* pairs, void* stream) {
    const int st = check_pool(pool);
    if (st != UBW_OK) return st;
    if (!room || !pairs) return UBW_EINVAL;
    if (!aligned4(room) || !aligned4(pairs)) return UBW_EALIGN;
    return hip_status(launch_pages_reserve(*pool, room, pairs, as_stream(stream)));
}

}  // extern "C"

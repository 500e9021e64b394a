// Internal declarations of the key/value cache calls (cache_api.hip, rope.hip, attn.hip, pages.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ubw.h"
#include "cache_plan.h"

namespace ubw {
namespace cache {

// A cache as the kernels take it: byte strides, one layer first.
struct Pages {
    char* k;
    char* v;
    int64_t k_layer, k_page, k_head, v_layer, v_page, v_head;  // bytes
    uint32_t k_row, v_row;                                     // bytes
    int pages, lps, heads;                                     // lps: log2 of the page size
    const float* k_scale;
    const float* v_scale;
};
inline Pages pages_of(const ubw_kv_cache& c) {
    const int64_t s = type_size(c.dtype);
    Pages p{};
    p.k = static_cast<char*>(c.k);
    p.v = static_cast<char*>(c.v);
    p.k_layer = c.k_stride[0] * s;
    p.k_page = c.k_stride[1] * s;
    p.k_head = c.k_stride[2] * s;
    p.k_row = (uint32_t)(c.k_stride[3] * s);
    p.v_layer = c.v_stride[0] * s;
    p.v_page = c.v_stride[1] * s;
    p.v_head = c.v_stride[2] * s;
    p.v_row = (uint32_t)(c.v_stride[3] * s);
    p.pages = c.pages;
    p.lps = log2_of(c.page_size);
    p.heads = c.kv_heads;
    p.k_scale = c.dtype == UBW_E4M3 ? c.k_scale : nullptr;
    p.v_scale = c.dtype == UBW_E4M3 ? c.v_scale : nullptr;
    return p;
}

struct RopeArgs {
    Pages c;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo;  // elements
    int tokens, heads;
    const float *qw, *kw;
    float eps;
    const float* inv_freq;
    int rot;
    const int32_t *positions, *slots;
    void* out;
    int cache_dtype, out_dtype;
};
hipError_t launch_rope(const RopeArgs& a, int in_dtype, int head_dim, bool interleaved, hipStream_t s);

struct AttnArgs {
    Pages c;
    const void* q;
    void* out;
    int64_t ldq, ldo;  // elements
    int tokens, heads, group, batch;
    const int32_t *q_start, *ctx_len, *table;
    int64_t ld_table;
    int table_cols, max_tree;
    const uint64_t* masks;
    float scale;
    float* lse;
    float* ws;
    int64_t max_items;  // pieces the workspace holds (ws != nullptr)
    int target;         // pieces aimed at; 0: contexts are not split
};
hipError_t launch_attn(const AttnArgs& a, int cache_dtype, int q_dtype, int head_dim, AttnTile t, hipStream_t s);

hipError_t launch_copy_pages(const Pages& c, int layers, int page_size, int row_bytes, const int32_t* pairs, int count,
                             hipStream_t s);
hipError_t launch_compact(const Pages& c, int layers, int row_bytes, const int32_t* table, int64_t ld_table,
                          int table_cols, const int32_t* ctx_len, const int32_t* keep, int width, int batch,
                          hipStream_t s);
hipError_t launch_pages_init(const ubw_page_pool& p, hipStream_t s);
hipError_t launch_pages_trim(const ubw_page_pool& p, const int32_t* new_len, hipStream_t s);
hipError_t launch_pages_fork(const ubw_page_pool& p, const int32_t* parents, hipStream_t s);
hipError_t launch_pages_reserve(const ubw_page_pool& p, const int32_t* room, int32_t* pairs, hipStream_t s);

}  // namespace cache
}  // namespace ubw

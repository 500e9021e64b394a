// Argument checks and launch planning of the key/value cache calls: plain integer arithmetic with
// no HIP dependency, shared by the host code, the kernels (functions marked UBW_HD) and a host test
// program built with address and undefined-behaviour sanitizers.
#pragma once
#include <stdint.h>

#include "plan.h"

namespace ubw {
namespace cache {

using plan::aligned16;
using plan::cdiv;

inline int type_size(int dtype) {
    return dtype == UBW_F32 ? 4 : dtype == UBW_F16 || dtype == UBW_BF16 ? 2 : dtype == UBW_E4M3 ? 1 : 0;
}
// Workgroups of 256 threads in one grid dimension: work-items there are counted in 32 bits.
constexpr int64_t kMaxGrid = (1 << 24) - 1;
constexpr int kCopyVecs = 4;  // 16-byte vectors a copying thread has in flight

inline bool page_size_ok(int ps) { return ps >= 16 && ps <= 1024 && (ps & (ps - 1)) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int log2_of(int pow2) {
    int l = 0;
    while ((1 << l) < pow2) ++l;
    return l;
}

// Strides of k or v: multiples of 16 bytes, rows of a page reached from the page's first element
// with 32-bit byte offsets over 16 rows, and offsets of the whole cache within 63 bits.
inline int check_strides(const int64_t* st, const ubw_kv_cache& c, int size) {
    const int64_t most = (int64_t)1 << 40;
    const int64_t n[4] = {c.layers, c.pages, c.kv_heads, c.page_size};
    for (int i = 0; i < 4; ++i) {
        if (st[i] < 0 || st[i] > most) return UBW_ERANGE;
        if ((st[i] * size) & 15) return UBW_EALIGN;
        if (n[i] > 1 && st[i] < c.head_dim) return UBW_EINVAL;
        if (st[i] > 0 && n[i] > ((int64_t)1 << 60) / st[i]) return UBW_ERANGE;
    }
    if (st[3] * size * 16 >= ((int64_t)1 << 31)) return UBW_ERANGE;
    return UBW_OK;
}

inline int check_cache(const ubw_kv_cache* c) {
    if (!c || !c->k || !c->v || c->layers < 1 || c->pages < 1 || c->kv_heads < 1) return UBW_EINVAL;
    if (c->dtype != UBW_F16 && c->dtype != UBW_BF16 && c->dtype != UBW_E4M3) return UBW_EUNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return UBW_EUNSUPPORTED;
    if (!page_size_ok(c->page_size)) return UBW_EUNSUPPORTED;
    if (c->pages > (1 << 24) || c->kv_heads > 4096 || c->layers > 65536) return UBW_ERANGE;
    if ((int64_t)c->pages * c->page_size > 0x7fffffff) return UBW_ERANGE;  // slots are int32
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale)) return UBW_EALIGN;
    const int size = type_size(c->dtype);
    int st = check_strides(c->k_stride, *c, size);
    return st != UBW_OK ? st : check_strides(c->v_stride, *c, size);
}

// Rows of heads x head_dim values, ld elements apart.
inline int check_rows(const void* p, int64_t ld, int64_t rows, int heads, int dim, int size) {
    if (!p) return UBW_EINVAL;
    if (rows > 1 && ld < (int64_t)heads * dim) return UBW_EINVAL;
    if (ld < 0 || ld > ((int64_t)1 << 36)) return UBW_ERANGE;
    if (!aligned16(p) || ((ld * size) & 15)) return UBW_EALIGN;
    return UBW_OK;
}

// Workgroups that copy one page in every layer, and that compact one sequence.
inline int64_t copy_grid(const ubw_kv_cache& c) {
    return cdiv((int64_t)c.kv_heads * c.page_size * (c.head_dim * type_size(c.dtype) / 16), 256 * kCopyVecs) * c.layers;
}
inline int64_t compact_grid(const ubw_kv_cache& c) {
    return cdiv((int64_t)c.layers * 2 * c.kv_heads * (c.head_dim * type_size(c.dtype) / 16), 256);
}

inline int check_pool(const ubw_page_pool* p) {
    if (!p || !p->ref || !p->free_bits || !p->table || !p->held || !p->len || !p->status) return UBW_EINVAL;
    if (p->pages < 1 || p->seqs < 1 || p->max_pages < 1) return UBW_EINVAL;
    if (!page_size_ok(p->page_size)) return UBW_EUNSUPPORTED;
    if (p->pages > (1 << 24) || p->seqs > UBW_MAX_SEQS || p->max_pages > (1 << 24)) return UBW_ERANGE;
    if ((int64_t)p->max_pages * p->page_size > 0x7fffffff) return UBW_ERANGE;  // lengths are int32
    if (!aligned4(p->ref) || !aligned4(p->free_bits) || !aligned4(p->table) || !aligned4(p->held) || !aligned4(p->len) ||
        !aligned4(p->status))
        return UBW_EALIGN;
    return UBW_OK;
}

// ---- tree attention -------------------------------------------------------------------------
// The rows of a (sequence, key/value head): row r is token r / G, query head h G + r % G (G =
// heads / kv_heads). A workgroup takes a block of rows and a run of positions, in units of 128.
// row_waves waves lie side by side over rows, each with `tiles` times 16 of them; waves over the same
// rows (four or two with one row wave, two with two) take 32 positions in turn.
struct AttnTile {
    int tiles, row_waves;
};
constexpr int kAttnUnit = 128;
UBW_HD inline int attn_rows(AttnTile t) { return 16 * t.tiles * t.row_waves; }
inline AttnTile attn_tile(int64_t max_rows, int head_dim) {
    if (head_dim == 256) return AttnTile{1, max_rows <= 16 ? 1 : 4};  // the sums of 256 dims take 64 registers per tile
    if (max_rows <= 16) return AttnTile{1, 1};
    if (max_rows <= 32) return AttnTile{2, 1};
    if (max_rows <= 64) return AttnTile{2, 2};
    return AttnTile{2, 4};
}

// Contexts of up to this many positions (with their tokens) are not split: a few more steps of one
// workgroup take less than cutting the batch and joining its pieces in a second launch. The limit goes by
// the positions that a workgroup takes in one step: 128 with one row wave (64 dims and 128), of 256 dims 64;
// two row waves 64, four 64 and of 256 dims 32. Times in us split / not, one sequence and (behind the
// semicolon) eight, 8 key/value heads, 16 bits:
//   128 dims:   8 rows at 500 positions 13.4 / 10.6; 15.0 / 12.0, at 760 13.5 / 12.9; 17.6 / 15.8, at 1000 13.4 / 15.2; 18.1 / 18.9
//              48 rows at 380 16.0 / 15.8; 19.6 / 16.4, at 760 16.0 / 20.9; 25.1 / 23.3
//             128 rows at 250 18.5 / 17.1; 27.0 / 17.5, at 380 18.8 / 20.5; 28.3 / 21.1, at 500 18.8 / 23.8; 34.3 / 24.5
//    64 dims:   8 rows at 760 12.0 / 9.8; 14.5 / 10.2, at 1000 11.9 / 11.1; 14.6 / 12.2
//              48 rows at 380 13.8 / 11.7; 15.9 / 12.0, at 760 13.9 / 15.3; 18.3 / 15.6
//             128 rows at 250 15.9 / 13.1; 20.8 / 13.3, at 380 16.2 / 15.7; 21.8 / 16.1
//   256 dims:   8 rows at 250 17.0 / 15.3; 18.6 / 15.9, at 380 17.1 / 19.0; 19.4 / 19.8
//              48 rows at 120 15.9 / 11.7; 16.2 / 12.0, at 250 18.3 / 16.7; 21.9 / 17.5
// 64 (sequence, key/value head) pairs or more, as the eight sequences here, use a quarter of the card
// without a split; for them the limit of more than 32 rows (64 and 128 dims) is twice as high.
inline int attn_unsplit(AttnTile t, int head_dim, int64_t pairs) {
    if (head_dim == 256) return t.row_waves == 1 ? 256 : 128;
    return t.row_waves == 1 ? 768 : (t.row_waves == 2 ? 384 : 256) * (pairs >= 64 ? 2 : 1);
}

// How a batch is cut: sequence b has blocks_b row blocks of units_b units of positions for each
// key/value head; a piece is one block over `chunk` units at most, a sequence's pieces of equal size
// but for one unit. chunk starts at total / target and grows while there are more pieces than that.
// How many pieces a batch is aimed to have, at most: with one row wave three for each workgroup that is
// resident, with more one (their sums are larger).
inline int attn_target(AttnTile t, int head_dim) { return t.row_waves == 1 ? 1536 : head_dim == 64 ? 768 : 512; }
// ... and for this many units: three a workgroup only where each still has kAttnLong units or more, so
// that starting a piece costs little beside it.
constexpr int kAttnLong = 8;
UBW_HD inline int attn_aim(int64_t total_units, int target, bool one_row_wave) {
    return one_row_wave && total_units < (int64_t)target * kAttnLong ? target / 3 : target;
}
constexpr int kAttnMostChunk = 1 << 25;  // more than the units of 2^31 positions
UBW_HD inline int attn_chunk(int64_t total_units, int target) {
    const int64_t c = (total_units + target - 1) / target;
    return (int)(c < 1 ? 1 : c < kAttnMostChunk ? c : kAttnMostChunk);
}
// (Where even whole sequences are more pieces than the target it would grow without end.)
UBW_HD inline int attn_larger_chunk(int chunk, int64_t pieces, int target) {
    const int64_t c = (chunk * pieces + target - 1) / target;
    const int64_t next = c > chunk ? c : chunk + (int64_t)1;
    return (int)(next < kAttnMostChunk ? next : kAttnMostChunk);
}
UBW_HD inline int attn_splits(int units, int chunk) { return units == 0 ? 0 : (units + chunk - 1) / chunk; }
UBW_HD inline void attn_range(int units, int splits, int s, int* u0, int* u1) {
    const int q = units / splits, r = units - q * splits;
    *u0 = s * q + (s < r ? s : r);
    *u1 = *u0 + q + (s < r ? 1 : 0);
}
// Most pieces of a batch: the sum over sequences of blocks kv ceil(units / chunk) is at most
// total / chunk + batch blocks kv <= target + batch blocks kv.
inline int64_t attn_max_items(int batch, int64_t max_rows, int kv_heads, int head_dim, AttnTile t) {
    return attn_target(t, head_dim) + (int64_t)batch * cdiv(max_rows, attn_rows(t)) * kv_heads;
}
// Scratch floats: each piece's rows (head_dim means, then the running maximum and the sum of weights),
// then the cut itself (units per piece, each sequence's first piece); for trees of max_tree tokens or
// fewer, whose pieces have other sizes.
inline int64_t attn_workspace_floats(int batch, int max_tree, int group, int kv_heads, int head_dim) {
    int64_t most = 0;
    for (int n = 1; n <= max_tree; ++n) {
        const int64_t rows = (int64_t)n * group;
        const AttnTile t = attn_tile(rows, head_dim);
        const int64_t x = attn_max_items(batch, rows, kv_heads, head_dim, t) * attn_rows(t) * (head_dim + 2);
        most = x > most ? x : most;
    }
    return most + batch + 1;
}

}  // namespace cache
}  // namespace ubw

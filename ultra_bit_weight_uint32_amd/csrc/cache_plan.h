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

// ---- attention over shared prefixes ---------------------------------------------------------
// An owner is a group, with its tokens' rows over its prefix, or a sequence, with its rows over what is behind it. Its
// rows lie in blocks of 128 (64 of 256 dims), the last up to 32 in a block of a smaller tile; a list is a block of a
// key/value head with the owner's positions, in units of 128. What lists cost is known well enough to deal them out
// beforehand (trees of 1 to 16 tokens behind five prefixes of 3K to 40K positions in 8 bits: 4.0 us a unit at any
// number of rows, with the small tile 1.5; single tokens behind one of 16K in 16 bits: 4.5 and 2.6; 8 to 10 us to begin
// and end a piece): every one of 512 workgroups is to have the same. So lists are cut into full pieces, one to a
// workgroup, as long as that allows, and a rest; the workgroups without a full piece share out the rests, the longest
// first, in runs of the same cost. (Where these would have too much the full pieces are made longer.)
constexpr int kPrefixWgs = 512;  // two on every CU
constexpr int kUnitCost = 7, kSmallUnitCost = 4, kSmallUnitCost8 = 3, kPieceCost = 16;  // in 0.64 us; 8: 8-bit caches
constexpr int kSmallRows = 32;
UBW_HD inline int prefix_rows(int head_dim) { return head_dim == 256 ? 64 : 128; }
// What a workgroup is to have, for lists of this cost in all.
UBW_HD inline int64_t prefix_goal(int64_t cost) { return (cost + kPrefixWgs - 1) / kPrefixWgs + kPieceCost; }
UBW_HD inline int prefix_full(int64_t goal, int unit_cost) {  // units of a full piece
    const int64_t n = (goal - kPieceCost) / unit_cost;
    return (int)(n < 1 ? 1 : n < kAttnMostChunk ? n : kAttnMostChunk);
}
// How a list of `units` is cut: full pieces, and what is behind them (an eighth of one or less is spread over them).
struct PrefixCut {
    int full, rest;
};
UBW_HD inline PrefixCut prefix_cut(int units, int length) {
    PrefixCut c{units / length, units % length};
    if (c.full > 0 && c.rest <= length / 8) c.rest = 0;
    return c;
}
// Full pieces: a list of u units has at most u / length of them, and length >= (goal - kPieceCost) / (2 unit_cost), so
// that they are at most 2 cost / (cost / 512).
constexpr int kPrefixFull = 2 * kPrefixWgs;
// The rests lie in buckets by what they cost, the dearest first. Costs and rooms are whole numbers, in 2^-16 of a goal, at
// most 2^17 for a rest and 2^41 for all: no sum of them depends on the order of summing, so that every workgroup finds
// its run's beginning by the same sums as the next one finds its end. (In 32 bits, each workgroup's rounded its own way, a run
// could begin one rest before the end of the one before it, whose workgroup then left out one of its long rests.)
constexpr int kRestBuckets = 64;
UBW_HD inline int rest_bucket(int rest, int unit_cost, float scale) {  // scale: kRestBuckets / goal
    const int x = (int)((float)rest * (float)unit_cost * scale);
    return kRestBuckets - 1 - (x < kRestBuckets - 1 ? x : kRestBuckets - 1);
}
UBW_HD inline int64_t rest_begin_cost(int64_t goal) { return ((int64_t)kPieceCost << 16) / goal; }  // (goal >= kPieceCost)
// What a rest of bucket b costs: the middle of the bucket, and to begin and end it.
UBW_HD inline int64_t rest_cost(int b, int64_t begin) { return (2 * (kRestBuckets - b) - 1) * ((int64_t)1 << 16) / (2 * kRestBuckets) + begin; }
// Workgroups for the rests: each XCD's that have no full piece (all, if it has as many full pieces as workgroups).
UBW_HD inline int rest_bins(int full) {
    const int per = (full + 7) >> 3;
    return per < kPrefixWgs / 8 ? kPrefixWgs - 8 * per : kPrefixWgs;
}
// Lengths are whole units, so that full pieces can be more than workgroups, or leave fewer of them to the rests, which
// cost `rests` in all, than they were to: longer ones then (64 single tokens behind six prefixes of 6K to 12K positions, one
// head of 256 dims, three units a piece: 64 rests on 8 workgroups 120 us, with longer pieces 55).
constexpr int kPrefixTurns = 6;
UBW_HD inline bool prefix_fits(int full, int64_t rests, int64_t goal, int64_t full_cost) {
    return full <= kPrefixWgs && (float)rests * (float)goal <= 1.25f * 65536.f * (float)full_cost * (float)rest_bins(full);
}
UBW_HD inline int64_t prefix_longer(int64_t full_cost) {
    const int64_t more = (full_cost - kPieceCost) / 8;
    return full_cost + (more > kUnitCost ? more : kUnitCost);
}
// Long rests, of more than a quarter of what such a workgroup is to have, go there and back over them; the others, in
// order, fill up what those leave free. The buckets of long ones:
UBW_HD inline int long_buckets(int64_t have, int64_t begin) {
    int lo = 0, hi = kRestBuckets;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (4 * rest_cost(mid, begin) > have) lo = mid + 1; else hi = mid;
    }
    return lo;
}
// The n-th of the long rests that the w-th of the workgroups has: there and back.
UBW_HD inline int rest_at(int n, int w, int bins) { return n * bins + (n & 1 ? bins - 1 - w : w); }
// What the long ones leave free of the w-th. before: rests in the buckets before each one.
UBW_HD inline int64_t rest_room(int w, int bins, int longs, int64_t have, const int* before, int64_t begin) {
    int64_t room = have;
    for (int n = 0;; ++n) {
        const int k = rest_at(n, w, bins);
        if (k >= longs) break;
        int from = 0, end = kRestBuckets;  // its bucket: the last that begins at k or before
        while (end - from > 1) {
            const int mid = (from + end) >> 1;
            if (before[mid] <= k) from = mid; else end = mid;
        }
        room -= rest_cost(from, begin);
    }
    return room > 0 ? room : 0;
}
// The first of the other rests of the workgroup that has `room` of `rooms` before it. before, cost: rests in the buckets
// before each one, and what they cost; longs: buckets of long ones. Where room ascends it does not descend: whole
// numbers of this size are doubles, a quotient, a product and a sum with the same numbers, however they are rounded,
// turn no order around, and a bucket's rests are all behind those of the one before it.
UBW_HD inline int rest_run(int64_t room, int64_t rooms, const int* before, const int64_t* cost, int longs, int64_t begin) {
    if (longs == kRestBuckets) return before[kRestBuckets];
    const double left = (double)(cost[kRestBuckets] - cost[longs]);
    const double from = (double)cost[longs] + (rooms > 0 ? (double)room / (double)rooms * left : 0.0);
    int b = longs, end = kRestBuckets;
    while (end - b > 1) {
        const int mid = (b + end) >> 1;
        if ((double)cost[mid] <= from) b = mid; else end = mid;
    }
    const int n = before[b + 1] - before[b];
    const double k = (from - (double)cost[b]) / (double)rest_cost(b, begin);  // (from >= cost[longs])
    const int up = (int)(k < (double)n ? k : (double)n);
    return before[b] + (up < n && (double)up < k ? up + 1 : up);
}
// What workgroup wg has of `full` full pieces, `longs` long rests and the others, which begin at run[w] for the w-th
// workgroup with rests. Each XCD has an eighth of the full pieces, in order.
struct PrefixShare {
    int full0, fulls;  // full pieces full0, full0 + kPrefixWgs / 8, ..
    int bin, bins;     // among the workgroups with rests
    int longs;         // long rests
    int rest0, rests;  // others
};
template <typename Run>
UBW_HD inline PrefixShare prefix_share(int wg, int full, int longs, Run run) {
    const int xcd = wg & 7, i = wg >> 3, per = (full + 7) >> 3, wide = kPrefixWgs / 8;
    const int left = full - xcd * per, mine = left < per ? left : per, taken = per < wide ? per : 0;
    PrefixShare s{xcd * per + i, i < mine ? (mine - i + wide - 1) / wide : 0, (i - taken) * 8 + xcd, rest_bins(full), 0, 0, 0};
    if (i >= taken) {
        s.rest0 = run[s.bin];
        s.rests = run[s.bin + 1] - s.rest0;
        while (rest_at(s.longs, s.bin, s.bins) < longs) ++s.longs;
    }
    return s;
}
// Its n-th piece, in the plan's list (the full ones, then the rests at kPrefixFull); -1 behind the last.
UBW_HD inline int prefix_work(const PrefixShare& s, int n) {
    if (n < s.fulls) return s.full0 + n * (kPrefixWgs / 8);
    const int k = n - s.fulls;
    if (k >= s.longs + s.rests) return -1;
    return kPrefixFull + (k < s.longs ? rest_at(k, s.bin, s.bins) : s.rest0 + k - s.longs);
}
// The workspace: sums of the full pieces (head_dim means, maximum, sum, two unused words a row), of the rests of each
// (token, head) over the own positions and over the prefix; the plan: a head, sixteen words an owner, two words a piece.
constexpr int kPlanHead = 16 + kPrefixWgs, kPlanOwner = 16;
struct PrefixSizes {
    int64_t lists;  // most lists
    int64_t rows;   // rows of sums
    int64_t words;  // of the plan
};
inline PrefixSizes prefix_sizes(int batch, int groups, int64_t tokens, int64_t max_rows, int group, int kv_heads, int head_dim) {
    const int rb = prefix_rows(head_dim);
    PrefixSizes p{};
    p.lists = ((groups > 0 ? tokens * group / rb + groups : 0) + batch * cdiv(max_rows, rb)) * kv_heads;
    p.rows = (int64_t)kPrefixFull * rb + 2 * tokens * group * kv_heads;
    p.words = kPlanHead + kPlanOwner * ((int64_t)groups + batch) + 2 * (kPrefixFull + p.lists);
    return p;
}
inline int64_t prefix_row_floats(int head_dim) { return head_dim + 4; }
inline int64_t prefix_workspace_floats(int batch, int groups, int64_t tokens, int max_tree, int group, int kv_heads, int head_dim) {
    const PrefixSizes p = prefix_sizes(batch, groups, tokens, (int64_t)max_tree * group, group, kv_heads, head_dim);
    const int64_t alone = attn_workspace_floats(batch, max_tree, group, kv_heads, head_dim);
    const int64_t x = p.rows * prefix_row_floats(head_dim) + p.words;
    return x > alone ? x : alone;
}
// Where all sequences' contexts, each as long as the longest may be, are up to 96 MiB of keys and values, tree attention
// goes through them: it has one launch or two, not three. Times in us, tree attention / shared; one group, 60 positions
// behind the prefix, 64 heads over 8 of 128 dims, 16 bits, single tokens unless stated:
//   4 sequences of 250 positions (5 MB) 10.9 / 21.7, of 1000 (17) 17.8 / 22.0, of 4000 (67) 24.4 / 27.2, of 16000 (263) 54.7 / 47.8
//   64 of 250 (82) 14.2 / 33.2; 16 of 1000 (70) 26.5 / 25.9, of 4000 (266) 54.7 / 34.7, of 4000 in 8 bits (133) 34.5 / 33.7
//   trees of 8: 4 of 4000 (67) 36.2 / 43.0, 16 of 1000 (70) 38.2 / 38.3, of 4000 (267) 63.5 / 56.6
//   32 heads over 32: 4 of 1000 (70) 27.1 / 24.1, 2 of 4000 (133) 31.7 / 33.1, 4 of 4000 (266) 53.1 / 33.4
//   16 heads over 2 of 256 dims: 16 of 1000 (35) 21.1 / 23.4, 4 of 16000 (132) 34.7 / 30.4
constexpr int64_t kPrefixLeast = (int64_t)96 << 20;
inline bool prefix_alone(int64_t batch, int64_t longest, int64_t position_bytes) { return batch * longest <= kPrefixLeast / position_bytes; }

// ---- selected blocks ------------------------------------------------------------------------
// Attention over them: a token and key/value head have their rows (the head's queries) and positions to
// themselves. Their number is bounded by the list's length, which the host knows, and so is the cut.
inline int64_t block_positions(int count, int page_size, int max_tree) { return (int64_t)count * page_size + page_size - 1 + max_tree; }
inline AttnTile block_tile(int group, int head_dim) {
    return group <= 16 ? AttnTile{1, 1} : AttnTile{head_dim == 256 ? 1 : 2, 4};
}
inline int64_t block_pairs(int64_t tokens, int group, int kv_heads, AttnTile t) { return tokens * kv_heads * cdiv(group, attn_rows(t)); }
constexpr int kBlockTarget = 512;  // pieces aimed at
inline int block_splits(int64_t pairs, int64_t positions) {
    const int64_t units = cdiv(positions, kAttnUnit), want = pairs > 0 ? cdiv(kBlockTarget, pairs) : 1;
    return (int)(want < units ? want : units);
}
inline int64_t block_cap(int64_t pairs) { return kBlockTarget + pairs; }
inline int64_t block_floats(int64_t tokens, int group, int kv_heads, int head_dim) {
    const AttnTile t = block_tile(group, head_dim);
    return block_cap(block_pairs(tokens, group, kv_heads, t)) * attn_rows(t) * (head_dim + 2);
}
inline int64_t block_workspace_floats(int64_t tokens, int group, int kv_heads, int head_dim) {
    return block_floats(tokens, group, kv_heads, head_dim) + tokens * kv_heads;
}

// Bounds of pages: a group of lanes takes one page of one head in one layer. Groups for each sequence: as many as
// its pages ask for, as far as the card holds them (each then takes several in turn).
inline int64_t bounds_groups(int64_t layers, int kv_heads, int batch, int64_t pages) {
    const int64_t all = layers * kv_heads * pages, most = cdiv((int64_t)1 << 18, batch);
    return all < most ? all : most;
}

// Scores of blocks: blocks of one sequence and head that a workgroup takes.
constexpr int kScoreBlocks = 64, kScoreBlocksTree = 256;
inline int64_t select_grid(int kv_heads, int64_t blocks, int max_tree) {
    const int64_t scores = cdiv(blocks, max_tree == 1 ? kScoreBlocks : kScoreBlocksTree) * kv_heads, rows = (int64_t)max_tree * kv_heads;
    return scores > rows ? scores : rows;
}

}  // namespace cache
}  // namespace ubw

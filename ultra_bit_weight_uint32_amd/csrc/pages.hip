// Pages of the key/value cache: copying them, drawing kept tokens together, and the pool that shares
// them out over sequences (who holds a page, what is free).
//
// The data calls move bytes and are bound by HBM (each byte read and written once) or, for a few
// pages, by one launch. Both address 16-byte vectors: a row of a head is 4 to 32 of them, page sizes
// are powers of two, so a vector's place in a page comes from shifts, and contiguous pages and pages
// inside a larger row (token-major caches) run through the same code.
//
// The pool calls work on small integer tables and are bound by launch and memory latency. Their
// results do not depend on timing: counts change by integer atomics (in any order the same), free
// pages are a bit set, and pages are handed out by rank (prefix sums), never by arrival.
#include "cache_internal.h"

namespace ubw {
namespace cache {
namespace {

constexpr uint32_t kNoPages = 1u, kNotServed = 2u;  // ubw_page_pool.status

// ---- copying pages: a workgroup takes kCopyVecs * 4 KiB of one page's keys (blockIdx.y = 0) or values.
// Both sides pass the caches by: 200 pages of 80 layers 418 us, 442 through them (5.0 and 4.7 TB/s).
typedef uint32_t Vec16 __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(256) void k_copy_pages(Pages c, int layers, int lrow, const int32_t* pairs, int vecs,
                                                    int pieces) {
    const uint32_t id = blockIdx.x;
    const uint32_t piece = id % pieces, rest = id / pieces;
    const uint32_t layer = rest % layers, i = rest / layers;
    const int src = pairs[2 * i], dst = pairs[2 * i + 1];
    if ((uint32_t)src >= (uint32_t)c.pages || (uint32_t)dst >= (uint32_t)c.pages || src == dst) return;
    const bool v = blockIdx.y != 0;
    const int64_t page = v ? c.v_page : c.k_page, head = v ? c.v_head : c.k_head;
    const uint32_t row = v ? c.v_row : c.k_row;
    char* base = (v ? c.v : c.k) + layer * (v ? c.v_layer : c.k_layer);
    const char* from = base + src * page;
    char* to = base + dst * page;
    Vec16 x[kCopyVecs];
    int64_t off[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
        const int n = (piece * kCopyVecs + j) * 256 + threadIdx.x;  // vector of the page
        const int r = n >> lrow;
        off[j] = n < vecs ? (r >> c.lps) * head + (int64_t)(r & ((1 << c.lps) - 1)) * row + (n & ((1 << lrow) - 1)) * 16 : -1;
        if (off[j] >= 0) x[j] = __builtin_nontemporal_load(reinterpret_cast<const Vec16*>(from + off[j]));
    }
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
        if (off[j] >= 0) __builtin_nontemporal_store(x[j], reinterpret_cast<Vec16*>(to + off[j]));
}

// ---- drawing kept tokens together: a workgroup takes 256 16-byte columns of a sequence's rows (a
// column: one 16 bytes of one head's rows in one layer, keys or values). Where each kept row comes from
// and goes to is looked up once, by 256 threads in parallel, into LDS (looked up by every thread in turn
// the same moves, 31 MB in 80 layers, took 19 us instead of 14.6 while they still went through the
// caches). Then a thread moves its column row by row, kMove at a time: a kept token's index is at least its
// place, so the rows read lie at or behind the rows written and nothing is overwritten unread; threads do
// not share columns. Both sides pass the caches by
// (15.0 -> 11.5 us: nothing is left in them for the kernel's end to write back).
constexpr int kMove = 16;

__global__ __launch_bounds__(256) void k_compact(Pages c, int layers, int lrow, const int32_t* table, int64_t ld_table,
                                                 int table_cols, const int32_t* ctx_len, const int32_t* keep, int width) {
    __shared__ int from_page[1024], to_page[1024];
    __shared__ int16_t from_row[1024], to_row[1024];
    __shared__ int ends;  // entries of the list
    const int b = blockIdx.y;
    const int ctx = ctx_len[b];
    if (ctx < 0) return;
    table += b * ld_table;
    keep += (int64_t)b * width;
    if (threadIdx.x == 0) ends = width;
    __syncthreads();
    const auto page_at = [&](int64_t p) -> int {  // of a position, or -1
        const int64_t col = p >> c.lps;
        if (col >= table_cols) return -1;
        const int pg = table[col];
        return (uint32_t)pg < (uint32_t)c.pages ? pg : -1;
    };
    const int mask = (1 << c.lps) - 1;
    for (int i = threadIdx.x; i < width; i += 256) {
        const int k = keep[i], before = i ? keep[i - 1] : -1;
        if (k < 0 || k <= before) {  // the list ends at the first of these
            atomicMin(&ends, i);
            from_page[i] = -1;
            continue;
        }
        const int64_t s = (int64_t)ctx + k, d = (int64_t)ctx + i;
        const int pt = page_at(d);
        from_page[i] = k == i || pt < 0 ? -1 : page_at(s);  // -1: nothing to move
        to_page[i] = pt;
        from_row[i] = (int16_t)(s & mask);
        to_row[i] = (int16_t)(d & mask);
    }
    __syncthreads();
    const int n_rows = ends;
    const uint32_t n = blockIdx.x * 256 + threadIdx.x;
    const uint32_t r = n >> lrow;
    const int h2 = (int)(r % (uint32_t)(2 * c.heads)), layer = (int)(r / (uint32_t)(2 * c.heads));
    if (layer >= layers) return;
    const bool v = h2 >= c.heads;
    const int64_t page = v ? c.v_page : c.k_page;
    const uint32_t row = v ? c.v_row : c.k_row;
    char* base = (v ? c.v : c.k) + layer * (v ? c.v_layer : c.k_layer) + (h2 - (v ? c.heads : 0)) * (v ? c.v_head : c.k_head) +
                 (n & ((1 << lrow) - 1)) * 16;
    for (int i0 = 0; i0 < n_rows; i0 += kMove) {
        Vec16 x[kMove];
#pragma unroll
        for (int j = 0; j < kMove; ++j)
            if (i0 + j < n_rows && from_page[i0 + j] >= 0)
                x[j] = __builtin_nontemporal_load(
                    reinterpret_cast<const Vec16*>(base + from_page[i0 + j] * page + (int64_t)from_row[i0 + j] * row));
#pragma unroll
        for (int j = 0; j < kMove; ++j)
            if (i0 + j < n_rows && from_page[i0 + j] >= 0)
                __builtin_nontemporal_store(
                    x[j], reinterpret_cast<Vec16*>(base + to_page[i0 + j] * page + (int64_t)to_row[i0 + j] * row));
    }
}

// ---- the pool
__device__ inline int pages_for(int len, int lps) { return (int)(((int64_t)len + (1 << lps) - 1) >> lps); }

__global__ __launch_bounds__(256) void k_pages_init(ubw_page_pool p) {
    const int64_t stride = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t i = first; i < (int64_t)p.seqs * p.max_pages; i += stride) p.table[i] = -1;
    for (int64_t i = first; i < p.pages; i += stride) p.ref[i] = 0;
    for (int64_t i = first; i < (p.pages + 31) / 32; i += stride) {
        const int64_t left = p.pages - i * 32;
        p.free_bits[i] = left >= 32 ? 0xffffffffu : (1u << left) - 1;
    }
    for (int64_t i = first; i < p.seqs; i += stride) p.held[i] = p.len[i] = 0;
    if (first == 0) *p.status = 0;
}

// One workgroup per sequence.
__global__ __launch_bounds__(256) void k_pages_trim(ubw_page_pool p, int lps, const int32_t* new_len) {
    const int s = blockIdx.x;
    const int n = new_len[s];
    if (n < 0) return;
    const int held = min(p.held[s], p.max_pages);
    const int cut = pages_for(n, lps);
    if (cut > held) {
        if (threadIdx.x == 0) atomicOr(p.status, kNotServed);
        return;
    }
    int32_t* row = p.table + (int64_t)s * p.max_pages;
    for (int j = cut + (int)threadIdx.x; j < held; j += 256) {
        const int pg = row[j];
        row[j] = -1;
        if ((uint32_t)pg < (uint32_t)p.pages && atomicSub(p.ref + pg, 1) == 1) atomicOr(p.free_bits + pg / 32, 1u << (pg & 31));
    }
    __syncthreads();  // every thread has read held
    if (threadIdx.x == 0) {
        p.held[s] = cut;
        p.len[s] = n;
    }
}

// One workgroup per sequence. A fork's parent is no fork of the same call, so no row that is read
// here is written here.
__global__ __launch_bounds__(256) void k_pages_fork(ubw_page_pool p, int lps, const int32_t* parents) {
    const int s = blockIdx.x;
    const int from = parents[s];
    if (from < 0) return;
    const bool known = from < p.seqs && from != s;
    const int n = known ? p.len[from] : 0;
    const int cut = pages_for(n, lps);
    if (!known || parents[from] >= 0 || p.held[s] != 0 || n < 0 || cut > min(p.held[from], p.max_pages)) {
        if (threadIdx.x == 0) atomicOr(p.status, kNotServed);
        return;
    }
    const int32_t* src = p.table + (int64_t)from * p.max_pages;
    int32_t* dst = p.table + (int64_t)s * p.max_pages;
    for (int j = threadIdx.x; j < cut; j += 256) {
        const int pg = src[j];
        dst[j] = pg;
        if ((uint32_t)pg < (uint32_t)p.pages) atomicAdd(p.ref + pg, 1);
    }
    __syncthreads();  // every thread has read held[s]
    if (threadIdx.x == 0) {
        p.held[s] = cut;
        p.len[s] = n;
    }
}

// The exclusive prefix sum over the workgroup's threads, in 64 bits (4096 sequences may ask for 2^24
// pages each); *total gets the sum. `lds` has 17 words.
__device__ inline int64_t wg_prefix(int64_t x, int64_t* lds, int64_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    int64_t y = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t z = __shfl_up((long long)y, d);
        if (lane >= d) y += z;
    }
    __syncthreads();  // lds may still be read from the call before
    if (lane == 63) lds[wave] = y;
    __syncthreads();
    if (threadIdx.x == 0) {
        int64_t sum = 0;
        for (int w = 0; w < waves; ++w) {
            const int64_t v = lds[w];
            lds[w] = sum;
            sum += v;
        }
        lds[16] = sum;
    }
    __syncthreads();
    *total = lds[16];
    return y - x + lds[wave];
}

// One workgroup: how many pages each sequence needs (a prefix sum over sequences), then the free pages
// in order of their number (a prefix sum over the words of the bit set), the r-th free page going to the
// sequence and place that r falls on. Free pages are listed in LDS by the threads that hold their words,
// kWindow at a time, and given out by all threads in parallel (each thread giving out those of its own
// words, up to 32 one after the other, took 34 us for 256 sequences instead of 16). The bit set is read
// beside the sequences' own loads, and all its changes are atomics, without a fence: 16 -> 9 us.
constexpr int kWindow = 4096;

__global__ __launch_bounds__(1024) void k_pages_reserve(ubw_page_pool p, int lps, const int32_t* room, int32_t* pairs) {
    __shared__ int before[UBW_MAX_SEQS + 1];  // pages needed by the sequences before s
    __shared__ int holds[UBW_MAX_SEQS];       // held[s], below 0 (-1 - held[s]) where the first page is a copy's
    __shared__ int list[kWindow];
    __shared__ int64_t lds[17];
    const int tid = threadIdx.x;
    constexpr int kPer = UBW_MAX_SEQS / 1024;
    int need[kPer], old[kPer], len_of[kPer], held_of[kPer];
    bool bad = false;
    int64_t total = 0;
    // free pages: this thread's words of the bit set (loads that do not wait for the sequences')
    const int words = (p.pages + 31) >> 5, per = (words + 1023) >> 10;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    const auto free_of = [&](int w) {  // bits past the last page are no pages, whatever they hold
        const int past = p.pages - w * 32;
        return p.free_bits[w] & (past >= 32 ? ~0u : (1u << past) - 1);
    };
    int have = 0;
    for (int w = w0; w < w1; ++w) have += __popc(free_of(w));
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int s = u * 1024 + tid;
        need[u] = 0;
        old[u] = -1;
        if (u * 1024 >= p.seqs) {  // alike in all threads
            before[s] = (int)total;
            continue;
        }
        if (s < p.seqs) {
            const int r = room[s], len = p.len[s], h = p.held[s];
            len_of[u] = len;
            held_of[u] = h;
            pairs[2 * s] = pairs[2 * s + 1] = -1;
            const int64_t want = ((int64_t)len + r + (1 << lps) - 1) >> lps;
            if (r > 0) {
                if (len < 0 || h < 0 || h > p.max_pages || want > p.max_pages || pages_for(len, lps) > h) {
                    bad = true;
                } else {
                    const int at = len >> lps;
                    need[u] = max(0, (int)want - h);
                    if (at < h) {
                        const int pg = p.table[(int64_t)s * p.max_pages + at];
                        if ((uint32_t)pg < (uint32_t)p.pages && p.ref[pg] > 1) {
                            old[u] = pg;
                            ++need[u];
                        }
                    }
                }
            }
            holds[s] = old[u] >= 0 ? -1 - h : h;
        }
        int64_t sum;
        before[s] = (int)(total + wg_prefix(need[u], lds, &sum));  // read only where all of it fits
        total += sum;
    }
    if (bad) atomicOr(p.status, kNotServed);
    if (tid == 0) before[UBW_MAX_SEQS] = (int)total;
    int64_t all;
    int rank = (int)wg_prefix(have, lds, &all);  // free pages before this thread's; its barriers also publish before[], holds[]
    if (total > all) {
        if (tid == 0) atomicOr(p.status, kNoPages);
        return;
    }
    int w = w0;
    uint32_t bits = w < w1 ? free_of(w) : 0u, left = bits;
    // Bits are taken and (for a page that two copies leave without a holder) set by atomics only, on bits
    // that no other thread changes, so their order is of no matter and no fence is needed.
    const auto took = [&] {
        if (left != bits) atomicAnd(p.free_bits + w, ~(bits ^ left));
    };
    for (int r0 = 0; r0 < total; r0 += kWindow) {
        const int r1 = (int)min((int64_t)r0 + kWindow, total);
        while (w < w1 && rank < r1) {  // this thread's pages of the window
            if (!left) {
                took();
                bits = left = ++w < w1 ? free_of(w) : 0u;
                continue;
            }
            list[rank - r0] = w * 32 + __ffs((int)left) - 1;
            left &= left - 1;
            ++rank;
        }
        __syncthreads();
        for (int r = r0 + tid; r < r1; r += 1024) {
            int lo = 0, hi = UBW_MAX_SEQS;  // the last s with before[s] <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (before[mid] <= r) lo = mid; else hi = mid;
            }
            const int pg = list[r - r0], h = holds[lo], j = r - before[lo];
            p.ref[pg] = 1;
            if (h < 0 && j == 0)
                pairs[2 * lo + 1] = pg;  // its place in the table is set below
            else
                p.table[(int64_t)lo * p.max_pages + (h < 0 ? -1 - h + j - 1 : h + j)] = pg;
        }
        __syncthreads();
    }
    if (w < w1) took();
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int s = u * 1024 + tid;
        if (need[u] == 0) continue;
        if (old[u] >= 0) {
            pairs[2 * s] = old[u];
            p.table[(int64_t)s * p.max_pages + (len_of[u] >> lps)] = pairs[2 * s + 1];
            if (atomicSub(p.ref + old[u], 1) == 1) atomicOr(p.free_bits + old[u] / 32, 1u << (old[u] & 31));
            p.held[s] = held_of[u] + need[u] - 1;
        } else {
            p.held[s] = held_of[u] + need[u];
        }
    }
}

}  // namespace

hipError_t launch_copy_pages(const Pages& c, int layers, int page_size, int row_bytes, const int32_t* pairs, int count,
                             hipStream_t s) {
    const int lrow = log2_of(row_bytes / 16);
    const int vecs = (c.heads * page_size) << lrow;
    const int pieces = (int)cdiv(vecs, 256 * kCopyVecs);
    const int64_t per_launch = kMaxGrid / ((int64_t)pieces * layers);  // at least 1 (checked by the caller)
    for (int64_t i = 0; i < count; i += per_launch) {
        const int64_t n = count - i < per_launch ? count - i : per_launch;
        k_copy_pages<<<dim3((unsigned)(n * layers * pieces), 2), 256, 0, s>>>(c, layers, lrow, pairs + 2 * i, vecs, pieces);
    }
    return hipGetLastError();
}

hipError_t launch_compact(const Pages& c, int layers, int row_bytes, const int32_t* table, int64_t ld_table,
                          int table_cols, const int32_t* ctx_len, const int32_t* keep, int width, int batch,
                          hipStream_t s) {
    const int lrow = log2_of(row_bytes / 16);
    const int64_t columns = ((int64_t)layers * 2 * c.heads) << lrow;
    k_compact<<<dim3((unsigned)cdiv(columns, 256), batch), 256, 0, s>>>(c, layers, lrow, table, ld_table, table_cols,
                                                                       ctx_len, keep, width);
    return hipGetLastError();
}

hipError_t launch_pages_init(const ubw_page_pool& p, hipStream_t s) {
    const int64_t n = (int64_t)p.seqs * p.max_pages > p.pages ? (int64_t)p.seqs * p.max_pages : p.pages;
    const int64_t wgs = cdiv(n, 1024) < 2048 ? cdiv(n, 1024) : 2048;
    k_pages_init<<<(unsigned)wgs, 256, 0, s>>>(p);
    return hipGetLastError();
}
hipError_t launch_pages_trim(const ubw_page_pool& p, const int32_t* new_len, hipStream_t s) {
    k_pages_trim<<<p.seqs, 256, 0, s>>>(p, log2_of(p.page_size), new_len);
    return hipGetLastError();
}
hipError_t launch_pages_fork(const ubw_page_pool& p, const int32_t* parents, hipStream_t s) {
    k_pages_fork<<<p.seqs, 256, 0, s>>>(p, log2_of(p.page_size), parents);
    return hipGetLastError();
}
hipError_t launch_pages_reserve(const ubw_page_pool& p, const int32_t* room, int32_t* pairs, hipStream_t s) {
    k_pages_reserve<<<1, 1024, 0, s>>>(p, log2_of(p.page_size), room, pairs);
    return hipGetLastError();
}

}  // namespace cache
}  // namespace ubw

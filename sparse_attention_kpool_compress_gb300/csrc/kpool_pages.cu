// Upkeep of a paged cache: copying pages, forking, extending and freeing
// sequences, writing rows, and compacting the pool.  include/kpool.h states
// each call's contract.
//
// A page holds page_size tokens; a sequence's tokens lie in the pages that its
// page-table row lists, and sequences forked from one parent list the same
// whole pages (ref_count says how many do).  Free page ids form a stack
// (free_list, free_count): allocation pops from its end, in the order of the
// call's list, so equal inputs give equal tables.
//
// fork, free, compact, and a copy of more than 1024 pages, are two kernels:
//   plan    one block: validates the whole list, takes pages from or accounts
//           for the pool, and writes what the second kernel has to do into the
//           workspace.  A list with a bad entry, or one the free pages do not
//           cover, changes nothing (its count of items becomes 0).
//   apply   all SMs: page-table rows, reference counts and page contents.
// extend is a plan alone; a smaller copy and a write check what they read in the
// blocks that move it.
// All are launched with programmatic stream serialisation: a kernel's blocks
// start while the one in front of it runs and wait for its end, which hides the
// launch.  No block waits for another one inside a kernel, but for the cluster
// barrier of a small write.
//
// Bound: contents by HBM (each byte read and written once, 16-byte accesses,
// four in flight per thread: copying 300 pages of four layers moves its 167 MB in
// 25 us alone, 6.7 TB/s, and in 30 in a graph of such calls); small calls by their
// launches and a handful of dependent loads (in a graph copy takes 2.5 us, fork 5.7,
// extend and write 7.0, free and compact 11.3).
#include <algorithm>
#include <climits>

#include "kpool_internal.h"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kChunk = 16 * 4 * kApplyThreads;   // bytes one block copies at a time
// Page-table entries that one block handles at a time.  A table is as wide as the
// longest sequence may become, and most rows end early: with 256 at a time, 4096 rows
// of 32768 entries that hold 8 pages each took compact 280 us and free 438; with 1024,
// 131 and 231.  8 rows that are full take the same either way (109 and 175).
constexpr int kSpan = 1024;
constexpr int kCluster = 8;                      // blocks of a call that is one cluster
constexpr int kWriteClusterThreads = 1024;
constexpr int kPlanPages = 8;                    // pages per thread and round of the compaction scan
constexpr uint32_t kFull = 0xFFFFFFFFu;

// workspace header (ints)
enum { W_TICKET = 0, W_STATUS = 1, W_COUNT = 2, W_LIVE = 3, W_HEADER = 64 };

struct Stores {
    kpool_page_store s[KPOOL_MAX_STORES];
    int n;
    int chunks[KPOOL_MAX_STORES];    // 16 KB pieces of a page
    int per_item;                    // pieces of a page over all stores and layers
};

// Where the plan leaves its lists (ints in the workspace behind the header).
struct Lists {
    int *a, *b, *c;      // per item
    int *mark;           // per sequence or per page
};

// Exclusive prefix sum of v over the block (kPlanThreads); *total gets the sum.
__device__ __forceinline__ int block_exclusive(int v, int *scratch, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                      // scratch of the previous call is read
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int t = lane < warps ? scratch[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFull, t, d);
            if (lane >= d) t += y;
        }
        scratch[lane] = t;
    }
    __syncthreads();
    *total = scratch[31];
    return x - v + (warp > 0 ? scratch[warp - 1] : 0);
}

__device__ __forceinline__ bool in_range(int i, int n) { return i >= 0 && i < n; }

// Block-wide: is any index of ids[0, n) out of [0, limit) or listed twice?
// mark[id] ends as the first place that lists id.
__device__ bool bad_or_twice(const int32_t *ids, int n, int limit, int *mark)
{
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        if (in_range(ids[i], limit)) mark[ids[i]] = INT_MAX;
        else bad = true;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (in_range(ids[i], limit)) atomicMin(mark + ids[i], i);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (in_range(ids[i], limit) && mark[ids[i]] != i) bad = true;
    return __syncthreads_or(bad) != 0;
}

// The same for a list of at most blockDim.x ids, in a table of 4 * blockDim.x words
// of shared memory: cleared before the block waits for the kernel in front, and
// filled while the loads that an id leads to are on their way.  Marks in global
// memory are three trips there: with them and with the free pages looked up behind
// the lengths, a fork of four took 0.5 us more, a free of three 0.7 and an extend by
// 1025 tokens of eight sequences 1.0.
__device__ __forceinline__ void clear_ids(int *table)
{
    for (int i = threadIdx.x; i < 4 * blockDim.x; i += blockDim.x) table[i] = -1;
}

__device__ __forceinline__ int id_place(int id, int mask)
{
    return static_cast<int>(static_cast<uint32_t>(id) * 2654435761u >> 8) & mask;
}

// Adds id (>= 0) to the table; true if it was there.  (A quarter of the table is
// filled at most: each search ends.)
__device__ __forceinline__ bool add_id(int *table, int mask, int id)
{
    for (int h = id_place(id, mask);; h = (h + 1) & mask) {
        const int old = atomicCAS(&table[h], -1, id);
        if (old == id) return true;
        if (old == -1) return false;
    }
}

// The page at place `rank` from the top of the free list, -1 if it is not a free one.
__device__ __forceinline__ int free_page(const kpool_page_pool &p, int fc, int rank)
{
    if (rank >= fc) return -1;
    const int page = p.free_list[fc - 1 - rank];
    return in_range(page, p.n_pages) && p.ref_count[page] == 0 ? page : -1;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// One 16 KB piece of one page: the block's threads copy `bytes` (a multiple of
// 16) from src to dst, all loads of a thread issued before its stores.
__device__ __forceinline__ void copy_piece(const char *src, char *dst, int bytes)
{
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int off = (k * kApplyThreads + threadIdx.x) * 16;
        if (off < bytes) v[k] = *reinterpret_cast<const uint4 *>(src + off);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int off = (k * kApplyThreads + threadIdx.x) * 16;
        if (off < bytes) *reinterpret_cast<uint4 *>(dst + off) = v[k];
    }
}

// Contents of `count` page pairs, page src[i] to page dst[i] in every store and
// layer: whole pages, or, given the sequences' lengths, the rows that a last
// page of that length uses.
__device__ void copy_pages(const Stores &st, const int *src, const int *dst, const int *lens,
                           int count, int page_size, int n_pages)
{
    const int64_t tasks = static_cast<int64_t>(count) * st.per_item;
    for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int item = static_cast<int>(t / st.per_item);
        int r = static_cast<int>(t - static_cast<int64_t>(item) * st.per_item);
        int s = 0;
        while (r >= st.s[s].n_layers * st.chunks[s]) r -= st.s[s].n_layers * st.chunks[s], ++s;
        const kpool_page_store &g = st.s[s];
        const int layer = r / st.chunks[s], piece = r - layer * st.chunks[s];
        const int a = src[item], b = dst[item];
        if (!in_range(a, n_pages) || !in_range(b, n_pages)) continue;
        const int tok = lens != nullptr ? lens[item] % page_size : page_size;
        // the store's rows that hold those tokens, the last one whole
        const int rows = static_cast<int>((static_cast<int64_t>(tok) * g.rows_per_page + page_size - 1) / page_size);
        const int64_t bytes = static_cast<int64_t>(rows) * g.row_bytes - static_cast<int64_t>(piece) * kChunk;
        if (bytes <= 0) continue;
        const int64_t base = layer * g.layer_stride + static_cast<int64_t>(piece) * kChunk;
        const char *p = static_cast<const char *>(g.data) + base;
        char *q = static_cast<char *>(g.data) + base;
        copy_piece(p + a * g.page_stride, q + b * g.page_stride, static_cast<int>(min(bytes, static_cast<int64_t>(kChunk))));
    }
}

// ---- copy --------------------------------------------------------------------

// Up to kPagesFusedCopy pairs: one kernel, whose blocks all check the whole list
// with a hash table in shared memory (about a microsecond each, side by side) and
// so agree without a plan in front.  Against plan and apply, with a host that
// allocates no marks: 5 pages 27 -> 17 us a call (3.5 -> 2.4 in a graph), 300 pages
// of four layers 35 -> 34 (31 -> 30 in a graph).
__global__ void __launch_bounds__(kApplyThreads) copy_fused(const __grid_constant__ Stores st, const int32_t *src,
                                                            const int32_t *dst, int n, int n_pages, int *ws)
{
    constexpr int kTable = 4 * kPagesFusedCopy;
    static_assert((kTable & (kTable - 1)) == 0, "a power of two");
    __shared__ int table[kTable];
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    for (int i = threadIdx.x; i < kTable; i += kApplyThreads) table[i] = -1;
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += kApplyThreads) {
        const int page = dst[i];
        if (!in_range(page, n_pages) || add_id(table, kTable - 1, page)) bad = true;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kApplyThreads) {
        const int page = src[i];
        if (!in_range(page, n_pages)) bad = true;
        for (int h = id_place(page, kTable - 1); table[h] != -1; h = (h + 1) & (kTable - 1))
            if (table[h] == page) {
                bad = true;
                break;
            }
    }
    bad = __syncthreads_or(bad) != 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) ws[W_STATUS] = bad ? KPOOL_STATUS_BAD_PAGE : 0;
    if (!bad) copy_pages(st, src, dst, nullptr, n, 1, n_pages);
}

__global__ void __launch_bounds__(kPlanThreads) copy_plan(const int32_t *src, const int32_t *dst, int n,
                                                          int n_pages, int *ws, Lists l)
{
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    bool bad = false;
    // a source may be listed several times, a destination once, a page not as both
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (in_range(src[i], n_pages)) l.mark[src[i]] = -1;
    __syncthreads();
    bad = bad_or_twice(dst, n, n_pages, l.mark);
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        bad |= !in_range(src[i], n_pages) || l.mark[src[i]] != -1;
    bad = __syncthreads_or(bad) != 0;
    if (threadIdx.x == 0) {
        ws[W_STATUS] = bad ? KPOOL_STATUS_BAD_PAGE : 0;
        ws[W_COUNT] = bad ? 0 : n;
    }
}

__global__ void __launch_bounds__(kApplyThreads) copy_apply(const __grid_constant__ Stores st, const int32_t *src,
                                                            const int32_t *dst, int n_pages, const int *ws)
{
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    copy_pages(st, src, dst, nullptr, ws[W_COUNT], 1, n_pages);
}

// ---- fork --------------------------------------------------------------------
// lists: a = source page of the partial page (or -1), b = its copy, c = length

__global__ void __launch_bounds__(kPlanThreads) fork_plan(const kpool_page_pool p, const int32_t *parents,
                                                          const int32_t *children, int n, int *ws, Lists l)
{
    __shared__ int scratch[32], table[4 * kPlanThreads], top[kPlanThreads];
    ptx::grid_dependents_launch();
    clear_ids(table);
    ptx::grid_dependency_wait();
    const int ps = p.page_size;
    const int64_t room = static_cast<int64_t>(p.max_pages) * ps;
    const bool few = n <= blockDim.x;
    bool bad = few ? false : bad_or_twice(children, n, p.n_seqs, l.mark);
    __syncthreads();                       // the table is clear
    int fc = *p.free_count;
    if (!in_range(fc, p.n_pages + 1)) bad = true, fc = 0;
    top[threadIdx.x] = free_page(p, fc, threadIdx.x);
    int need = 0;                          // pages taken by the items before this round
    bool short_of = false;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + threadIdx.x;
        int len = 0, last = -1, part = 0;
        if (i < n) {
            const int pa = parents[i], ch = children[i];
            if (!in_range(pa, p.n_seqs) || !in_range(ch, p.n_seqs) || pa == ch) bad = true;
            else {
                len = p.seq_lens[pa];
                if (p.seq_lens[ch] != 0) bad = true;
                if (few && add_id(table, 4 * blockDim.x - 1, ch)) bad = true;
                if (len < 0 || len > room) bad = true, len = 0;
                part = len % ps;
                if (part > 0) {
                    last = p.page_table[static_cast<int64_t>(pa) * p.max_pages + len / ps];
                    if (!in_range(last, p.n_pages)) bad = true;
                }
            }
        }
        int total;
        const int rank = need + block_exclusive(part > 0, scratch, &total);
        need += total;
        if (i < n) {
            int page = -1;
            if (part > 0) {
                if (rank >= fc) short_of = true;
                else {
                    page = rank < blockDim.x ? top[rank] : free_page(p, fc, rank);
                    if (page < 0) bad = true;
                }
            }
            l.a[i] = last;
            l.b[i] = page;
            l.c[i] = len;
        }
    }
    bad = __syncthreads_or(bad) != 0;
    short_of = __syncthreads_or(short_of) != 0;
    const bool ok = !bad && !short_of;
    if (ok)
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            p.seq_lens[children[i]] = l.c[i];
            if (l.b[i] >= 0) p.ref_count[l.b[i]] = 1;
        }
    if (threadIdx.x == 0) {
        if (ok) *p.free_count = fc - need;
        ws[W_STATUS] = (bad ? KPOOL_STATUS_BAD_PAGE : 0) | (short_of && !bad ? KPOOL_STATUS_NO_PAGES : 0);
        ws[W_COUNT] = ok ? n : 0;
    }
}

__global__ void __launch_bounds__(kApplyThreads) fork_apply(const __grid_constant__ Stores st, const kpool_page_pool p,
                                                            const int32_t *parents, const int32_t *children,
                                                            int *ws, Lists l)
{
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int n = ws[W_COUNT];
    const int spans = ceil_div(p.max_pages, kSpan);
    // the children's page-table rows, and one more reference on each whole page
    for (int64_t t = blockIdx.x; t < static_cast<int64_t>(n) * spans; t += gridDim.x) {
        const int i = static_cast<int>(t / spans), first = static_cast<int>(t - static_cast<int64_t>(i) * spans) * kSpan;
        const int whole = l.c[i] / p.page_size;
        int32_t *row = p.page_table + static_cast<int64_t>(children[i]) * p.max_pages;
        const int32_t *from = p.page_table + static_cast<int64_t>(parents[i]) * p.max_pages;
        if (first <= whole && whole < first + kSpan && threadIdx.x == 0 && l.b[i] >= 0) row[whole] = l.b[i];
        for (int j = first + threadIdx.x; j < min(whole, first + kSpan); j += kApplyThreads) {
            const int page = from[j];
            row[j] = page;
            if (in_range(page, p.n_pages)) atomicAdd(p.ref_count + page, 1);
            else atomicOr(ws + W_STATUS, KPOOL_STATUS_BAD_PAGE);
        }
    }
    // the used rows of each partial page
    copy_pages(st, l.a, l.b, l.c, n, p.page_size, p.n_pages);
}

// ---- extend ------------------------------------------------------------------
// lists: a = pages taken before item i's, b = length afterwards, c = pages to take (n_new
// is not read again once lengths change: it may be seq_lens itself)

__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const kpool_page_pool p, const int32_t *seqs,
                                                              const int32_t *n_new, int n, int32_t *begin,
                                                              int *ws, Lists l)
{
    __shared__ int scratch[32], table[4 * kPlanThreads], top[kPlanThreads];
    ptx::grid_dependents_launch();
    clear_ids(table);
    ptx::grid_dependency_wait();
    const int ps = p.page_size;
    const int64_t room = static_cast<int64_t>(p.max_pages) * ps;
    const bool few = n <= blockDim.x;
    bool bad = few ? false : bad_or_twice(seqs, n, p.n_seqs, l.mark);
    __syncthreads();                       // the table is clear
    int fc = *p.free_count;
    if (!in_range(fc, p.n_pages + 1)) bad = true, fc = 0;
    top[threadIdx.x] = free_page(p, fc, threadIdx.x);
    int64_t need = 0;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + threadIdx.x;
        int had = 0, take = 0, len = -1, to = 0;
        const int s = i < n ? seqs[i] : 0;
        if (!in_range(s, p.n_seqs)) bad = true;
        else if (i < n) {
            const int add = n_new[i];
            len = p.seq_lens[s];
            if (few && add_id(table, 4 * blockDim.x - 1, s)) bad = true;
            if (len < 0 || add < 0 || static_cast<int64_t>(len) + add > room) bad = true;
            else {
                had = ceil_div(len, ps);
                to = len + add;
                take = ceil_div(to, ps) - had;
                if (add > 0 && len % ps != 0) {
                    // the rows go on in the last page, which must be the sequence's own
                    const int last = p.page_table[static_cast<int64_t>(s) * p.max_pages + had - 1];
                    if (!in_range(last, p.n_pages) || p.ref_count[last] != 1) bad = true;
                }
            }
        }
        int total;
        const int rank = block_exclusive(take, scratch, &total);
        if (i < n) {
            l.a[i] = static_cast<int>(min(need + rank, static_cast<int64_t>(INT_MAX)));
            l.b[i] = to;
            l.c[i] = take;
            begin[i] = len;
        }
        need += total;
    }
    const bool short_of = need > fc;
    bad = __syncthreads_or(bad) != 0;
    bool ok = !bad && !short_of;
    // the pages that will be popped must be free ones
    if (ok)
        for (int i = threadIdx.x; i < need; i += blockDim.x)
            if ((i < blockDim.x ? top[i] : free_page(p, fc, i)) < 0) bad = true;
    bad = __syncthreads_or(bad) != 0;
    ok = ok && !bad;
    if (ok) {
        const int lane = threadIdx.x & 31;
        for (int i = threadIdx.x >> 5; i < n; i += blockDim.x >> 5) {
            const int s = seqs[i], take = l.c[i];
            int32_t *row = p.page_table + static_cast<int64_t>(s) * p.max_pages + ceil_div(begin[i], ps);
            for (int j = lane; j < take; j += 32) {
                const int k = l.a[i] + j;
                const int page = k < blockDim.x ? top[k] : p.free_list[fc - 1 - k];
                row[j] = page;
                p.ref_count[page] = 1;
            }
            if (lane == 0) p.seq_lens[s] = l.b[i];
        }
    } else {
        for (int i = threadIdx.x; i < n; i += blockDim.x) begin[i] = -1;
    }
    if (threadIdx.x == 0) {
        if (ok) *p.free_count = fc - static_cast<int>(need);
        ws[W_STATUS] = (bad ? KPOOL_STATUS_BAD_PAGE : 0) | (short_of && !bad ? KPOOL_STATUS_NO_PAGES : 0);
    }
}

// ---- write -------------------------------------------------------------------

// The last i with cu[i] <= r (n + 1 offsets), one warp probing 32 of them per round.
__device__ __forceinline__ int segment_of(const int32_t *cu, int n, int r, int lane)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const unsigned m = __ballot_sync(kFull, at < hi && cu[at] <= r);
        if (m == 0) return lo;             // offsets that do not begin at or before r
        const int nlo = lo + (31 - __clz(m)) * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo;
}

// The status word has to be 0 before a block adds to it.  Up to 256 rows (over the
// layers) take one cluster of eight blocks, one row per warp: its first block clears
// the word, and its barrier orders that before the end of the others.  More take a
// kernel in front that does.  256 rows of 1152 bytes take 3.8 us so in a graph and 7.6
// in a call, against 3.5 and 9.9; 512 would take 5.6 and 7.7.  (A memset in front took
// 6.4 and 8.9.)
__global__ void clear_status(int *ws)
{
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    ws[W_STATUS] = 0;
}

template <bool kOne>
__global__ void __launch_bounds__(kOne ? kWriteClusterThreads : kApplyThreads) write_kernel(const kpool_page_pool p, const int32_t *seqs,
                                                              const int32_t *begin, const int32_t *cu_rows, int n,
                                                              int64_t total, const char *rows,
                                                              int64_t rows_layer_stride, const kpool_page_store g,
                                                              int *ws)
{
    // One warp per row and layer (one per row for all layers measured slower: 11.8
    // against 9.4 us for 8200 rows in two layers).
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    bool bad = false;
    const int named = blockIdx.x == 0 && threadIdx.x == 0 ? cu_rows[n] : 0;
    if (kOne) {
        if (blockIdx.x == 0 && threadIdx.x == 0) ws[W_STATUS] = 0;
        ptx::cluster_arrive();
    }
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         t < total * g.n_layers; t += warps) {
        const int layer = static_cast<int>(t / total);
        const int r = static_cast<int>(t - layer * total);
        const char *src = rows + layer * rows_layer_stride + static_cast<int64_t>(r) * g.row_bytes;
        // the row's first 2 KB, on their way while its place is looked up
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (lane * 16 + 512 * q < g.row_bytes) v[q] = __ldcs(reinterpret_cast<const uint4 *>(src + lane * 16 + 512 * q));
        const int i = segment_of(cu_rows, n, r, lane);
        const int k = r - cu_rows[i], seq = seqs[i], from = begin[i];
        bool ok = k >= 0 && r < cu_rows[i + 1] && in_range(seq, p.n_seqs) && from >= 0;
        int page = -1, row = 0;
        if (ok) {
            // rows behind the sequence's length (rows_per_page of every page_size tokens) are not its own
            const int64_t at = static_cast<int64_t>(from) + k;
            const int64_t held = static_cast<int64_t>(p.seq_lens[seq]) * g.rows_per_page;
            const int64_t col = at / g.rows_per_page;
            row = static_cast<int>(at - col * g.rows_per_page);
            ok = at * p.page_size < held && col < p.max_pages;
            if (ok) page = p.page_table[static_cast<int64_t>(seq) * p.max_pages + col];
            ok = ok && in_range(page, p.n_pages) && p.ref_count[page] == 1;
        }
        if (!ok) {
            bad = true;
            continue;
        }
        char *dst = static_cast<char *>(g.data) + layer * g.layer_stride + page * g.page_stride +
                    static_cast<int64_t>(row) * g.row_bytes;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (lane * 16 + 512 * q < g.row_bytes) *reinterpret_cast<uint4 *>(dst + lane * 16 + 512 * q) = v[q];
        for (int off = 2048 + lane * 16; off < g.row_bytes; off += 512)
            *reinterpret_cast<uint4 *>(dst + off) = __ldcs(reinterpret_cast<const uint4 *>(src + off));
    }
    bad |= named > total;                  // rows that the list names and nobody brought
    if (kOne) ptx::cluster_wait();
    if (bad && lane == 0) atomicOr(ws + W_STATUS, KPOOL_STATUS_BAD_PAGE);
}

// ---- free --------------------------------------------------------------------
// lists: c = length of each listed sequence; mark = bit per page that lost its
// last reference (after the per-sequence marks of the plan)

__global__ void __launch_bounds__(kPlanThreads) free_plan(const kpool_page_pool p, const int32_t *seqs, int n,
                                                          int *ws, Lists l, int *bits)
{
    __shared__ int table[4 * kPlanThreads];
    ptx::grid_dependents_launch();
    clear_ids(table);
    ptx::grid_dependency_wait();
    const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
    const bool few = n <= blockDim.x;
    bool bad = few ? false : bad_or_twice(seqs, n, p.n_seqs, l.mark);
    __syncthreads();                       // the table is clear
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = seqs[i];
        if (!in_range(s, p.n_seqs)) bad = true;
        else {
            const int len = p.seq_lens[s];
            if (few && add_id(table, 4 * blockDim.x - 1, s)) bad = true;
            if (len < 0 || len > room) bad = true;
            l.c[i] = len;
        }
    }
    if (!in_range(*p.free_count, p.n_pages + 1)) bad = true;
    for (int w = threadIdx.x; w < ceil_div(p.n_pages, 32); w += blockDim.x) bits[w] = 0;
    bad = __syncthreads_or(bad) != 0;
    if (!bad)
        for (int i = threadIdx.x; i < n; i += blockDim.x) p.seq_lens[seqs[i]] = 0;
    if (threadIdx.x == 0) {
        ws[W_TICKET] = 0;
        ws[W_STATUS] = bad ? KPOOL_STATUS_BAD_PAGE : 0;
        ws[W_COUNT] = bad ? 0 : n;
    }
}

__global__ void __launch_bounds__(kApplyThreads) free_apply(const kpool_page_pool p, const int32_t *seqs, int *ws,
                                                            Lists l, int *bits)
{
    __shared__ int scratch[32];
    __shared__ int ticket;
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int n = ws[W_COUNT];
    if (n == 0) return;                    // refused: the count stays too, whatever it is
    const int spans = ceil_div(p.max_pages, kSpan);
    for (int64_t t = blockIdx.x; t < static_cast<int64_t>(n) * spans; t += gridDim.x) {
        const int i = static_cast<int>(t / spans), first = static_cast<int>(t - static_cast<int64_t>(i) * spans) * kSpan;
        const int held = ceil_div(l.c[i], p.page_size);
        int32_t *row = p.page_table + static_cast<int64_t>(seqs[i]) * p.max_pages;
        for (int j = first + threadIdx.x; j < min(held, first + kSpan); j += kApplyThreads) {
            const int page = row[j];
            row[j] = -1;
            int had = 0;
            if (in_range(page, p.n_pages)) {
                had = atomicSub(p.ref_count + page, 1);
                if (had == 1) atomicOr(bits + (page >> 5), 1 << (page & 31));
                if (had <= 0) atomicAdd(p.ref_count + page, 1);  // it had no reference to give back
            }
            if (had <= 0) atomicOr(ws + W_STATUS, KPOOL_STATUS_BAD_PAGE);
        }
    }
    // the block that comes last pushes the freed pages, in ascending order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) ticket = atomicAdd(ws + W_TICKET, 1);
    __syncthreads();
    if (ticket != static_cast<int>(gridDim.x) - 1) return;
    __threadfence();
    const int words = ceil_div(p.n_pages, 32);
    int top = *p.free_count;
    for (int base = 0; base < words; base += kApplyThreads) {
        const int w = base + threadIdx.x;
        uint32_t m = w < words ? static_cast<uint32_t>(__ldcg(bits + w)) : 0u;
        int total;
        int at = top + block_exclusive(__popc(m), scratch, &total);
        for (; m != 0u; m &= m - 1u, ++at)
            if (at < p.n_pages) p.free_list[at] = 32 * w + __ffs(m) - 1;
        top += total;
    }
    if (threadIdx.x == 0) {
        if (top > p.n_pages) atomicOr(ws + W_STATUS, KPOOL_STATUS_BAD_PAGE);
        *p.free_count = min(top, p.n_pages);
    }
}

// ---- compact -----------------------------------------------------------------
// With k pages referenced, the i-th referenced page at or above k moves to the
// i-th unreferenced page below k.  lists: a = sources, b = destinations,
// mark = where each page at or above k goes (-1: nowhere)

__global__ void __launch_bounds__(kPlanThreads) compact_plan(const kpool_page_pool p, int *ws, Lists l)
{
    __shared__ int scratch[32];
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int n = p.n_pages;
    // (the count and the first lengths are held back, so that all loads are in flight at once)
    const int fc = *p.free_count, len0 = threadIdx.x < p.n_seqs ? p.seq_lens[threadIdx.x] : 0;
    int mine = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) mine += p.ref_count[i] > 0;
    int k;
    block_exclusive(mine, scratch, &k);
    const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
    bool bad = !in_range(fc, n + 1) || len0 < 0 || len0 > room;
    for (int s = threadIdx.x + blockDim.x; s < p.n_seqs; s += blockDim.x) {
        const int len = p.seq_lens[s];
        bad |= len < 0 || len > room;
    }
    int from = 0, to = 0;                  // movers and holes before this round
    for (int base = 0; base < n; base += kPlanPages * blockDim.x) {
        const int p0 = base + kPlanPages * threadIdx.x;
        // bit q: page p0 + q moves, or is a hole; a round's eight pages lie on
        // both sides of k at most once, so both kinds are counted apart
        uint32_t mv = 0, ho = 0;
#pragma unroll
        for (int q = 0; q < kPlanPages; ++q) {
            const int page = p0 + q;
            if (page >= n) break;
            const bool live = p.ref_count[page] > 0;
            if (page >= k) l.mark[page] = -1;
            if (live && page >= k) mv |= 1u << q;
            if (!live && page < k) ho |= 1u << q;
        }
        int tm, th;
        int am = from + block_exclusive(__popc(mv), scratch, &tm);
        int ah = to + block_exclusive(__popc(ho), scratch, &th);
        for (; mv != 0u; mv &= mv - 1u) l.a[am++] = p0 + __ffs(mv) - 1;
        for (; ho != 0u; ho &= ho - 1u) l.b[ah++] = p0 + __ffs(ho) - 1;
        from += tm;
        to += th;
    }
    if (__syncthreads_or(bad)) {           // (so far only the workspace was written)
        if (threadIdx.x == 0) {
            ws[W_STATUS] = KPOOL_STATUS_BAD_PAGE;
            ws[W_COUNT] = 0;
            ws[W_LIVE] = n;                // every page stays where it is
        }
        return;
    }
    // as many pages move as there are holes: both are k less the referenced pages below k
    for (int i = threadIdx.x; i < from; i += blockDim.x) {
        const int s = l.a[i], d = l.b[i];
        l.mark[s] = d;
        p.ref_count[d] = p.ref_count[s];
        p.ref_count[s] = 0;
    }
    for (int i = threadIdx.x; i < n - k; i += blockDim.x) p.free_list[i] = n - 1 - i;
    if (threadIdx.x == 0) {
        *p.free_count = n - k;
        ws[W_STATUS] = 0;
        ws[W_COUNT] = from;
        ws[W_LIVE] = k;
    }
}

__global__ void __launch_bounds__(kApplyThreads) compact_apply(const __grid_constant__ Stores st,
                                                               const kpool_page_pool p, int *ws, Lists l)
{
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int k = ws[W_LIVE];
    const int spans = ceil_div(p.max_pages, kSpan);
    for (int64_t t = blockIdx.x; t < static_cast<int64_t>(p.n_seqs) * spans; t += gridDim.x) {
        const int s = static_cast<int>(t / spans), first = static_cast<int>(t - static_cast<int64_t>(s) * spans) * kSpan;
        const int64_t len = p.seq_lens[s];
        const int held = static_cast<int>(min((len + p.page_size - 1) / p.page_size, static_cast<int64_t>(p.max_pages)));
        int32_t *row = p.page_table + static_cast<int64_t>(s) * p.max_pages;
        for (int j = first + threadIdx.x; j < min(held, first + kSpan); j += kApplyThreads) {
            const int page = row[j];
            const int now = !in_range(page, p.n_pages) ? -1 : page < k ? page : l.mark[page];
            if (now < 0) atomicOr(ws + W_STATUS, KPOOL_STATUS_BAD_PAGE);
            else if (now != page) row[j] = now;
        }
    }
    copy_pages(st, l.a, l.b, nullptr, ws[W_COUNT], 1, p.n_pages);
}

// ---- host --------------------------------------------------------------------

Lists lists(void *ws, int64_t n)
{
    int *base = static_cast<int *>(ws) + W_HEADER;
    return Lists{base, base + n, base + 2 * n, base + 3 * n};
}

Stores pack(const kpool_page_store *stores, int n_stores)
{
    Stores st{};
    st.n = n_stores;
    for (int i = 0; i < n_stores; ++i) {
        st.s[i] = stores[i];
        st.chunks[i] = static_cast<int>((static_cast<int64_t>(stores[i].rows_per_page) * stores[i].row_bytes + kChunk - 1) / kChunk);
        st.per_item += st.chunks[i] * stores[i].n_layers;
    }
    return st;
}

// Blocks for `tasks` block-sized pieces of work: at most eight per SM, which
// keep the copies' loads in flight (2048 threads).
int grid_for(int64_t tasks)
{
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tasks, 8LL * num_sms())));
}

// A plan's block: short lists take a small one, whose barriers and scans are shorter.
int plan_threads(int n) { return n <= 256 ? 256 : kPlanThreads; }

template <typename... P, typename... A>
cudaError_t launch_clusters_after(int cluster, void (*kernel)(P...), int grid, int threads, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int threads, cudaStream_t s, A... args)
{
    return launch_clusters_after(1, kernel, grid, threads, s, args...);
}

}  // namespace

size_t pages_workspace_bytes(int64_t n, int n_seqs, int n_pages)
{
    // three lists of the call's items (or of the pages, when compacting), the
    // marks, and a bit per page
    const int64_t items = std::max<int64_t>(n, n_pages);
    return static_cast<size_t>(4 * (W_HEADER + 3 * items + std::max(n_seqs, n_pages) + (n_pages + 31) / 32 + 64));
}

int run_pages_copy(const int32_t *src, const int32_t *dst, int n, int n_pages, const kpool_page_store *stores,
                   int n_stores, void *ws, cudaStream_t s)
{
    const Stores st = pack(stores, n_stores);
    int *w = static_cast<int *>(ws);
    if (n <= kPagesFusedCopy) {
        KPOOL_CUDA_CHECK(launch_after(copy_fused, grid_for(static_cast<int64_t>(n) * st.per_item), kApplyThreads, s, st, src,
                                      dst, n, n_pages, w));
        return KPOOL_OK;
    }
    KPOOL_CUDA_CHECK(launch_after(copy_plan, 1, plan_threads(n), s, src, dst, n, n_pages, w, lists(ws, n)));
    KPOOL_CUDA_CHECK(launch_after(copy_apply, grid_for(static_cast<int64_t>(n) * st.per_item), kApplyThreads, s, st, src, dst,
                                       n_pages, static_cast<const int *>(w)));
    return KPOOL_OK;
}

int run_pages_fork(const kpool_page_pool &p, const int32_t *parents, const int32_t *children, int n,
                   const kpool_page_store *stores, int n_stores, void *ws, cudaStream_t s)
{
    const Stores st = pack(stores, n_stores);
    const Lists l = lists(ws, n);
    int *w = static_cast<int *>(ws);
    KPOOL_CUDA_CHECK(launch_after(fork_plan, 1, plan_threads(n), s, p, parents, children, n, w, l));
    const int64_t spans = (p.max_pages + kSpan - 1) / kSpan;
    KPOOL_CUDA_CHECK(launch_after(fork_apply, grid_for(n * std::max<int64_t>(spans, st.per_item)), kApplyThreads, s, st, p,
                                       parents, children, w, l));
    return KPOOL_OK;
}

int run_pages_extend(const kpool_page_pool &p, const int32_t *seqs, const int32_t *n_new, int n, int32_t *begin,
                     void *ws, cudaStream_t s)
{
    KPOOL_CUDA_CHECK(launch_after(extend_kernel, 1, plan_threads(n), s, p, seqs, n_new, n, begin, static_cast<int *>(ws), lists(ws, n)));
    return KPOOL_OK;
}

int run_pages_write(const kpool_page_pool &p, const int32_t *seqs, const int32_t *begin, const int32_t *cu_rows,
                    int n, int64_t total, const void *rows, int64_t rows_layer_stride, const kpool_page_store &g,
                    void *ws, cudaStream_t s)
{
    const int64_t tasks = total * g.n_layers;
    if (n > 0 && tasks * 32 <= kCluster * kWriteClusterThreads) {
        const int blocks = std::max(1, static_cast<int>((tasks * 32 + kWriteClusterThreads - 1) / kWriteClusterThreads));
        KPOOL_CUDA_CHECK(launch_clusters_after(blocks, write_kernel<true>, blocks, kWriteClusterThreads, s, p, seqs, begin, cu_rows, n, total,
                                      static_cast<const char *>(rows), rows_layer_stride, g, static_cast<int *>(ws)));
        return KPOOL_OK;
    }
    KPOOL_CUDA_CHECK(launch_after(clear_status, 1, 1, s, static_cast<int *>(ws)));
    if (n == 0) return KPOOL_OK;
    // (more blocks than fit at once: a warp has one row's chain of lookups to wait for)
    const int64_t blocks = std::min<int64_t>((tasks * 32 + kApplyThreads - 1) / kApplyThreads, 1 << 20);
    KPOOL_CUDA_CHECK(launch_after(write_kernel<false>, static_cast<int>(blocks), kApplyThreads, s, p, seqs, begin, cu_rows, n, total,
                                  static_cast<const char *>(rows), rows_layer_stride, g, static_cast<int *>(ws)));
    return KPOOL_OK;
}

int run_pages_free(const kpool_page_pool &p, const int32_t *seqs, int n, void *ws, cudaStream_t s)
{
    const Lists l = lists(ws, n);
    int *w = static_cast<int *>(ws), *bits = l.mark + std::max(p.n_seqs, p.n_pages);
    KPOOL_CUDA_CHECK(launch_after(free_plan, 1, plan_threads(n), s, p, seqs, n, w, l, bits));
    const int64_t spans = (p.max_pages + kSpan - 1) / kSpan;
    KPOOL_CUDA_CHECK(launch_after(free_apply, grid_for(n * spans), kApplyThreads, s, p, seqs, w, l, bits));
    return KPOOL_OK;
}

int run_pages_compact(const kpool_page_pool &p, const kpool_page_store *stores, int n_stores, void *ws,
                      cudaStream_t s)
{
    const Stores st = pack(stores, n_stores);
    const Lists l = lists(ws, p.n_pages);
    int *w = static_cast<int *>(ws);
    KPOOL_CUDA_CHECK(launch_after(compact_plan, 1, kPlanThreads, s, p, w, l));
    const int64_t spans = (p.max_pages + kSpan - 1) / kSpan;
    KPOOL_CUDA_CHECK(launch_after(
        compact_apply, grid_for(std::max<int64_t>(p.n_seqs * spans, static_cast<int64_t>(p.n_pages) / 2 * st.per_item)),
        kApplyThreads, s, st, p, w, l));
    return KPOOL_OK;
}

}  // namespace kpool

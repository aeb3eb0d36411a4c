// Attention of a batch whose sequences share prefixes, over a paged latent
// cache (absorbed form: latent rows are keys and values).  include/kpool.h
// states the contract.  For query row (t, h) of sequence b, over the tokens
// j < vis(t) that it sees:
//
//   s_j = scale * q[t, h, :] . c_b[j, :]
//   o[t, h, :] = sum_j softmax_j(s) c_b[j, :],   lse[t, h] = ln sum_j exp(s_j)
//
// The (query, head) rows of a group are one flat matrix, and so are those of a
// sequence.  A unit is 128 such rows against a span of tokens: a group's rows
// against its shared tokens, read once for all of them, or a sequence's rows
// against its own.  Three kernels:
//   plan      one block: lengths, units, and an even cut of all units' tiles
//             (256 tokens each) over the CTA pairs.  A cut may fall inside a
//             unit, so a long prefix under few rows still fills the GPU.
//   attend    one CTA pair per piece of a unit, persistent: unnormalised
//             softmax with a running maximum, FP32 partial rows and their
//             log-sum-exp to the workspace.
//   combine   a block per row where rows are few, a warp per row otherwise: joins a
//             row's pieces, the shared ones and its own.
//
// attend, per CTA pair.  The output of 128 rows x 512 columns fills all of one
// SM's tensor memory, so two SMs share it: tcgen05.mma with cta_group::2,
// M = 128, gives each CTA 64 rows, as 2 x 64 lanes (lanes 0-63 the first half of
// the N columns, lanes 64-127 the second).  Each CTA then holds
//   O  [64 x 512]  256 columns of tensor memory, and
//   S  [64 x 256]  128 columns, twice, so that the scores of the next tile run
//                  while the softmax works on this one.
// Both products take N = 256, at which the pair form runs at full rate (64
// cycles per 128 x 256 x 16 MMA measured; N = 128 takes 49, for half the work).
// Operand B is split: for the scores each CTA brings 128 of the tile's 256
// tokens (K-major), for the output 256 of the 512 latent columns of all its
// tokens (MN-major).  Each product has a ring of four 16 KB chunks, each
// feeding four MMAs.  (Keeping the quarter of a tile that both products use
// would need 64 KB that the 64 KB of queries, the 32 KB of P and the rings
// leave no room for.)
//   warp 0       TMA producer of queries and scores chunks
//   warp 1       issuer of the scores' MMAs (CTA 0)
//   warp 2       issuer of the output's MMAs (CTA 0).  Two issuers, because one
//                that waits and commits for every four MMAs reaches 98 cycles
//                an MMA, two together the pipe's 64 (measured)
//   warp 3       TMA producer of values chunks
//   warps 4-11   softmax and output: thread (lane, half of the columns) has 64
//                of a row's 256 scores
//   warp 12      clears the rows of a chunk of values that lie outside the span,
//                so that nothing there, NaN included, meets a weight of 0.  (Ahead
//                of the issuer, while the softmax works: in the issuer's own loop
//                the first and last chunks of a short span took 2 us: 16 samples
//                over 8191 shared tokens 34.0 -> 32.7 us a call, 64 queries each
//                over 8192 of their own 195 -> 184.)
// All loads and arrivals meet on CTA 0's barriers, where the issuers wait.  P
// passes in four parts of 64 tokens, so that the output of a tile's first part
// begins while the last one is exponentiated, and the next tile's P is written
// behind the parts that are still being read.
#include <cuda_bf16.h>

#include <algorithm>

#include "kpool_internal.h"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kDc = 512;
constexpr int kRows = 128;               // rows of a unit
constexpr int kCtaRows = 64;             // of them in each CTA
constexpr int kTile = 256;               // tokens of a tile
constexpr int kOverhead = 3;             // a piece's start and end, in tiles (for the even cut: 2 takes 194 us where 3 takes 191, 64 samples over 32768 shared tokens)
constexpr int kThreads = 416;
constexpr int kSmWarps = 8;
constexpr int kClearWarp = 4 + kSmWarps;
constexpr int kPlanThreads = 1024;
// What the plan keeps in shared memory: its lists up to about 6000 sequences, and the
// units that fit beside them.  (With room for 1024 of each, 1000 sequences in 50 groups
// planned in 22.7 us and 2000 in 43.6, now in 19.7 and 34.4: one block plans them all.)
constexpr int kPlanListBytes = 96 * 1024, kPlanSmem = 200 * 1024;
constexpr int kMaxClusters = 80;         // CTA pairs that a workspace has room for
constexpr int64_t kBlockRows = 512;      // rows up to which combine takes a block for each
constexpr float kRescale = 8.f;          // headroom of the reference maximum (log2)
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint64_t kLandNs = 2000000ull;
constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kTmemCols = 512;           // O: 0..255, S: 256..383 and 384..511
constexpr int kTmemS = 256;

// shared memory (from a 1024-byte aligned base)
constexpr int kChunk = 16384;
constexpr int kRing = 4;                 // chunks of each ring
constexpr int kOffQ = 0;                           // 8 x [64 rows x 64 columns]
constexpr int kOffP = kOffQ + 8 * 8192;            // 4 x [64 rows x 64 tokens]
constexpr int kOffK = kOffP + 4 * 8192;            // scores chunks
constexpr int kOffV = kOffK + kRing * kChunk;      // values chunks
constexpr int kOffRed = kOffV + kRing * kChunk;    // [4][64] floats
constexpr int kOffWord = kOffRed + 4 * kCtaRows * 4; // agreement words [2 groups][2][4]
constexpr int kOffBar = kOffWord + 64;
enum {
    B_KFULL = 0, B_KEMPTY = B_KFULL + kRing, B_VFULL = B_KEMPTY + kRing, B_VEMPTY = B_VFULL + kRing,
    B_VEDGE = B_VEMPTY + kRing, B_PFULL = B_VEDGE + kRing, B_PFREE = B_PFULL + 4, B_SFULL = B_PFREE + 4,
    B_SFREE = B_SFULL + 2, B_QFULL = B_SFREE + 2, B_QEMPTY, B_DRAIN, N_BARS = B_DRAIN + 2
};
constexpr int kOffMisc = kOffBar + N_BARS * 8;     // [0] tmem base, [1] abort flag
constexpr int kSmemBytes = kOffMisc + 16 + 1024;   // and alignment slack
static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");

// workspace header (ints)
enum { H_STATUS = 1, H_OK = 2, H_INTS = 64 };

struct Unit {
    int row0, nrows;         // flat (query, head) rows
    int table_row;           // page-table row its tokens are read through
    int t0, t1, tiles;       // tokens t0 .. t1 - 1, in tiles from t0's box on
    int c0, pieces;          // cut into pieces, for the clusters c0, c0 + 1, ...
    int64_t w0;              // first position of the unit in the cut work
    int64_t out0;            // first partial row
};
static_assert(sizeof(Unit) == 48, "Unit");

struct Token {               // per query
    int vis;                 // tokens it sees
    int pu, prow0;           // its group's first unit, and that unit's first row
    int su, srow0;           // its sequence's
};

// Where a cluster begins: all that it reads before its first loads, in one place.
struct __align__(16) Start {
    int u, units;            // its first unit and the number of them, among those with tiles
    int64_t from, to;        // its share of the work
    Unit first;
};

struct Work {
    int *head;               // header
    Token *tok;              // [Tq]
    int *lists;              // [3 B + 2 G]: the plan's, when they do not fit shared memory
    Start *start;            // [clusters]
    Unit *unit;              // all, in the order of the rows
    Unit *live;              // those with tiles
    float *lse;              // [partial rows], base 2
    float *o;                // [partial rows, 512]
};

constexpr int kFewStarts = 16;            // start entries that one thread writes

struct Params {
    PrefixMlaArgs a;
    Work w;
    int clusters;
    int box, box_log;        // rows of a TMA box, and its logarithm
    int page_log;
    float c_scale;           // softmax scale * log2(e)
    int wait_tries;          // see Sync
    uint32_t wait_nap_ns;
    uint64_t wait_limit_ns;
    int plan_units;          // units that fit the plan's shared memory
    bool plan_lists;         // do its lists?
};

__device__ __forceinline__ bool in_range(int i, int n) { return i >= 0 && i < n; }

// ---- plan --------------------------------------------------------------------

// The last i in [0, n) with cu[i] <= r.
__device__ int segment_of(const int32_t *cu, int n, int r)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Exclusive prefix sum over the block; *total gets the sum.
__device__ int64_t block_exclusive(int64_t v, int64_t *scratch, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t t = lane < static_cast<int>(blockDim.x >> 5) ? scratch[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, t, d);
            if (lane >= d) t += y;
        }
        scratch[lane] = t;
    }
    __syncthreads();
    *total = scratch[31];
    return x - v + (warp > 0 ? scratch[warp - 1] : 0);
}

// Reads its lists once, into shared memory where they fit (any realistic
// batch), so that the searches and scans behind it do not wait for the L2.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Params p)
{
    extern __shared__ __align__(16) uint8_t plan_smem[];
    __shared__ int64_t scratch[32];
    __shared__ int status;
    const PrefixMlaArgs &a = p.a;
    const Work &w = p.w;
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();         // what came before in the stream
    if (threadIdx.x == 0) status = 0;
    __syncthreads();
    const int entities = a.G + a.B;          // groups, then sequences
    const bool small = p.plan_lists;
    int *lists = small ? reinterpret_cast<int *>(plan_smem + p.plan_units * sizeof(Unit)) : w.lists;
    int *len = lists, *shared = len + a.B, *row = shared + a.G, *unit0 = row + a.B;
    const int32_t *cu_q = a.cu_q, *cu_g = a.cu_groups;
    // (the first entry of each list is held back, so that all loads are in flight at once)
    int my_q = 0, my_g = 0, my_p = 0;
    if (threadIdx.x < a.B) my_q = a.cu_q[threadIdx.x];
    if (threadIdx.x < a.G) my_g = a.cu_groups[threadIdx.x], my_p = a.prefix_lens[threadIdx.x];
    const int last_q = a.cu_q[a.B], last_g = a.cu_groups[a.G];
    const int64_t room = static_cast<int64_t>(a.max_pages) * a.page_size;
    // a sequence's length, cut to what its table row holds
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        int r = a.seq_ids != nullptr ? a.seq_ids[b] : b;
        int64_t n = -1;
        if (in_range(r, a.n_rows)) n = a.seq_lens[r];
        else r = 0;
        if (n < 0 || n > room) {
            atomicOr(&status, KPOOL_STATUS_BAD_PAGE);
            n = n < 0 ? 0 : room;
        }
        row[b] = r;
        len[b] = static_cast<int>(n);
    }
    if (threadIdx.x < a.G) shared[threadIdx.x] = my_p;
    for (int i = threadIdx.x + blockDim.x; i < a.G; i += blockDim.x) shared[i] = a.prefix_lens[i];
    if (small) {
        int *q = unit0 + entities, *g = q + a.B + 1;
        const int i = threadIdx.x;
        if (i < a.B) q[i] = my_q;
        if (i < a.G) g[i] = my_g;
        for (int j = i + blockDim.x; j < a.B; j += blockDim.x) q[j] = a.cu_q[j];
        for (int j = i + blockDim.x; j < a.G; j += blockDim.x) g[j] = a.cu_groups[j];
        if (i == 0) q[a.B] = last_q, g[a.G] = last_g;
        cu_q = q;
        cu_g = g;
    }
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i <= a.B; i += blockDim.x) bad |= i == 0 ? cu_q[0] != 0 : cu_q[i] < cu_q[i - 1];
    for (int i = threadIdx.x; i <= a.G; i += blockDim.x) bad |= i == 0 ? cu_g[0] != 0 : cu_g[i] < cu_g[i - 1];
    bad |= last_q != a.Tq || last_g != a.B;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            w.head[H_STATUS] = KPOOL_STATUS_BAD_SEQLENS;
            w.head[H_OK] = 0;
        }
        for (int c = threadIdx.x; c < p.clusters; c += blockDim.x) w.start[c] = Start{};
        return;
    }
    // units of every group, then of every sequence
    int64_t units = 0;
    for (int base = 0; base < entities; base += blockDim.x) {
        const int e = base + threadIdx.x;
        int n = 0;
        if (e < entities) {
            const int b0 = e < a.G ? cu_g[e] : e - a.G;
            const int b1 = e < a.G ? cu_g[e + 1] : b0 + 1;
            n = static_cast<int>((static_cast<int64_t>(cu_q[b1] - cu_q[b0]) * a.H + kRows - 1) / kRows);
            // shared tokens are read through the group's first sequence
            if (e < a.G) shared[e] = b1 > b0 ? min(max(shared[e], 0), len[b0]) : 0;
        }
        int64_t total;
        const int64_t at = units + block_exclusive(n, scratch, &total);
        if (e < entities) unit0[e] = static_cast<int>(at);
        units += total;
    }
    __syncthreads();
    // each unit's span, and its place in the work; how many have tiles (one scan for
    // both: units are below 2^26)
    constexpr int kLow = 26;
    constexpr int64_t kLowMask = (int64_t(1) << kLow) - 1;
    Unit *unit = units <= p.plan_units ? reinterpret_cast<Unit *>(plan_smem) : w.unit;
    int64_t work = 0;
    int live = 0;
    for (int64_t base = 0; base < units; base += blockDim.x) {
        const int64_t k = base + threadIdx.x;
        Unit u{};
        if (k < units) {
            const int e = segment_of(unit0, entities, static_cast<int>(k));
            const int b0 = e < a.G ? cu_g[e] : e - a.G;
            const int b1 = e < a.G ? cu_g[e + 1] : b0 + 1;
            const int r0 = cu_q[b0] * a.H, rows = cu_q[b1] * a.H - r0, at = (static_cast<int>(k) - unit0[e]) * kRows;
            u.row0 = r0 + at;
            u.nrows = min(kRows, rows - at);
            u.table_row = row[b0];
            if (e < a.G) {
                u.t1 = shared[e];
            } else {
                // up to what the last of the rows' queries sees
                const int last = (u.row0 + u.nrows - 1) / a.H;
                u.t0 = shared[segment_of(cu_g, a.G, b0)];
                u.t1 = len[b0] - (cu_q[b1] - 1 - last);
            }
            u.tiles = u.t1 > u.t0 ? (u.t1 - (u.t0 & -p.box) + kTile - 1) / kTile : 0;
        }
        int64_t total;
        u.w0 = work + (block_exclusive(u.tiles > 0 ? static_cast<int64_t>(u.tiles + kOverhead) << kLow | 1 : 0, scratch,
                                       &total) >> kLow);
        if (k < units) unit[k] = u;
        work += total >> kLow;
        live += static_cast<int>(total & kLowMask);
    }
    // queries
    for (int t = threadIdx.x; t < a.Tq; t += blockDim.x) {
        const int b = segment_of(cu_q, a.B, t), g = segment_of(cu_g, a.G, b);
        Token x;
        x.vis = max(0, len[b] - (cu_q[b + 1] - 1 - t));
        x.pu = unit0[g];
        x.prow0 = cu_q[cu_g[g]] * a.H;
        x.su = unit0[a.G + b];
        x.srow0 = cu_q[b] * a.H;
        w.tok[t] = x;
    }
    // the even cut: where each cluster begins, and each unit's partial rows
    const int64_t share = max(static_cast<int64_t>(1), (work + p.clusters - 1) / p.clusters);
    for (int c = threadIdx.x; c < p.clusters; c += blockDim.x)
        if (c * share >= work) w.start[c] = Start{};
    int64_t rows = 0;
    int place = 0;
    for (int64_t base = 0; base < units; base += blockDim.x) {
        const int64_t k = base + threadIdx.x;
        Unit u{};
        if (k < units) {
            u = unit[k];
            if (u.tiles > 0) {
                // the clusters whose share of the work touches its tiles
                const int64_t c0 = (u.w0 + kOverhead) / share;
                u.c0 = static_cast<int>(c0);
                u.pieces = static_cast<int>((u.w0 + kOverhead + u.tiles - 1) / share - c0) + 1;
            }
        }
        int64_t total;
        // (partial rows, below 2^33, and units with tiles in one scan)
        const int64_t before = block_exclusive(
            u.tiles > 0 ? (static_cast<int64_t>(u.pieces) * u.nrows) << kLow | 1 : 0, scratch, &total);
        u.out0 = rows + (before >> kLow);
        const int j = place + static_cast<int>(before & kLowMask);
        int c0 = 0, c1 = 0;                  // the clusters that begin in it
        if (k < units) {
            w.unit[k] = u;
            if (u.tiles > 0) {
                w.live[j] = u;
                c0 = static_cast<int>((u.w0 + share - 1) / share);
                c1 = static_cast<int>((u.w0 + u.tiles + kOverhead + share - 1) / share);
            }
        }
        // a thread writes a few; the many of a long unit its whole warp (one sequence of
        // 131072 tokens: 53 -> 48.4 us)
        const bool many = c1 - c0 > kFewStarts;
        for (int c = c0; c < c1 && !many; ++c) w.start[c] = Start{j, live, c * share, (c + 1) * share, u};
        for (unsigned m = __ballot_sync(kFull, many); m != 0; m &= m - 1) {
            const int from = __ffs(m) - 1;
            Unit v;
            const int *src = reinterpret_cast<const int *>(&u);
            int *dst = reinterpret_cast<int *>(&v);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(Unit) / 4); ++i) dst[i] = __shfl_sync(kFull, src[i], from);
            const int vj = __shfl_sync(kFull, j, from), end = __shfl_sync(kFull, c1, from);
            for (int c = __shfl_sync(kFull, c0, from) + static_cast<int>(threadIdx.x & 31); c < end; c += 32)
                w.start[c] = Start{vj, live, c * share, (c + 1) * share, v};
        }
        rows += total >> kLow;
        place += static_cast<int>(total & kLowMask);
    }
    if (threadIdx.x == 0) {
        w.head[H_STATUS] = status;
        w.head[H_OK] = 1;
    }
}

// ---- attend ------------------------------------------------------------------

struct Sync {
    volatile uint32_t *abort_flag;
    int *status;
    int tries;               // before the timer is read
    uint32_t nap_ns;         // one try's suspension
    uint64_t limit_ns;
};

// Bounded mbarrier wait: completion, then the CTA abort flag, then a timer that
// raises the flag and KPOOL_STATUS_TIMEOUT.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Sync &sy)
{
    // (the timer is slow to read: it would add its latency to each hop of the pipeline)
#pragma unroll 1
    for (int i = 0; i < sy.tries; ++i)
        if (ptx::mbar_try_wait_ns(bar, parity, sy.nap_ns)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        if (ptx::mbar_try_wait_ns(bar, parity, sy.nap_ns)) return true;
        if (*sy.abort_flag) return false;
        if (ptx::globaltimer() - t0 > sy.limit_ns) {
            *sy.abort_flag = 1u;
            atomicOr(sy.status, KPOOL_STATUS_TIMEOUT);
            return false;
        }
    }
}

// All lanes wait; false when any of them gave up.
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, const Sync &sy)
{
    const bool ok = wait_bar(bar, parity, sy);
    return __all_sync(kFull, ok);
}

// A wait that other tiles may pass in front of: `pace`, whose phase turns with each
// of them, starts the limit anew.  (Polled much faster than tiles go by: a wait that
// suspends may see every second one.  A counter that another warp writes costs
// that warp 1% of a long call.)
__device__ __forceinline__ bool wait_paced_warp(uint32_t bar, uint32_t parity, uint32_t pace, const Sync &sy)
{
    bool ok = ptx::mbar_test(bar, parity), turn = ptx::mbar_test(pace, 0);
    for (uint64_t t0 = ptx::globaltimer(); !ok; ok = ptx::mbar_test(bar, parity)) {
        if (*sy.abort_flag) break;
        const bool now = ptx::mbar_test(pace, 0);
        if (now != turn) {
            turn = now;
            t0 = ptx::globaltimer();
        } else if (ptx::globaltimer() - t0 > sy.limit_ns) {
            *sy.abort_flag = 1u;
            atomicOr(sy.status, KPOOL_STATUS_TIMEOUT);
            break;
        }
        __nanosleep(100);
    }
    return __all_sync(kFull, ok);
}

// A wait for work in flight before the CTA ends: blind to the abort flag, and bounded.
__device__ __forceinline__ void wait_landed(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer() - t0 > kTimeoutNs) break;
}

// One cluster's share of a unit.
struct Piece {
    int row0, nrows, table_row, t0, t1;
    int base, tiles;         // token at which its first tile begins; tiles
    int64_t out;             // first partial row

    // what the issuing warps read, broadcast to be the same in all lanes
    __device__ void uniform()
    {
        row0 = __shfl_sync(kFull, row0, 0);
        t0 = __shfl_sync(kFull, t0, 0);
        t1 = __shfl_sync(kFull, t1, 0);
        base = __shfl_sync(kFull, base, 0);
        tiles = __shfl_sync(kFull, tiles, 0);
    }
};

struct Walk {
    const Unit *live;
    Unit x;                  // unit u
    int u, units, box, cluster;
    int64_t from, to;

    __device__ Walk(const Params &p, int c) : live(p.w.live), box(p.box), cluster(c)
    {
        const Start s = p.w.start[c];
        u = s.u;
        units = s.units;
        from = s.from;
        to = s.to;
        x = s.first;
    }
    __device__ bool next(Piece *q)
    {
        while (u < units && x.w0 < to) {
            const int64_t begin = x.w0 + kOverhead;
            const int64_t lo = max(begin, from), hi = min(begin + x.tiles, to);
            const bool some = lo < hi;
            if (some) {
                q->row0 = x.row0;
                q->nrows = x.nrows;
                q->table_row = x.table_row;
                q->t0 = x.t0;
                q->t1 = x.t1;
                q->base = (x.t0 & -box) + static_cast<int>(lo - begin) * kTile;
                q->tiles = static_cast<int>(hi - lo);
                q->out = x.out0 + static_cast<int64_t>(cluster - x.c0) * x.nrows;
            }
            if (++u < units) x = live[u];
            if (some) return true;
        }
        return false;
    }
};

// Tokens of the tile that begins at `base`, of those before t1.
__device__ __forceinline__ int tile_tokens(const Piece &q, int base) { return min(kTile, q.t1 - base); }

// Does the chunk of values that holds tokens 64 kb .. of the tile at `base` have
// rows outside the span?
__device__ __forceinline__ bool has_edge(const Piece &q, int base, int kb)
{
    return q.t0 - base > 64 * kb || tile_tokens(q, base) < 64 * kb + 64;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                  const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t sQ = sbase + kOffQ, sP = sbase + kOffP, sK = sbase + kOffK, sV = sbase + kOffV;
    auto bar = [&](int i) { return sbase + kOffBar + 8 * i; };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    // (a broadcast, so that the compiler sees that a warp takes one role together)
    const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;             // of the CTA in its pair
    const int cluster = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        // (CTA 0's of the "full" barriers are the ones in use)
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(bar(B_KFULL + i), 2);             // a producer of each CTA
            ptx::mbar_init(bar(B_KEMPTY + i), 1);
            ptx::mbar_init(bar(B_VFULL + i), 2);             // a producer, or the clearing warp, of each
            ptx::mbar_init(bar(B_VEMPTY + i), 1);
            ptx::mbar_init(bar(B_VEDGE + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(bar(B_PFULL + i), 4);             // two softmax warps of each CTA
            ptx::mbar_init(bar(B_PFREE + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(B_SFULL + i), 1);
            ptx::mbar_init(bar(B_SFREE + i), 2 * kSmWarps);  // the softmax warps of both CTAs
            ptx::mbar_init(bar(B_DRAIN + i), 1);
        }
        ptx::mbar_init(bar(B_QFULL), 2);
        ptx::mbar_init(bar(B_QEMPTY), 1);
        misc[1] = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(&misc[0]), kTmemCols);
        ptx::tmem_relinquish_pair();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::cluster_sync();                 // no remote arrival before the peer's barriers exist
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, misc[0], 0);
    const Sync sy{reinterpret_cast<volatile uint32_t *>(&misc[1]), p.w.head + H_STATUS, p.wait_tries, p.wait_nap_ns, p.wait_limit_ns};
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();         // the plan

    if (warp == 0 || warp == 3) {
        // ---------------- producers ----------------
        const int box = p.box, bl = p.box_log, pl = p.page_log, in_page = p.a.page_size - 1;
        if (lane == 0) {
            ptx::tma_prefetch_desc(&tm_q);
            ptx::tma_prefetch_desc(&tm_kv);
        }
        // Queries and scores chunks: as for the MMAs, the loop runs in all lanes on
        // operands that are the same in all, and one lane issues.  Values chunks: a
        // lane per load, whose coordinates stay in registers over both halves of the
        // columns.  (Measured against each other on 64 sequences over 32768 shared
        // tokens: the values by one lane 194 us, this 189; the scores by lanes 189, but
        // 21.2 against 20.6 us on four short sequences.)
        const bool one = ptx::elect_one();
        const int r128 = 128 * static_cast<int>(rank);
        bool ok = true;
        uint32_t g = 0, np = 0;          // chunks and pieces so far
        Walk walk(p, cluster);
        Piece pc;
        // page of each of a tile's boxes, lane j that of box j
        auto pages_at = [&](int base) {
            int page = 0;
            if (lane * box < tile_tokens(pc, base)) {
                // (an ordinary load: the read-only path asks for data that stay as they are
                // from the grid's start, and a call that changes the table may still run then)
                page = p.a.page_table[static_cast<int64_t>(pc.table_row) * p.a.max_pages + ((base + lane * box) >> pl)];
                if (!in_range(page, p.a.n_pages)) {
                    atomicOr(sy.status, KPOOL_STATUS_BAD_PAGE);
                    page = p.a.n_pages;  // out of the map's bounds: reads as zeros
                }
            }
            return page;
        };
        // waits for the next slot of the ring and announces `bytes` for it
        auto take = [&](int empty, uint32_t to, uint32_t s, int bytes) {
            ok = wait_bar_warp(bar(empty + s), ((g / kRing) & 1u) ^ 1u, sy);
            if (ok && one) ptx::mbar_arrive_expect_tx_cluster(to, bytes);
            ++g;
        };
        while (ok && walk.next(&pc)) {
            pc.uniform();
            if (warp == 0) {
                int page = pages_at(pc.base);
                ok = wait_bar_warp(bar(B_QEMPTY), (np & 1u) ^ 1u, sy);
                if (!ok) break;
                const uint32_t qbar = ptx::map_to_rank(bar(B_QFULL), 0);
                if (one) {
                    ptx::mbar_arrive_expect_tx_cluster(qbar, 8 * 8192);
                    for (int k = 0; k < 8; ++k)
                        ptx::tma_load_2d_pair(sQ + k * 8192, &tm_q, qbar, 64 * k, pc.row0 + kCtaRows * static_cast<int>(rank));
                }
                ++np;
                for (int i = 0; i < pc.tiles && ok; ++i) {
                    // this CTA's 128 tokens, 64 columns at a time
                    const int base = pc.base + i * kTile;
                    const int next = i + 1 < pc.tiles ? pages_at(base + kTile) : 0;
                    const int n = max(0, min(128, tile_tokens(pc, base) - r128));
                    const int boxes = (n + box - 1) >> bl;
                    for (int k = 0; k < 8 && ok; ++k) {
                        const uint32_t s = g % kRing, to = ptx::map_to_rank(bar(B_KFULL + s), 0);
                        take(B_KEMPTY, to, s, boxes * box * 128);
                        if (!ok) break;
                        for (int j = 0; j < boxes; ++j) {
                            const int at = (r128 >> bl) + j;
                            const int pg = __shfl_sync(kFull, page, at);
                            if (one)
                                ptx::tma_load_3d_pair(sK + s * kChunk + j * box * 128, &tm_kv, to, 64 * k,
                                                      (base + at * box) & in_page, pg);
                        }
                    }
                    page = next;
                }
            } else {
                int page = pages_at(pc.base);
                for (int i = 0; i < pc.tiles && ok; ++i) {
                    // 64 tokens x 128 of this CTA's 256 columns: lanes 2j and 2j + 1 bring
                    // the two 64-column halves of box j
                    const int base = pc.base + i * kTile;
                    const int next = i + 1 < pc.tiles ? pages_at(base + kTile) : 0;
                    const int n = tile_tokens(pc, base);
                    for (int kb = 0; 64 * kb < n && ok; ++kb) {
                        const int boxes = (min(64, n - 64 * kb) + box - 1) >> bl;
                        const bool edge = has_edge(pc, base, kb);
                        const int at = (64 * kb >> bl) + (lane >> 1);
                        const int pg = __shfl_sync(kFull, page, at & 31);
                        const int y = (base + at * box) & in_page;
                        for (int j = 0; j < 2 && ok; ++j) {
                            const uint32_t s = g % kRing;
                            const uint32_t to = edge ? ptx::map_to_rank(bar(B_VEDGE + s), rank)
                                                     : ptx::map_to_rank(bar(B_VFULL + s), 0);
                            take(B_VEMPTY, to, s, 2 * boxes * box * 128);
                            if (ok && lane < 2 * boxes)
                                ptx::tma_load_3d_pair(sV + s * kChunk + (lane & 1) * 8192 + (lane >> 1) * box * 128, &tm_kv,
                                                      to, 256 * static_cast<int>(rank) + 128 * j + 64 * (lane & 1), y, pg);
                        }
                    }
                    page = next;
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- issuer of the scores ----------------
        // The whole warp runs the loop and one lane issues: operands that are the
        // same in all lanes stay in uniform registers, which the MMAs take them
        // from (a lone thread's loop moves each one over first: 120 cycles an MMA).
        if (rank == 0) {
            constexpr uint32_t idesc = ptx::make_idesc(1u, kRows, kTile);
            bool ok = true, any = false;
            uint32_t g = 0, np = 0, gs = 0;          // chunks, pieces and tiles so far
            const bool one = ptx::elect_one();
            Walk walk(p, cluster);
            Piece pc;
            while (ok && walk.next(&pc)) {
                pc.uniform();
                ok = wait_bar_warp(bar(B_QFULL), np & 1u, sy);
                ++np;
                for (int i = 0; i < pc.tiles && ok; ++i, ++gs) {
                    // the tile before the last has been read
                    ok = wait_bar_warp(bar(B_SFREE + (gs & 1u)), ((gs >> 1) & 1u) ^ 1u, sy);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + kTmemS + (gs & 1u) * 128;
                    for (int k = 0; k < 8; ++k, ++g) {
                        const uint32_t s = g % kRing;
                        ok = wait_bar_warp(bar(B_KFULL + s), (g / kRing) & 1u, sy);
                        if (!ok) break;
                        const uint64_t ad = ptx::smem_desc_sw128(sQ + k * 8192);
                        const uint64_t bd = ptx::smem_desc_sw128(sK + s * kChunk);
                        if (one) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                ptx::mma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
                            ptx::mma_commit_pair(bar(B_KEMPTY + s));
                        }
                        any = true;
                    }
                    if (ok && one) {
                        ptx::mma_commit_pair(bar(B_SFULL + (gs & 1u)));
                        if (i + 1 == pc.tiles) ptx::mma_commit_pair(bar(B_QEMPTY));
                    }
                }
            }
            if (any) {
                // none of these MMAs is in flight once this has arrived
                if (one) ptx::mma_commit_pair(bar(B_DRAIN));
                wait_landed(bar(B_DRAIN), 0);
            }
        }
    } else if (warp == 2) {
        // ---------------- issuer of the output ----------------
        if (rank == 0) {
            constexpr uint32_t idesc = ptx::make_idesc(1u, kRows, kTile) | ptx::kIdescBMajorMN;
            bool ok = true, any = false;
            uint32_t g = 0, gp = 0;                      // chunks and tiles so far
            const bool one = ptx::elect_one();
            Walk walk(p, cluster);
            Piece pc;
            while (ok && walk.next(&pc)) {
                pc.uniform();
                for (int i = 0; i < pc.tiles && ok; ++i, ++gp) {
                    const int n = tile_tokens(pc, pc.base + i * kTile);
                    for (int kb = 0; 64 * kb < n && ok; ++kb) {
                        ok = wait_bar_warp(bar(B_PFULL + kb), gp & 1u, sy);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const int steps = min(4, (n - 64 * kb + 15) / 16);
                        for (int j = 0; j < 2; ++j, ++g) {
                            const uint32_t s = g % kRing;
                            ok = wait_bar_warp(bar(B_VFULL + s), (g / kRing) & 1u, sy);
                            if (!ok) break;
                            const uint64_t ad = ptx::smem_desc_sw128(sP + kb * 8192);
                            const uint64_t bd = ptx::smem_desc_mn_sw128(sV + s * kChunk, 8192);
                            const uint32_t d = tmem + j * 128;
                            const bool more = i > 0 || kb > 0;
                            if (one) {
                                if (steps == 4) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        ptx::mma_bf16_pair(d, ad + 2 * kk, bd + 128 * kk, idesc, more || kk > 0);
                                } else {
                                    for (int kk = 0; kk < steps; ++kk)
                                        ptx::mma_bf16_pair(d, ad + 2 * kk, bd + 128 * kk, idesc, more || kk > 0);
                                }
                                ptx::mma_commit_pair(bar(B_VEMPTY + s));
                                if (j == 1) ptx::mma_commit_pair(bar(B_PFREE + kb));
                            }
                            any = true;
                        }
                    }
                    // parts without a token pass as well
                    for (int kb = (n + 63) / 64; kb < 4 && ok; ++kb) {
                        ok = wait_bar_warp(bar(B_PFULL + kb), gp & 1u, sy);
                        if (ok && one) ptx::mma_commit_pair(bar(B_PFREE + kb));
                    }
                }
            }
            if (any) {
                if (one) ptx::mma_commit_pair(bar(B_DRAIN + 1));
                wait_landed(bar(B_DRAIN + 1), 0);
            }
        }
    } else if (warp == kClearWarp) {
        // ---------------- clearing ----------------
        bool ok = true;
        uint32_t g = 0, par = 0;                     // chunks so far; parity of each slot's edge barrier
        Walk walk(p, cluster);
        Piece pc;
        while (ok && walk.next(&pc)) {
            pc.uniform();
            for (int i = 0; i < pc.tiles && ok; ++i) {
                const int base = pc.base + i * kTile;
                const int n = tile_tokens(pc, base), lo = pc.t0 - base;
                for (int kb = 0; 64 * kb < n && ok; ++kb) {
                    if (!has_edge(pc, base, kb)) {
                        g += 2;
                        continue;
                    }
                    // rows outside the span, up to the last 16 that the MMAs read
                    const int steps = min(4, (n - 64 * kb + 15) / 16);
                    const int cut0 = lo - 64 * kb, cut1 = n - 64 * kb;
                    for (int j = 0; j < 2; ++j, ++g) {
                        const uint32_t s = g % kRing;
                        // (this warp goes past the chunks without an edge at once)
                        ok = wait_paced_warp(bar(B_VEDGE + s), par >> s & 1u, bar(B_PFREE), sy);
                        if (!ok) break;
                        par ^= 1u << s;
                        for (int r = lane >> 4; r < 16 * steps; r += 2)
                            if (r < cut0 || r >= cut1)
                                ptx::st_shared_v4(sV + s * kChunk + (lane >> 3 & 1) * 8192 + r * 128 + (lane & 7) * 16,
                                                  0u, 0u, 0u, 0u);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(bar(B_VFULL + s), 0));
                        __syncwarp();
                    }
                }
            }
        }
    } else {
        // ---------------- softmax and output ----------------
        const int sw = warp - 4;
        const int quarter = warp & 3;                 // lanes 32 * quarter .. of tensor memory
        const int half = quarter >> 1;                // tokens 128 * half .. of the tile, columns 256 * half .. of the output
        const int part = sw >> 2;                     // 64 of those tokens, 128 of those columns
        const int r = 32 * (quarter & 1) + lane;      // row of this CTA
        const int x0 = 128 * half + 64 * part;        // first of this thread's tokens
        const int group = quarter & 1;                // the four warps that share rows
        const int member = 2 * part + half;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        float *red = reinterpret_cast<float *>(smem + kOffRed);
        volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(smem + kOffWord) + 8 * group;
        const int kb = 2 * half + part;               // part of P that holds them
        const uint32_t prow = sP + kb * 8192 + r * 128;
        const uint32_t p_full = ptx::map_to_rank(bar(B_PFULL + kb), 0);
        const float c = p.c_scale;
        bool ok = true;
        uint32_t gt = 0, rounds = 0;
        // the four warps pass each agreement together: 0 in the common round,
        // else all of their words
        auto agree = [&](uint32_t word) {
            if (!ptx::named_bar_or(1 + group, 128, word != 0u)) return 0u;
            volatile uint32_t *f = words + 4 * (rounds & 1u);
            ++rounds;
            if (lane == 0) f[member] = word;
            ptx::named_bar_sync(3 + group, 128);
            return f[0] | f[1] | f[2] | f[3];
        };
        Walk walk(p, cluster);
        Piece pc;
        bool stop = false;
        while (!stop && walk.next(&pc)) {
            const int row = kCtaRows * static_cast<int>(rank) + r;        // of the unit
            const int vis = row < pc.nrows ? p.w.tok[(pc.row0 + row) / p.a.H].vis : 0;
            const int end = min(pc.t1, vis);
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < pc.tiles; ++i, ++gt) {
                const int base = pc.base + i * kTile;
                ok = ok && wait_bar_warp(bar(B_SFULL + (gt & 1u)), (gt >> 1) & 1u, sy);
                ptx::tc_fence_after();
                float v[64];
                {
                    uint32_t a0[32], a1[32];
                    const uint32_t at = lanes + kTmemS + (gt & 1u) * 128 + 64 * part;
                    ptx::tmem_ld32(at, a0);
                    ptx::tmem_ld32(at + 32, a1);
                    ptx::tmem_ld_wait2(a0, a1);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        v[k] = __uint_as_float(a0[k]);
                        v[32 + k] = __uint_as_float(a1[k]);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(bar(B_SFREE + (gt & 1u)), 0));
                // tokens lo .. hi - 1 of this thread's 64 count
                const int lo = pc.t0 - base - x0, hi = end - base - x0;
                if (__any_sync(kFull, lo > 0 || hi < 64)) {
#pragma unroll
                    for (int k = 0; k < 64; ++k) v[k] = (k >= lo && k < hi) ? v[k] : -INFINITY;
                }
                float top = fmaxf(v[0], v[1]);
#pragma unroll
                for (int k = 2; k < 64; ++k) top = fmaxf(top, v[k]);
                const bool need = top * c > m + kRescale;
                const uint32_t all = agree((ok ? 0u : 1u) | (__any_sync(kFull, need) ? 2u : 0u));
                if (all & 1u) {
                    stop = true;
                    break;
                }
                if (all & 2u) {
                    // the row's exact maximum so far becomes the reference
                    red[member * kCtaRows + r] = top;
                    ptx::named_bar_sync(3 + group, 128);
                    const float t4 = fmaxf(fmaxf(red[r], red[kCtaRows + r]),
                                           fmaxf(red[2 * kCtaRows + r], red[3 * kCtaRows + r]));
                    const float mn = fmaxf(m, t4 * c);
                    const float f = mn == -INFINITY ? 1.f : ptx::ex2_approx(m - mn);
                    m = mn;
                    l *= f;
                    if (i > 0) {
                        // the output so far, once its MMAs are done (the four warps have
                        // met since each waited for its part of the tile before the last,
                        // so these parities mean the last one)
                        for (int k = 0; k < 4; ++k) ok = wait_bar_warp(bar(B_PFREE + k), (gt - 1u) & 1u, sy) && ok;
                        ptx::tc_fence_after();
                        if (__any_sync(kFull, f != 1.f)) {
#pragma unroll 1
                            for (int k = 0; k < 4; ++k) {
                                uint32_t o[32];
                                const uint32_t at = lanes + 128 * part + 32 * k;
                                ptx::tmem_ld32(at, o);
                                ptx::tmem_ld_wait(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                ptx::tmem_st32(at, o);
                            }
                            ptx::tmem_st_wait();
                        }
                    }
                    // red is read, and all of the rows' output rescaled before any
                    // part of the new P lets its MMAs begin
                    ptx::tc_fence_before();
                    ptx::named_bar_sync(3 + group, 128);
                    ptx::tc_fence_after();
                }
                const float ref = m == -INFINITY ? 0.f : m;
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    v[k] = ptx::ex2_approx(fmaf(v[k], c, -ref));
                    sum += v[k];
                }
                l += sum;
                // this part of P is free once the previous tile's MMAs have read it
                if (gt > 0) ok = wait_bar_warp(bar(B_PFREE + kb), (gt - 1u) & 1u, sy) && ok;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t w4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]);
                        w4[e] = *reinterpret_cast<const uint32_t *>(&b2);
                    }
                    ptx::st_shared_v4(prow + ((k ^ (r & 7)) << 4), w4[0], w4[1], w4[2], w4[3]);
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(p_full);
            }
            if (stop) break;
            // the piece's rows: sum over the four threads of each, then the output
            red[member * kCtaRows + r] = l;
            ptx::named_bar_sync(3 + group, 128);
            for (int k = 0; k < 4; ++k) ok = wait_bar_warp(bar(B_PFREE + k), (gt - 1u) & 1u, sy) && ok;
            l = (red[r] + red[kCtaRows + r]) + (red[2 * kCtaRows + r] + red[3 * kCtaRows + r]);
            ptx::named_bar_sync(3 + group, 128);
            ptx::tc_fence_after();
            const float inv = l != 0.f ? 1.f / l : 0.f;      // (0: no token; NaN goes on)
            // 32 columns at a time through this warp's own part of P (which no MMA
            // reads any more), so that a store covers whole lines of four rows: straight
            // from the registers, one row a lane, the stores take twice as long
            const uint32_t stage = prow - lane * 128;
            const int row0 = row - lane;
            float *out = p.w.o + (pc.out + row0) * kDc + 256 * half + 128 * part + 4 * (lane & 7);
#pragma unroll 1
            for (int k = 0; k < 4 && row0 < pc.nrows; ++k) {
                uint32_t o[32];
                ptx::tmem_ld32(lanes + 128 * part + 32 * k, o);
                ptx::tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ptx::st_shared_v4(prow + ((e ^ (lane & 7)) << 4), o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int rr = 4 * e + (lane >> 3);
                    const float4 y = ptx::ld_shared_v4(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                    if (row0 + rr < pc.nrows) *reinterpret_cast<float4 *>(out + rr * kDc + 32 * k) = y;
                }
            }
            __syncwarp();
            if (member == 0 && row < pc.nrows) p.w.lse[pc.out + row] = l != 0.f ? m + log2f(l) : -INFINITY;
            ptx::tc_fence_before();
        }
    }

    // Neither CTA ends while the other may still signal it or read its memory, nor
    // with a load in flight: all have landed when the last tile's MMAs are done,
    // except after an expired wait.  CTA 1's loads complete on CTA 0's barriers,
    // where it cannot wait for them, so it then lets far more time pass than a
    // load takes.
    __syncthreads();
    if (*sy.abort_flag != 0u && threadIdx.x == 0) {
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < kLandNs) __nanosleep(1000);
    }
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
    ptx::cluster_sync();
}

// ---- combine -----------------------------------------------------------------

// The pieces of one row: the shared ones, then the sequence's own.
struct Pieces {
    int64_t shared0, own0;   // partial row of the first of each
    int shared_n, own_n, shared_rows, own_rows;

    __device__ Pieces(const Params &p, int64_t row, const Token &x)
    {
        const int ks = static_cast<int>(row - x.prow0), ko = static_cast<int>(row - x.srow0);
        const Unit us = p.w.unit[x.pu + ks / kRows], uo = p.w.unit[x.su + ko / kRows];
        shared_n = us.pieces;
        own_n = uo.pieces;
        shared0 = us.out0 + ks % kRows;
        own0 = uo.out0 + ko % kRows;
        shared_rows = us.nrows;
        own_rows = uo.nrows;
    }
    __device__ int count() const { return shared_n + own_n; }
    __device__ int64_t at(int i) const
    {
        return i < shared_n ? shared0 + static_cast<int64_t>(i) * shared_rows
                            : own0 + static_cast<int64_t>(i - shared_n) * own_rows;
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// A block per row, a piece per warp at a time, then a sum over the warps: for few
// rows, whose pieces may be many and are then all on their way at once.  With many
// rows the blocks do not fit at once, and rows have few pieces.  A call of 64 heads in
// a graph, in us, this form against a warp per row:
//   shared tokens   64 rows      256 rows     512 rows      1024 rows     2048 rows
//   203             18.2 / 18.0  19.2 / 19.5  19.2 / 19.4   23.4 / 21.0   32.5 / 24.7
//   8191            21.8 / 30.8  23.2 / 27.4  25.0 / 28.6   32.1 / 32.0   48.0 / 42.2
//   131072          48.4 / 72.6  62.0 / 74.6  109.3 / 116.6 195 / 197     400 / 395
// so up to kBlockRows rows, whatever the pieces.
__global__ void __launch_bounds__(256) combine_block_kernel(const Params p)
{
    constexpr int kWarps = 8;
    static_assert(2 * kMaxClusters <= 256, "a thread per piece");
    __shared__ float weight[256], top[kWarps], sums[kWarps];
    __shared__ float4 part[kWarps][kDc / 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int query = static_cast<int>(row / p.a.H);
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int ok = p.w.head[H_OK];
    const Token x = p.w.tok[query];
    if (!ok) return;
    const Pieces pc(p, row, x);
    const int n = pc.count();
    const float s = static_cast<int>(threadIdx.x) < n ? p.w.lse[pc.at(threadIdx.x)] : -INFINITY;
    float m = s;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    if (lane == 0) top[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = fmaxf(m, top[i]);
    const float ref = m == -INFINITY ? 0.f : m;      // (the maximum passes over NaN, the weights do not)
    const float f = ptx::ex2_approx(s - ref);
    weight[threadIdx.x] = f;
    float l = f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(kFull, l, d);
    if (lane == 0) sums[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) l += sums[i];
    float4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = warp; i < n; i += kWarps) {
        const float4 *from = reinterpret_cast<const float4 *>(p.w.o) + pc.at(i) * (kDc / 4) + lane;
        const float g = weight[i];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float4 y = __ldcg(from + 32 * v);
            acc[v].x = fmaf(y.x, g, acc[v].x);
            acc[v].y = fmaf(y.y, g, acc[v].y);
            acc[v].z = fmaf(y.z, g, acc[v].z);
            acc[v].w = fmaf(y.w, g, acc[v].w);
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) part[warp][32 * v + lane] = acc[v];
    __syncthreads();
    // columns 2 threadIdx.x and the next
    float2 y = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const float2 z = reinterpret_cast<const float2 *>(part[i])[threadIdx.x];
        y.x += z.x;
        y.y += z.y;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;      // (0: no token; NaN goes on)
    reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.a.o) + row * kDc)[threadIdx.x] = pack_bf16(y.x * inv, y.y * inv);
    if (threadIdx.x == 0) p.a.lse[row] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// A warp per row, for more rows than the GPU holds blocks of the other form.
__global__ void __launch_bounds__(256) combine_kernel(const Params p)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
    if (row >= p.a.Tq * p.a.H) return;
    const int query = static_cast<int>(row / p.a.H);
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int ok = p.w.head[H_OK];
    const Token x = p.w.tok[query];
    if (!ok) return;
    const Pieces pc(p, row, x);
    const int n = pc.count();
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, p.w.lse[pc.at(i)]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < n; base += 32) {
        const float mine = base + lane < n ? ptx::ex2_approx(p.w.lse[pc.at(base + lane)] - ref) : 0.f;
        const int here = min(32, n - base);
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
            const float f = __shfl_sync(kFull, mine, i);
            const float4 *from = reinterpret_cast<const float4 *>(p.w.o) + pc.at(base + i) * (kDc / 4) + lane;
            l += f;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float4 y = __ldcg(from + 32 * v);
                acc[v].x = fmaf(y.x, f, acc[v].x);
                acc[v].y = fmaf(y.y, f, acc[v].y);
                acc[v].z = fmaf(y.z, f, acc[v].z);
                acc[v].w = fmaf(y.w, f, acc[v].w);
            }
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;      // (0: no token; NaN goes on)
    uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.a.o) + row * kDc) + lane;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        out[32 * v] = make_uint2(pack_bf16(acc[v].x * inv, acc[v].y * inv), pack_bf16(acc[v].z * inv, acc[v].w * inv));
    if (lane == 0) p.a.lse[row] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// ---- host --------------------------------------------------------------------

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int64_t most_units(int64_t Tq, int H, int B, int G)
{
    return 2 * (Tq * H / kRows) + std::min<int64_t>(G, Tq) + std::min<int64_t>(B, Tq);
}

// Lays the workspace out from `base` (NULL to size it); the bytes it takes.
size_t lay_out(Work *w, uint8_t *base, int64_t Tq, int H, int B, int G, int clusters)
{
    const int64_t rows = Tq * H, units = most_units(Tq, H, B, G);
    // every row in one piece of its shared and one of its own tokens, and at
    // most one more piece per cluster
    const int64_t partial = 2 * rows + static_cast<int64_t>(clusters) * kRows;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *q = base + at;
        at += round_up(bytes, 256);
        return q;
    };
    w->head = reinterpret_cast<int *>(take(4 * H_INTS));
    w->tok = reinterpret_cast<Token *>(take(Tq * static_cast<int64_t>(sizeof(Token))));
    w->lists = reinterpret_cast<int *>(take(4 * (3 * static_cast<int64_t>(B) + 2 * static_cast<int64_t>(G))));
    w->start = reinterpret_cast<Start *>(take(clusters * static_cast<int64_t>(sizeof(Start))));
    w->unit = reinterpret_cast<Unit *>(take(units * static_cast<int64_t>(sizeof(Unit))));
    w->live = reinterpret_cast<Unit *>(take(units * static_cast<int64_t>(sizeof(Unit))));
    w->lse = reinterpret_cast<float *>(take(4 * partial));
    w->o = reinterpret_cast<float *>(take(4 * kDc * partial));
    return static_cast<size_t>(at);
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTA pairs: one per two SMs.  (The size must not depend on the device that a
// caller sizes its workspace on, so it is bounded rather than exact there.)
int clusters() { return std::max(1, std::min(kMaxClusters, num_sms() / 2)); }

}  // namespace

size_t prefix_mla_workspace_bytes(int64_t Tq, int H, int B, int G)
{
    Work w;
    return lay_out(&w, nullptr, Tq, H, B, G, kMaxClusters);
}

int run_prefix_mla(const PrefixMlaArgs &a, cudaStream_t s)
{
    Params p{};
    p.a = a;
    p.clusters = clusters();
    lay_out(&p.w, static_cast<uint8_t *>(a.workspace), a.Tq, a.H, a.B, a.G, kMaxClusters);
    p.box = std::min(a.page_size, 64);
    while (1 << p.box_log < p.box) ++p.box_log;
    while (1 << p.page_log < a.page_size) ++p.page_log;
    p.c_scale = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.wait_limit_ns = get_wait_limit_ns();
    p.wait_tries = p.wait_limit_ns >= 10000000u ? 1000 : 0;
    p.wait_nap_ns = static_cast<uint32_t>(std::min<uint64_t>(p.wait_limit_ns, 1000));
    const int64_t rows = a.Tq * a.H;
    CUtensorMap mq, mkv;
    if (rows > 0) {
        int rc = encode_bf16_tmap(&mq, a.q, kDc, static_cast<uint64_t>(rows), kCtaRows);
        if (rc) return rc;
        rc = encode_bf16_pages_tmap(&mkv, a.kv, kDc, a.page_size, a.n_pages, a.kv_page_stride, p.box);
        if (rc) return rc;
        KPOOL_CUDA_CHECK(
            cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
    }
    KPOOL_CUDA_CHECK(cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmem));
    // a small batch takes a small block, whose barriers and scans are shorter (2 us of a 22 us call)
    const int plan_threads = std::max({static_cast<int64_t>(a.B), static_cast<int64_t>(a.G), a.Tq}) <= 256 ? 256 : kPlanThreads;
    int64_t list_bytes = 4 * (4 * static_cast<int64_t>(a.B) + 3 * static_cast<int64_t>(a.G) + 2);
    p.plan_lists = list_bytes <= kPlanListBytes;
    if (!p.plan_lists) list_bytes = 0;
    constexpr int64_t kUnitBytes = sizeof(Unit);
    p.plan_units = static_cast<int>(std::min(most_units(a.Tq, a.H, a.B, a.G), (kPlanSmem - list_bytes) / kUnitBytes));
    const int plan_smem = static_cast<int>(p.plan_units * kUnitBytes + list_bytes);
    KPOOL_CUDA_CHECK(launch_after(plan_kernel, 1, plan_threads, plan_smem, s, p));
    if (rows == 0) return KPOOL_OK;
    KPOOL_CUDA_CHECK(launch_after(attend_kernel, 2 * p.clusters, kThreads, kSmemBytes, s, mq, mkv, p));
    if (rows <= kBlockRows)
        KPOOL_CUDA_CHECK(launch_after(combine_block_kernel, static_cast<int>(rows), 256, 0, s, p));
    else
        KPOOL_CUDA_CHECK(launch_after(combine_kernel, static_cast<int>((rows + 7) / 8), 256, 0, s, p));
    return KPOOL_OK;
}

}  // namespace kpool

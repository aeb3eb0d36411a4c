// Sparse attention of a chunk of new tokens over a paged latent cache: the
// absorbed NoPE form of kpool_mla.cu, whose latent rows are read through the
// sequences' page tables.  For query row t, at position tau of its sequence,
// and head h, over the tokens J(t) of its selected pools and its causal tail:
//
//   s_j = scale * q[t, h, :] . c[j, :]
//   o[t, h, :] = sum_j softmax_j(s) c[j, :],   lse[t, h] = ln sum_j exp(s_j)
//
// Design (one persistent CTA per SM, 24 warps; a unit is a row, or a run of a row's
// blocks where rows are few; units are handed out by an atomic counter).  Per block of
// 80 listed tokens C [80 x 512], in tensor memory:
//   S    [64 heads x 80]  = Q . C^T        (M = 64; A, B K-major)
//   O^T  [512 x 64 heads] += C^T . P^T     (four parts of M = 128; A MN-major, B K-major)
// The rows go through a ring of seven slots of 128 columns, of which a block takes four:
// the output's MMAs free them in order, and three quarters of the next block land, and
// its scores are begun, while this one's softmax runs (S is there twice).
//   warp 0       control: units, and per block a record with the places of its rows
//   warp 1       MMA issuer (the loop in all lanes, one issues)
//   warp 2       Q (TMA), ahead into L2
//   warps 4-11   softmax: four warps have the first 40 tokens of a block, four the
//                others; four threads share a head's 40 scores
//   warps 12-15  output, while the next unit's first scores run
//   warps 16-23  loaders: 16-byte cp.async, all of them on each quarter, up to three
//                quarters in flight
// One reference maximum per head, raised (and O^T rescaled) only when a block's
// scores exceed it by more than 8 in the base-2 exponent, so P <= 256; P goes to
// shared memory in BF16 (the MMA's operand type: 2^-8 of each at most), sums and
// statistics are FP32.
//
// What bounds it: 4 * 64 * 512 FLOP and 1 KB gathered, mostly from L2, a (row, token).
// 8192 rows of 2051 tokens take 3.16 ms: 697 TFLOP/s, 5.4 TB/s (1.15 ms at the rate of a
// library product).  The tensor pipe is 43% busy, shared memory's operands 46%: a block's
// chain (its last quarter lands, scores, softmax, first quarter of the output) is longer
// than its MMAs, and the next block's rows can only be three quarters there, next to the
// 64 KB of Q.  Steps: 64-token blocks, two in flight, four softmax warps 4.40 ms (the
// MMAs fell behind one another's latencies); divisions by multiplication in control 4.24;
// 128-token blocks, one in flight 3.70; the ring of 80-token blocks 3.73, but 128 decode
// steps 99 -> 87 us; all loader warps on each quarter 3.49 and 81 us; rolled issue loops
// 3.38; one look for all quarters that have landed 3.23; whole blocks' output MMAs
// unrolled 3.16.  Slower: the scores' loops unrolled (3.53), the MMAs' operands made uniform
// by a shuffle (3.73).
//
// Where rows are few (half the SMs or less), a row's blocks are cut into even runs, one
// for each CTA; FP32 outputs of the runs go to the workspace with their log-sums, and a
// second kernel joins them (and the CTAs' status words, so that none has to be cleared
// in front of the call: a launch less).  Otherwise a first kernel clears the counter and
// the status.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "kpool_internal.h"
#include "kpool_mla_rows.cuh"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kH = 64;                  // heads
constexpr int kDc = 512;                // latent width
constexpr int kBT = 80;                 // listed tokens per block
constexpr int kThreads = 768;
constexpr int kSoftWarps = 8;           // warps 4..11
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kOutWarp0 = 12, kOutWarps = 4;
// register split (setmaxnreg): 768 threads x 80 at launch
constexpr int kRegsSoftmax = 104, kRegsControl = 80, kRegsOther = 64;
static_assert(kSoftThreads * kRegsSoftmax + 128 * kRegsControl + (kThreads - kSoftThreads - 128) * kRegsOther <= kThreads * 80,
              "register split above the launch's registers");
constexpr int kLoaderWarp0 = 16, kLoaderWarps = 8;
constexpr int kChunk = kBT * 128;       // 64 latent columns of a block
constexpr int kQuarters = 4;            // 128 columns each
constexpr int kRing = 7;                // slots of a quarter of a block
constexpr int kSlot = 2 * kChunk;
constexpr int kInfoSlots = 4;
constexpr float kRescale = 8.f;         // headroom of the reference maximum (log2)
constexpr int kMaxSplit = 32;           // runs of a row
constexpr int kMaxSms = 160;            // that a workspace has room for
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kTmemCols = 512;          // O^T: 0..255, S: 256..335 and 336..415
constexpr int kTmemS = 256;

// shared memory (from a 1024-byte aligned base)
constexpr int kOffQ = 0;                               // 8 chunks [64 heads x 64 columns]
constexpr int kOffC = kOffQ + 8 * 8192;
constexpr int kOffP = kOffC + kRing * kSlot;           // [64 heads x 64 tokens], and 16 tokens
constexpr int kOffInv = kOffP + 2 * 8192;              // 1 / sums of a unit [2][64]
constexpr int kOffScale = kOffInv + 2 * kH * 4;        // rescale factors [64]
constexpr int kOffTop = kOffScale + kH * 4;            // maxima, sums of the halves [2][64]
constexpr int kOffInfo = kOffTop + 2 * kH * 4;
constexpr int kOffAt = kOffInfo + kInfoSlots * 32;     // places of the rows [kInfoSlots][80] int64
constexpr int kOffBar = kOffAt + kInfoSlots * kBT * 8;
enum {
    BQ_FULL = 0, BQ_EMPTY, BC_FULL, BC_EMPTY = BC_FULL + kRing, BS_FULL = BC_EMPTY + kRing, BP_FULL, BO_FULL,
    BO_EMPTY, BL_FULL, BL_EMPTY = BL_FULL + 2, BI_FULL = BL_EMPTY + 2, BI_EMPTY = BI_FULL + kInfoSlots,
    BDRAIN = BI_EMPTY + kInfoSlots, NBARS
};
constexpr int kOffMisc = kOffBar + NBARS * 8;          // [0] tmem base, [1] abort flag
constexpr int kSmemBytes = kOffMisc + 16 + 1024;       // and alignment slack
static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");

// n / d for 0 <= n < 2^31, d >= 2: with 2^(s-1) < d <= 2^s and mul = floor(2^(31+s) / d) + 1,
// mul * d exceeds 2^(31+s) by at most 2^s, so n * mul / 2^(31+s) exceeds n / d by less
// than 1 / d.  (The control warp divides for every listed token; the compiler's own
// divisions kept the loaders waiting: 2400 of 2900 cycles a block.)
struct Divisor {
    uint32_t mul, shift;        // mul = 0: d = 1
};

Divisor divisor(int d)
{
    if (d <= 1) return {0, 0};
    int s = 1;
    while (s < 31 && (int64_t(1) << s) < d) ++s;
    return {static_cast<uint32_t>((uint64_t(1) << (31 + s)) / static_cast<uint32_t>(d) + 1), static_cast<uint32_t>(s - 1)};
}

__device__ __forceinline__ int divide(int n, const Divisor &d)
{
    return d.mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), d.mul) >> d.shift) : n;
}

// workspace: header (ints: unit counter, status, each CTA's status where rows are cut),
// outputs and log-sums of the runs
constexpr int kHeadInts = 256, kHeadCtas = 64;
static_assert(kHeadCtas + kMaxSms <= kHeadInts, "a status word for each CTA");

struct Params {
    PagedMlaArgs a;
    Divisor by_pool, by_page;
    float c_scale;              // softmax scale * log2(e)
    int split;                  // runs of a row (1: rows are whole)
    int *ws;                    // header
    float *part_lse;            // [Tq * split, 64], base 2
    float *part_o;              // [Tq * split, 64, 512]
    uint64_t wait_limit_ns;
};

// What lists the tokens of one row.
struct PagedRow {
    const int32_t *table;       // its sequence's pages (NULL: no such sequence)
    int len;                    // tokens of the sequence, cut to its table's room
    int t, n_slots, n_pooled, tau, pool_lo, pool_hi;
    bool bad;                   // a sequence or length out of range
};

// Does row t belong to a sequence of the batch?  Others are left as they were.
__device__ __forceinline__ bool in_batch(const PagedMlaArgs &p, int t) { return t >= p.cu_q[0] && t < p.cu_q[p.B]; }

__device__ __forceinline__ PagedRow paged_row(const PagedMlaArgs &p, int t, int lane)
{
    PagedRow m{};
    const int b = doc_of_row(p.cu_q, p.B, t, lane);
    const int id = p.seq_ids != nullptr ? p.seq_ids[b] : b;
    m.t = t;
    m.bad = id < 0 || id >= p.n_rows;
    if (!m.bad) {
        const int room = p.max_pages * p.page_size, len = p.seq_lens[id];
        m.table = p.page_table + static_cast<int64_t>(id) * p.max_pages;
        m.len = max(0, min(len, room));
        m.bad = len != m.len;
    }
    m.pool_lo = p.cu_pools[b];
    m.pool_hi = p.cu_pools[b + 1];
    const int64_t tau = static_cast<int64_t>(p.q_pos[b]) + t - p.cu_q[b];
    m.bad |= tau < 0 || tau >= m.len;
    m.tau = static_cast<int>(max(int64_t(-1), min(tau, static_cast<int64_t>(m.len) - 1)));
    const int nc = min((m.tau + 1) / p.kpool, m.pool_hi - m.pool_lo);
    m.n_pooled = max(0, min(nc, p.Kp)) * p.kpool;
    m.n_slots = m.n_pooled + (p.tail ? (m.tau + 1) % p.kpool : 0);
    return m;
}

// The pool that slot j of the row is in (-1: none, or the tail).
__device__ __forceinline__ int pool_of(const Params &p, const PagedRow &m, int j)
{
    return j < m.n_pooled ? p.a.pool_idx[static_cast<int64_t>(m.t) * p.a.Kp + divide(j, p.by_pool)] : -1;
}

// Where slot j of the row, in pool g, lies in the pages, in elements (-1: no token there).
__device__ __forceinline__ int64_t paged_at(const Params &p, const PagedRow &m, int j, int g, bool &bad)
{
    if (j >= m.n_slots) return -1;
    int64_t v;
    if (j < m.n_pooled) {
        if (g < m.pool_lo || g >= m.pool_hi) return -1;
        v = static_cast<int64_t>(g - m.pool_lo) * p.a.kpool + (j - divide(j, p.by_pool) * p.a.kpool);
    } else {
        v = m.tau + 1 - (m.n_slots - j);
    }
    if (v >= m.len) {
        bad = true;
        return -1;
    }
    const int page = divide(static_cast<int>(v), p.by_page);
    const int id = m.table[page];
    if (id < 0 || id >= p.a.n_pages) {
        bad = true;
        return -1;
    }
    return id * p.a.kv_page_stride + static_cast<int64_t>(static_cast<int>(v) - page * p.a.page_size) * kDc;
}

// One block of a unit.
struct BInfo {
    int unit, b, nb, ksteps;    // b-th of the unit's nb blocks
    uint32_t mask[3], pad;      // bit r of mask[r / 32]: listed token r is valid
};
static_assert(sizeof(BInfo) == 32, "BInfo slot");

__device__ __forceinline__ void prefetch_l2(const void *from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// 16 lanes x 256 bits over 40 columns: for the columns 8 j + 2 (t % 4) and the next,
// registers 4 j .. 4 j + 3 are (lane t / 4, both), (lane t / 4 + 8, both).
__device__ __forceinline__ void tmem_ld_40(uint32_t taddr, uint32_t (&r)[20])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%20];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%16,%17,%18,%19}, [%21];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
          "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]),
          "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}

// All but the thread's last N groups of copies have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void st_shared(uint32_t saddr, uint32_t v)
{
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_mla_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t sQ = sbase + kOffQ, sC = sbase + kOffC, sP = sbase + kOffP;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    BInfo *info = reinterpret_cast<BInfo *>(smem + kOffInfo);
    int64_t *ats = reinterpret_cast<int64_t *>(smem + kOffAt);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    int *status = p.split > 1 ? p.ws + kHeadCtas + blockIdx.x : p.ws + 1;

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar(BQ_FULL), 1);
        ptx::mbar_init(bar(BQ_EMPTY), 1);
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(bar(BC_FULL + i), kLoaderWarps);
            ptx::mbar_init(bar(BC_EMPTY + i), 1);
        }
        ptx::mbar_init(bar(BS_FULL), 1);
        ptx::mbar_init(bar(BP_FULL), kSoftWarps);
        ptx::mbar_init(bar(BO_FULL), 1);
        ptx::mbar_init(bar(BO_EMPTY), kOutWarps);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(BL_FULL + i), 4);       // the softmax warps of the first half
            ptx::mbar_init(bar(BL_EMPTY + i), kOutWarps);
        }
        ptx::mbar_init(bar(BDRAIN), 1);
        for (int i = 0; i < kInfoSlots; ++i) {
            ptx::mbar_init(bar(BI_FULL + i), 1);
            ptx::mbar_init(bar(BI_EMPTY + i), 2 + kSoftWarps + kOutWarps + kLoaderWarps);
        }
        misc[1] = 0u;
        if (p.split > 1) *status = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&misc[0]), kTmemCols);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc[0];
    const Sync sy{reinterpret_cast<volatile uint32_t *>(&misc[1]), status, p.wait_limit_ns, p.wait_limit_ns < kPollBelowNs};
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();        // the cleared counter and status (whole rows)

    // the block records, one after another, for every role but the loaders
    auto next_info = [&](int g, BInfo &in) {
        const int is = g % kInfoSlots;
        if (!wait_bar_warp(bar(BI_FULL + is), (g / kInfoSlots) & 1, sy)) return false;
        in = info[is];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BI_EMPTY + is));
        return in.unit >= 0;
    };

    if (warp < 4) {
    ptx::setmaxnreg_dec<kRegsControl>();
    if (warp == 0) {
        // ---------------- control: units and their blocks ----------------
        const int units = static_cast<int>(p.a.Tq) * p.split;
        bool ok = true, bad = false;
        int g = 0, run = blockIdx.x;    // blocks published
        while (ok) {
            int u = -1;
            if (p.split > 1) {
                u = run;                // a CTA for each
                run = -1;
            } else {
                if (lane == 0 && !*sy.abort_flag) u = atomicAdd(p.ws, 1);
                u = __shfl_sync(kFull, u, 0);
            }
            if (u < 0 || u >= units) break;
            const int t = u / p.split;
            if (!in_batch(p.a, t)) continue;
            const PagedRow m = paged_row(p.a, t, lane);
            bad |= m.bad;
            // (a row may list up to 2^31 - 1 tokens: rounded up without a sign)
            const int all = static_cast<int>((static_cast<uint32_t>(m.n_slots) + kBT - 1) / kBT);
            const int per = (all + p.split - 1) / p.split;
            const int b0 = (u - t * p.split) * per, nb = max(0, min(all - b0, per));
            if (nb == 0) {
                // nothing listed: what the output warps would write
                float *l = p.split > 1 ? p.part_lse + static_cast<int64_t>(u) * kH : p.a.lse + static_cast<int64_t>(t) * kH;
                l[lane] = l[32 + lane] = -INFINITY;
                if (p.split == 1) {
                    uint4 *o = static_cast<uint4 *>(p.a.o) + static_cast<int64_t>(t) * (kH * kDc / 8);
                    for (int i = lane; i < kH * kDc / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            for (int b = 0; b < nb; ++b, ++g) {
                // lane's tokens 32 i + lane of the block
                const int end = min(kBT, m.n_slots - (b0 + b) * kBT), j0 = (b0 + b) * kBT + lane;
                int pool[3];
                int64_t at[3];
                uint32_t mask[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) pool[i] = 32 * i + lane < end ? pool_of(p, m, j0 + 32 * i) : -1;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    at[i] = 32 * i + lane < end ? paged_at(p, m, j0 + 32 * i, pool[i], bad) : -1;
                    mask[i] = __ballot_sync(kFull, at[i] >= 0);
                }
                const int is = g % kInfoSlots;
                ok = wait_bar_warp(bar(BI_EMPTY + is), ((g / kInfoSlots) & 1) ^ 1, sy);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (32 * i + lane < kBT) ats[is * kBT + 32 * i + lane] = at[i];
                if (lane == 0) {
                    info[is].unit = u;
                    info[is].b = b;
                    info[is].nb = nb;
                    info[is].ksteps = (end + 15) / 16;
#pragma unroll
                    for (int i = 0; i < 3; ++i) info[is].mask[i] = mask[i];
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(BI_FULL + is));
            }
        }
        // end of the block stream for every consumer
        const int is = g % kInfoSlots;
        if (ok && wait_bar_warp(bar(BI_EMPTY + is), ((g / kInfoSlots) & 1) ^ 1, sy) && lane == 0) {
            info[is].unit = -1;
            ptx::mbar_arrive(bar(BI_FULL + is));
        }
        if (__any_sync(kFull, bad) && lane == 0) atomicOr(sy.status, KPOOL_STATUS_BAD_PAGE);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t idesc_s = ptx::make_idesc(1u, 64, kBT);
        constexpr uint32_t idesc_o = ptx::make_idesc(1u, 128, 64) | ptx::kIdescAMajorMN;
        const bool one = ptx::elect_one();
        uint32_t q_ph = 0, o_ph = 0;
        bool any = false;
        // a quarter of block g's scores
        auto scores = [&](int g, int sl) {
            ptx::tc_fence_after();
            if (one) {
                const uint32_t at = (static_cast<uint32_t>(g) * kQuarters + sl) % kRing;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t ad = ptx::smem_desc_sw128(sQ + (2 * sl + h) * 8192);
                    const uint64_t bd = ptx::smem_desc_sw128(sC + at * kSlot + h * kChunk);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_bf16(tmem + kTmemS + (g & 1) * kBT, ad + 2 * kk, bd + 2 * kk, idesc_s, (sl | h | kk) != 0);
                }
            }
            any = true;
        };
        auto landed = [&](int g, int sl, uint32_t &at) {
            const uint32_t n = static_cast<uint32_t>(g) * kQuarters + sl;
            at = bar(BC_FULL + n % kRing);
            return (n / kRing) & 1;
        };
        BInfo in, nx;
        bool more = next_info(0, in);
        int ahead = 0;                                     // quarters of this block's scores that are issued
        for (int g = 0; more; ++g) {
            uint32_t at;
            bool ok = in.b > 0 || wait_bar_warp(bar(BQ_FULL), q_ph, sy);
            if (in.b == 0) q_ph ^= 1;
            // (the scores of two blocks ago were read before their P was complete)
            // (rolled loops: unrolled, 8192 queries over 65536 tokens take 3.53 ms, so 3.15)
#pragma unroll 1
            for (int sl = ahead; sl < kQuarters && ok; ++sl) {
                const uint32_t ph = landed(g, sl, at);
                ok = wait_bar_warp(at, ph, sy);
                if (ok) scores(g, sl);
            }
            if (!ok) break;
            if (one) {
                ptx::mma_commit(bar(BS_FULL));
                if (in.b == in.nb - 1) ptx::mma_commit(bar(BQ_EMPTY));
            }
            // while the softmax works on them, the next block's scores as far as it has landed
            ahead = 0;
            const bool known = __shfl_sync(kFull, ptx::mbar_test(bar(BI_FULL + (g + 1) % kInfoSlots), ((g + 1) / kInfoSlots) & 1), 0);
            if (known) {
                more = next_info(g + 1, nx);
                // (quarters land in order: the last one says it of the others)
                int here = more && nx.b > 0 ? kQuarters - 1 : 0;
#pragma unroll 1
                for (; here > 0; --here) {
                    const uint32_t ph = landed(g + 1, here - 1, at);
                    if (__shfl_sync(kFull, ptx::mbar_test(at, ph), 0)) break;
                }
#pragma unroll 1
                for (; ahead < here; ++ahead) scores(g + 1, ahead);
            }
            ok = wait_bar_warp(bar(BP_FULL), g & 1, sy);
            if (in.b == 0) {
                ok = ok && wait_bar_warp(bar(BO_EMPTY), o_ph ^ 1, sy);
                o_ph ^= 1;
            }
            if (!ok) break;
            ptx::tc_fence_after();
            if (one) {
                const uint64_t bd = ptx::smem_desc_sw128(sP);
                for (int sl = 0; sl < kQuarters; ++sl) {
                    const uint32_t slot = (static_cast<uint32_t>(g) * kQuarters + sl) % kRing;
                    const uint64_t ad = ptx::smem_desc_mn_sw128(sC + slot * kSlot, kChunk);
                    auto step = [&](int kk) {
                        ptx::mma_bf16(tmem + sl * 64, ad + kk * 128, bd + (kk >> 2) * 512 + (kk & 3) * 2, idesc_o,
                                      in.b > 0 || kk > 0);
                    };
                    if (in.ksteps == kBT / 16) {           // (whole blocks unrolled: 3.23 -> 3.16 ms)
#pragma unroll
                        for (int kk = 0; kk < kBT / 16; ++kk) step(kk);
                    } else {
                        for (int kk = 0; kk < in.ksteps; ++kk) step(kk);
                    }
                    ptx::mma_commit(bar(BC_EMPTY + slot));
                }
                if (in.b == in.nb - 1) ptx::mma_commit(bar(BO_FULL));
            }
            if (!known) more = next_info(g + 1, nx);
            in = nx;
        }
        if (any) {
            if (one) ptx::mma_commit(bar(BDRAIN));
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar(BDRAIN), 0))
                if (ptx::globaltimer() - t0 > kTimeoutNs) break;
        }
    } else if (warp == 2) {
        // ---------------- Q ----------------
        if (lane == 0) ptx::tma_prefetch_desc(&tm_q);
        uint32_t q_ph = 0;
        bool issued = false;
        BInfo in;
        for (int g = 0; next_info(g, in); ++g) {
            if (in.b > 0) continue;
            const int t = in.unit / p.split;
            // (known some blocks ahead: into L2 meanwhile)
            if (lane == 0)
                prefetch_l2(static_cast<const uint16_t *>(p.a.q) + static_cast<int64_t>(t) * kH * kDc, kH * kDc * 2);
            if (!wait_bar_warp(bar(BQ_EMPTY), q_ph ^ 1, sy)) break;
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar(BQ_FULL), 8 * 8192);
            __syncwarp();
            if (lane < 8) ptx::tma_load_2d(sQ + lane * 8192, &tm_q, bar(BQ_FULL), 64 * lane, t * kH);
            issued = true;
            q_ph ^= 1;
        }
        // no load of Q may still be in flight when the CTA ends: a wait of its own,
        // bounded by the default limit and blind to the abort flag
        if (issued) {
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar(BQ_FULL), q_ph ^ 1))
                if (ptx::globaltimer() - t0 > kTimeoutNs) break;
        }
    }
    } else if (warp < kOutWarp0) {
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        // ---------------- softmax ----------------
        const int sub = warp & 3, half = (warp - 4) >> 2;
        const int h0 = 16 * sub + (lane >> 2);             // this thread's heads: h0 and h0 + 8
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * sub) << 16);
        const uint32_t row = sP + h0 * 128 + (lane & 3) * 4;
        float *inv = reinterpret_cast<float *>(smem + kOffInv), *factor = reinterpret_cast<float *>(smem + kOffScale);
        float *halves = reinterpret_cast<float *>(smem + kOffTop);
        float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
        int nu = 0;                                        // units so far
        // the warps meet once a block, and leave together
        for (int g = 0;; ++g) {
            BInfo in;
            in.unit = -1;
            bool ok = next_info(g, in) && wait_bar_warp(bar(BS_FULL), g & 1, sy);
            // this half's 40 validity bits, from its thread's first token on
            const uint32_t lo = (half ? in.mask[1] >> 8 | in.mask[2] << 24 : in.mask[0]) >> (2 * (lane & 3));
            const uint32_t hi = (half ? in.mask[2] >> 8 : in.mask[1]) >> (2 * (lane & 3));
            // v[k][2 j + e]: the score of token 40 half + 8 j + 2 (lane % 4) + e, base 2
            auto load = [&](float (&v)[2][10]) {
                uint32_t r[20];
                tmem_ld_40(lanes + kTmemS + (g & 1) * kBT + 40 * half, r);
#pragma unroll
                for (int j = 0; j < 5; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            v[k][2 * j + e] = (j < 4 ? lo >> (8 * j + e) : hi >> e) & 1u
                                                  ? __uint_as_float(r[4 * j + 2 * k + e]) * p.c_scale : -INFINITY;
            };
            float w[2][10];                                // 2^(score - m)
            bool over = false;
            if (ok) {
                ptx::tc_fence_after();
                load(w);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // (a head without tokens so far has m = -inf, and any score exceeds it)
                    const float ref = m[k] == -INFINITY ? 0.f : m[k], most = m[k] + kRescale;
#pragma unroll
                    for (int i = 0; i < 10; ++i) {
                        over |= w[k][i] > most;
                        w[k][i] = ptx::ex2_approx(w[k][i] - ref);
                    }
                }
            }
            if (ptx::named_bar_or(1, kSoftThreads, !ok || over || in.b == 0)) {
                // some warp leaves, a unit begins, or some head's reference rises
                if (ptx::named_bar_or(2, kSoftThreads, !ok)) break;
                load(w);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float top = w[k][0];
#pragma unroll
                    for (int i = 1; i < 10; ++i) top = fmaxf(top, w[k][i]);
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                    if ((lane & 3) == 0) halves[half * kH + h0 + 8 * k] = top;
                }
                ptx::named_bar_sync(2, kSoftThreads);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float t = fmaxf(halves[h0 + 8 * k], halves[kH + h0 + 8 * k]);
                    const float now = in.b == 0 || t > m[k] + kRescale ? t : m[k];
                    const float f = now == m[k] ? 1.f : ptx::ex2_approx(m[k] - now);
                    m[k] = now;
                    l[k] = in.b == 0 ? 0.f : l[k] * f;
                    if (half == 0 && (lane & 3) == 0) factor[h0 + 8 * k] = f;
                    const float ref = now == -INFINITY ? 0.f : now;
#pragma unroll
                    for (int i = 0; i < 10; ++i) w[k][i] = ptx::ex2_approx(w[k][i] - ref);
                }
                ptx::named_bar_sync(2, kSoftThreads);
                if (in.b > 0) {
                    // (the last block's output MMAs are done: this one's scores came behind them)
#pragma unroll 1
                    for (int c = 4 * half; c < 4 * half + 4; ++c) {
                        uint32_t x[32];
                        ptx::tmem_ld32(lanes + 32 * c, x);
                        ptx::tmem_ld_wait(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * factor[32 * (c & 1) + i]);
                        ptx::tmem_st32(lanes + 32 * c, x);
                    }
                    ptx::tmem_st_wait();
                    ptx::named_bar_sync(2, kSoftThreads);  // the factors have been read
                }
            }
            // (and have read P)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 5; ++j) {
                    const int piece = 5 * half + j;        // eight tokens
                    st_shared(row + (piece >> 3) * 8192 + k * 1024 + (((piece & 7) ^ (lane >> 2)) << 4),
                              pack_bf16(w[k][2 * j], w[k][2 * j + 1]));
                }
            ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BP_FULL));
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 10; ++i) l[k] += w[k][i];
            if (in.b == in.nb - 1) {
                ok = wait_bar_warp(bar(BL_EMPTY + (nu & 1)), ((nu >> 1) & 1) ^ 1, sy);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    l[k] += __shfl_xor_sync(kFull, l[k], 1);
                    l[k] += __shfl_xor_sync(kFull, l[k], 2);
                    if (half == 1 && (lane & 3) == 0) halves[h0 + 8 * k] = l[k];
                }
                if (ptx::named_bar_or(2, kSoftThreads, !ok)) break;
                if (half == 0) {
                    float *out = p.split > 1 ? p.part_lse + static_cast<int64_t>(in.unit) * kH
                                             : p.a.lse + static_cast<int64_t>(in.unit) * kH;
                    if ((lane & 3) == 0)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int h = h0 + 8 * k;
                            const float sum = l[k] + halves[h];
                            // (no listed token: 0; NaN goes on)
                            inv[(nu & 1) * kH + h] = sum != 0.f ? 1.f / sum : 0.f;
                            const float lse = sum != 0.f ? m[k] + log2f(sum) : -INFINITY;
                            out[h] = p.split > 1 ? lse : lse * 0.69314718055994531f;
                        }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(BL_FULL + (nu & 1)));
                }
                ++nu;
            }
        }
    } else if (warp < kLoaderWarp0) {
        ptx::setmaxnreg_dec<kRegsOther>();
        // ---------------- output ----------------
        const int sub = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * sub) << 16);
        int nu = 0;
        BInfo in;
        for (int g = 0; next_info(g, in); ++g) {
            if (in.b < in.nb - 1) continue;
            if (!wait_bar_warp(bar(BL_FULL + (nu & 1)), (nu >> 1) & 1, sy)) break;
            if (!wait_bar_warp(bar(BO_FULL), nu & 1, sy)) break;
            ptx::tc_fence_after();
            const float *inv = reinterpret_cast<const float *>(smem + kOffInv) + (nu & 1) * kH;
            const int64_t at = static_cast<int64_t>(in.unit) * kH * kDc + 32 * sub + lane;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                uint32_t x[32];
                ptx::tmem_ld32(lanes + 32 * c, x);
                ptx::tmem_ld_wait(x);
                if (c == 7) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(BO_EMPTY));
                }
                const int64_t to = at + (c >> 1) * 128 + static_cast<int64_t>(32 * (c & 1)) * kDc;
                if (p.split > 1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        p.part_o[to + i * kDc] = __uint_as_float(x[i]) * inv[32 * (c & 1) + i];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const __nv_bfloat16 b = __float2bfloat16_rn(__uint_as_float(x[i]) * inv[32 * (c & 1) + i]);
                        static_cast<uint16_t *>(p.a.o)[to + i * kDc] = *reinterpret_cast<const uint16_t *>(&b);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BL_EMPTY + (nu & 1)));
            ++nu;
        }
    } else {
        ptx::setmaxnreg_dec<kRegsOther>();
        // ---------------- loaders ----------------
        const int tid = threadIdx.x - 32 * kLoaderWarp0;
        const int k = tid & 15, r0 = tid >> 4;             // 16-byte piece of a quarter's 256 bytes; rows r0 + 16 i
        const char *kvb = static_cast<const char *>(p.a.kv) + k * 16;
        const uint32_t dst = sC + (k >> 3) * kChunk + r0 * 128 + (((k & 7) ^ (r0 & 7)) << 4);
        int64_t at[kBT / 16];
        uint32_t n = 0, done = 0;                          // quarters sent for, quarters landed
        bool known = false, end = false, ok = true;
        // has the phase completed?  Waits for it where nothing is in flight
        auto ready = [&](uint32_t b, uint32_t ph) -> bool {
            if (n != done) return __shfl_sync(kFull, ptx::mbar_test(b, ph), 0) != 0;
            ok = wait_bar_warp(b, ph, sy);
            return ok;
        };
        while (true) {
            bool sent = false;
            if (!end && n - done < 3) {
                const int g = n / kQuarters, is = g % kInfoSlots;
                if (!known && ready(bar(BI_FULL + is), (g / kInfoSlots) & 1)) {
                    end = info[is].unit < 0;
#pragma unroll
                    for (int i = 0; i < kBT / 16; ++i) at[i] = ats[is * kBT + r0 + 16 * i];
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(BI_EMPTY + is));
                    known = !end;
                }
                const uint32_t slot = n % kRing;
                if (known && ready(bar(BC_EMPTY + slot), ((n / kRing) & 1) ^ 1)) {
                    const int64_t column = (n % kQuarters) * 256;
#pragma unroll
                    for (int i = 0; i < kBT / 16; ++i)
                        ptx::cp_async16(dst + slot * kSlot + i * 2048, kvb + (at[i] >= 0 ? 2 * at[i] + column : 0),
                                        at[i] >= 0 ? 16u : 0u);
                    ptx::cp_async_commit();
                    known = ++n % kQuarters != 0;
                    sent = true;
                }
            }
            if (!ok) break;
            if (sent) continue;
            if (n == done) {
                if (end) break;
                continue;
            }
            if (n - done == 3) cp_async_wait<2>();
            else if (n - done == 2) cp_async_wait<1>();
            else cp_async_wait<0>();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BC_FULL + done % kRing));
            ++done;
        }
        ptx::cp_async_wait_all();
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// The status that cu_q gives: it has to be 0 .. Tq and non-decreasing.  One block.
__device__ __forceinline__ int status_of(const int32_t *cu_q, int B, int64_t Tq)
{
    bool bad = cu_q[0] != 0 || cu_q[B] != Tq;
    for (int i = threadIdx.x; i < B; i += blockDim.x) bad |= cu_q[i] > cu_q[i + 1];
    return __syncthreads_or(bad) ? KPOOL_STATUS_BAD_SEQLENS : 0;
}

// In front of whole rows: a cleared counter, and the status.
__global__ void __launch_bounds__(256) start_kernel(const int32_t *cu_q, int B, int64_t Tq, int *ws)
{
    ptx::grid_dependents_launch();
    const int status = status_of(cu_q, B, Tq);
    if (threadIdx.x < 2) ws[threadIdx.x] = threadIdx.x == 1 ? status : 0;
}

// Joins the runs of a (row, head), a warp each: sum of 2^(lse_s - max) o_s over that of
// 2^(lse_s - max).
__global__ void __launch_bounds__(128) join_kernel(const Params p)
{
    const int lane = threadIdx.x & 31;
    const int64_t r = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
    const int64_t t = r / kH, h = r % kH, u0 = t * p.split;
    ptx::grid_dependency_wait();
    if (blockIdx.x == 0) {
        int status = status_of(p.a.cu_q, p.a.B, p.a.Tq);
        for (int u = threadIdx.x; u < p.a.Tq * p.split; u += 128) status |= p.ws[kHeadCtas + u];
        status |= __syncthreads_or(status & KPOOL_STATUS_BAD_PAGE) ? KPOOL_STATUS_BAD_PAGE : 0;
        status |= __syncthreads_or(status & KPOOL_STATUS_TIMEOUT) ? KPOOL_STATUS_TIMEOUT : 0;
        if (threadIdx.x == 0) p.ws[1] = status;
    }
    if (!in_batch(p.a, static_cast<int>(t))) return;
    const float mine = lane < p.split ? p.part_lse[(u0 + lane) * kH + h] : -INFINITY;
    float top = mine;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    float w = ptx::ex2_approx(mine - (top == -INFINITY ? 0.f : top)), sum = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    const float inv = sum != 0.f ? 1.f / sum : 0.f;        // (0: no token; NaN goes on)
    float4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < p.split; ++s) {
        const float f = __shfl_sync(kFull, w, s) * inv;
        if (f == 0.f) continue;                            // (an empty run has written no row)
        const float4 *from = reinterpret_cast<const float4 *>(p.part_o + ((u0 + s) * kH + h) * kDc) + lane;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float4 y = from[32 * v];
            acc[v].x = fmaf(y.x, f, acc[v].x);
            acc[v].y = fmaf(y.y, f, acc[v].y);
            acc[v].z = fmaf(y.z, f, acc[v].z);
            acc[v].w = fmaf(y.w, f, acc[v].w);
        }
    }
    uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.a.o) + r * kDc) + lane;
#pragma unroll
    for (int v = 0; v < 4; ++v) out[32 * v] = make_uint2(pack_bf16(acc[v].x, acc[v].y), pack_bf16(acc[v].z, acc[v].w));
    if (lane == 0) p.a.lse[r] = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
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

// Runs of a row, where rows are at most half of the SMs: as many as fill them.  More rows
// are whole, one to a CTA at a time, so that a last round that is not full costs a whole
// one (76 rows 52 us, 77 to 152 73 to 79, 153 133).  (2049
// tokens a row, us a call in a graph, cut and whole: 1 row 22 and 69, 8 rows 29 and 70,
// 38 rows 37 and 73, 76 rows, in two runs each, 55 and 77.)
int runs(int64_t Tq, int Kp, int kpool, int sms)
{
    if (Tq == 0 || 2 * Tq > sms) return 1;
    const int64_t blocks = (static_cast<int64_t>(Kp) * kpool + kpool - 1 + kBT - 1) / kBT;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({sms / Tq, blocks, kMaxSplit})));
}

}  // namespace

// (The size must not depend on the device that a caller sizes its workspace on, so the
// number of SMs is bounded there.)
size_t paged_mla_workspace_need(int64_t Tq, int Kp, int kpool)
{
    const int n = runs(Tq, Kp, kpool, kMaxSms);
    return kHeadInts * 4 + (n > 1 ? static_cast<size_t>(Tq) * n * kH * (kDc + 1) * 4 : 0);
}

// (Few rows need more than many, which are not cut: the most that Tq rows or fewer need, so
// that a workspace for the largest batch serves the smaller ones.)
size_t paged_mla_workspace_bytes(int64_t Tq, int Kp, int kpool)
{
    size_t most = paged_mla_workspace_need(Tq, Kp, kpool);
    for (int64_t t = std::min<int64_t>(Tq, kMaxSms / 2); t > 0; --t)
        most = std::max(most, paged_mla_workspace_need(t, Kp, kpool));
    return most;
}

int run_paged_mla(const PagedMlaArgs &a, cudaStream_t s)
{
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    Params p{};
    p.a = a;
    p.c_scale = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    const int sms = std::min(num_sms(), kMaxSms);
    p.by_pool = divisor(a.kpool);
    p.by_page = divisor(a.page_size);
    p.split = runs(a.Tq, a.Kp, a.kpool, sms);
    p.ws = reinterpret_cast<int *>(ws);
    p.part_o = reinterpret_cast<float *>(ws + kHeadInts * 4);
    p.part_lse = p.part_o + a.Tq * p.split * kH * kDc;
    p.wait_limit_ns = get_wait_limit_ns();
    CUtensorMap mq;
    if (a.Tq > 0) {
        const int rc = encode_bf16_tmap(&mq, a.q, kDc, static_cast<uint64_t>(a.Tq) * kH, kH);
        if (rc) return rc;
        KPOOL_CUDA_CHECK(
            cudaFuncSetAttribute(paged_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
    }
    if (p.split > 1) {
        paged_mla_kernel<<<static_cast<unsigned>(a.Tq * p.split), kThreads, kSmemBytes, s>>>(mq, p);
        KPOOL_CUDA_CHECK(cudaGetLastError());
        KPOOL_CUDA_CHECK(launch_after(join_kernel, static_cast<int>(a.Tq * (kH / 4)), 128, 0, s, p));
        return KPOOL_OK;
    }
    start_kernel<<<1, 256, 0, s>>>(a.cu_q, a.B, a.Tq, p.ws);
    KPOOL_CUDA_CHECK(cudaGetLastError());
    if (a.Tq > 0)
        KPOOL_CUDA_CHECK(launch_after(paged_mla_kernel, static_cast<int>(std::min<int64_t>(sms, a.Tq)), kThreads,
                                      kSmemBytes, s, mq, p));
    return KPOOL_OK;
}

}  // namespace kpool

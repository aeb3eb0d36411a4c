// Which tokens a query row of the sparse attention lists (an explicit list, or
// selected pools and a causal tail), and the bounded waits of its kernels.
#pragma once
#include <cstdint>

#include "kpool_internal.h"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

struct RowLists {
    const int32_t *tok;         // [T, W] or NULL (pool mode)
    const int32_t *pool_idx;    // [T, Kp] (pool mode)
    const int32_t *cu_seqlens, *q_pos, *cu_k, *cu_pools;
    int n_docs;
    int T, Tk, W, kp, Kp, tail;
};

RowLists row_lists(const SparseMlaArgs &a)
{
    RowLists l{};
    l.tok = a.tok_idx;
    l.pool_idx = a.pool_idx;
    l.cu_seqlens = a.cu_seqlens;
    l.q_pos = a.q_pos;
    l.cu_k = a.cu_k;
    l.cu_pools = a.cu_pools;
    l.n_docs = a.n_docs;
    l.T = static_cast<int>(a.T);
    l.Tk = static_cast<int>(a.Tk);
    l.W = a.W;
    l.kp = a.kpool;
    l.Kp = a.Kp;
    l.tail = a.tail;
    return l;
}

// What lists the tokens of one row.
struct RowMsg {
    int64_t key0;               // first key token of the row's document
    int t, n_slots, tau, pool_lo, pool_hi, n_sel, n_tail, pad;
};
static_assert(sizeof(RowMsg) <= 48, "RowMsg slot");

// Limits below this are waited for by probes that do not suspend the thread: a suspended
// one may see nothing until its barrier completes, so that a limit of 1 ns was not told of
// by calls whose waits are short (backward pass, 1 to 77 rows).
constexpr uint64_t kPollBelowNs = 1000000ull;

struct Sync {
    volatile uint32_t *abort_flag;
    int *status;
    uint64_t limit_ns;
    bool poll = false;          // probes do not suspend the thread
};

__device__ __forceinline__ bool probe_bar(uint32_t bar, uint32_t parity, const Sync &sy)
{
    return sy.poll ? ptx::mbar_test(bar, parity) : ptx::mbar_try_wait(bar, parity);
}

// Bounded mbarrier wait (completion, then the CTA abort flag, then a timer
// that raises the flag and KPOOL_STATUS_TIMEOUT).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Sync &sy)
{
    if (probe_bar(bar, parity, sy)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        if (probe_bar(bar, parity, sy)) return true;
        if (*sy.abort_flag) return false;
        if (ptx::globaltimer() - t0 > sy.limit_ns) {
            *sy.abort_flag = 1u;
            atomicOr(sy.status, KPOOL_STATUS_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, const Sync &sy)
{
    const bool ok = wait_bar(bar, parity, sy);
    return __all_sync(kFull, ok);
}

// Document of row t (largest d with cu[d] <= t, 0 if there is none), one warp
// probing 32 evenly spaced offsets per round.  Every lane gets the answer.
__device__ __forceinline__ int doc_of_row(const int32_t *cu, int n_docs, int t, int lane)
{
    int lo = 0, hi = n_docs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int idx = lo + lane * step;
        const bool le = idx < hi && cu[idx] <= t;
        const unsigned m = __ballot_sync(kFull, le);
        if (m == 0) break;
        const int nlo = lo + (31 - __clz(m)) * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo;
}

// Key token of slot j of the row (-1: none).  Pool mode lists the selected
// pools' tokens in order, then the tail (the expansion of the selection).
__device__ __forceinline__ int token_of(const RowLists &p, const RowMsg &m, int j)
{
    if (j >= m.n_slots) return -1;
    if (p.tok != nullptr) {
        const int v = __ldg(p.tok + static_cast<int64_t>(m.t) * p.W + j);
        return (v >= 0 && v < p.Tk) ? v : -1;
    }
    const int npt = m.n_sel * p.kp;
    int64_t v = -1;
    if (j < npt) {
        const int e = j / p.kp;
        const int g = __ldg(p.pool_idx + static_cast<int64_t>(m.t) * p.Kp + e);
        if (g >= m.pool_lo && g < m.pool_hi)
            v = m.key0 + static_cast<int64_t>(g - m.pool_lo) * p.kp + (j - e * p.kp);
    } else {
        v = m.key0 + m.tau - m.n_tail + 1 + (j - npt);
    }
    return (v >= 0 && v < p.Tk) ? static_cast<int>(v) : -1;
}

// Row t's message, from one warp; every lane gets it.
__device__ __forceinline__ RowMsg row_msg(const RowLists &p, int t, int lane)
{
    RowMsg m{};
    m.t = t;
    if (p.tok != nullptr) {
        // extent of the listed tokens: one past the last valid entry
        int last = -1;
        const int32_t *row = p.tok + static_cast<int64_t>(m.t) * p.W;
        for (int j = lane; j < p.W; j += 32) {
            const int v = __ldg(row + j);
            if (v >= 0 && v < p.Tk) last = j;
        }
        m.n_slots = __reduce_max_sync(kFull, last + 1);
        return m;
    }
    int64_t doc_start = 0;
    m.key0 = 0;
    int pos0 = 0;
    m.pool_lo = 0;
    m.pool_hi = p.Tk / p.kp;
    if (p.cu_seqlens != nullptr) {
        const int d = doc_of_row(p.cu_seqlens, p.n_docs, m.t, lane);
        doc_start = p.cu_seqlens[d];
        m.key0 = p.cu_k != nullptr ? p.cu_k[d] : doc_start;
        pos0 = p.q_pos != nullptr ? p.q_pos[d] : 0;
        m.pool_lo = p.cu_pools[d];
        m.pool_hi = p.cu_pools[d + 1];
    }
    m.tau = pos0 + static_cast<int>(m.t - doc_start);
    const int nc = min((m.tau + 1) / p.kp, m.pool_hi - m.pool_lo);
    m.n_sel = max(0, min(nc, p.Kp));
    m.n_tail = p.tail ? (m.tau + 1) % p.kp : 0;
    m.n_slots = m.n_sel * p.kp + m.n_tail;
    return m;
}

}  // namespace
}  // namespace kpool

// Sparse attention of a chunk of new tokens over a paged latent cache: the
// absorbed NoPE form of kpool_mla.cu, whose latent rows are read through the
// sequences' page tables.  For query row t, at position tau of its sequence,
// and head h, over the tokens J(t) of its selected pools and its causal tail:
//
//   s_j = scale * q[t, h, :] . c[j, :]
//   o[t, h, :] = sum_j softmax_j(s) c[j, :],   lse[t, h] = ln sum_j exp(s_j)
//
// First form: a block per row, a warp per eight heads, lanes over the columns,
// running maximum and sum.
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

struct Params {
    PagedMlaArgs a;
    int *status;
};

// What lists the tokens of one row.
struct PagedRow {
    const int32_t *table;       // its sequence's pages (NULL: no such sequence)
    int len;                    // tokens of the sequence, cut to its table's room
    int t, n_slots, tau, pool_lo, pool_hi, n_sel, n_tail;
    bool bad;                   // a sequence or length out of range
};

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
    m.n_sel = max(0, min(nc, p.Kp));
    m.n_tail = p.tail ? (m.tau + 1) % p.kpool : 0;
    m.n_slots = m.n_sel * p.kpool + m.n_tail;
    return m;
}

// Where slot j of the row lies in the pages, in elements (-1: no token there).
__device__ __forceinline__ int64_t paged_at(const PagedMlaArgs &p, const PagedRow &m, int j, bool &bad)
{
    if (j >= m.n_slots) return -1;
    const int npt = m.n_sel * p.kpool;
    int64_t v;
    if (j < npt) {
        const int e = j / p.kpool;
        const int g = __ldg(p.pool_idx + static_cast<int64_t>(m.t) * p.Kp + e);
        if (g < m.pool_lo || g >= m.pool_hi) return -1;
        v = static_cast<int64_t>(g - m.pool_lo) * p.kpool + (j - e * p.kpool);
    } else {
        v = m.tau - m.n_tail + 1 + (j - npt);
    }
    if (v >= m.len) {
        bad = true;
        return -1;
    }
    const int page = static_cast<int>(v) / p.page_size;
    const int id = m.table[page];
    if (id < 0 || id >= p.n_pages) {
        bad = true;
        return -1;
    }
    return id * p.kv_page_stride + static_cast<int64_t>(static_cast<int>(v) - page * p.page_size) * kDc;
}

__device__ __forceinline__ void load16(const uint16_t *row, int lane, float (&v)[16])
{
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + 256 * half + 8 * lane);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * half + 2 * i] = __uint_as_float(w[i] << 16);
            v[8 * half + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__global__ void __launch_bounds__(256) paged_mla_kernel(const Params p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    const PagedRow m = paged_row(p.a, t, lane);
    const int64_t base = (static_cast<int64_t>(t) * kH + 8 * warp) * kDc;
    float o[8][16], top[8], sum[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        top[h] = -INFINITY;
        sum[h] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[h][i] = 0.f;
    }
    bool bad = m.bad;
    for (int j = 0; j < m.n_slots; ++j) {
        const int64_t at = paged_at(p.a, m, j, bad);
        if (at < 0) continue;
        float c[16];
        load16(static_cast<const uint16_t *>(p.a.kv) + at, lane, c);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            float a[16], s = 0.f;
            load16(static_cast<const uint16_t *>(p.a.q) + base + h * kDc, lane, a);
#pragma unroll
            for (int i = 0; i < 16; ++i) s = fmaf(a[i], c[i], s);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
            s *= p.a.scale;
            const float now = fmaxf(top[h], s), keep = expf(top[h] - now), w = expf(s - now);
            top[h] = now;
            sum[h] = fmaf(sum[h], keep, w);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[h][i] = fmaf(o[h][i], keep, w * c[i]);
        }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        const float inv = sum[h] != 0.f ? 1.f / sum[h] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __nv_bfloat16 v = __float2bfloat16_rn(o[h][i] * inv);
            static_cast<uint16_t *>(p.a.o)[base + h * kDc + (i >> 3) * 256 + 8 * lane + (i & 7)] =
                *reinterpret_cast<const uint16_t *>(&v);
        }
        if (lane == 0)
            p.a.lse[static_cast<int64_t>(t) * kH + 8 * warp + h] =
                sum[h] != 0.f ? top[h] + logf(sum[h]) : -INFINITY;
    }
    if (bad) atomicOr(p.status, KPOOL_STATUS_BAD_PAGE);
}

// cu_q has to be 0 .. Tq and non-decreasing.
__global__ void check_kernel(const int32_t *cu_q, int B, int64_t Tq, int *status)
{
    bool bad = cu_q[0] != 0 || cu_q[B] != Tq;
    for (int i = threadIdx.x; i < B; i += blockDim.x) bad |= cu_q[i] > cu_q[i + 1];
    if (bad) atomicOr(status, KPOOL_STATUS_BAD_SEQLENS);
}

}  // namespace

size_t paged_mla_workspace_bytes(int64_t Tq, int Kp, int kpool)
{
    (void)Tq;
    (void)Kp;
    (void)kpool;
    return 256;
}

int run_paged_mla(const PagedMlaArgs &a, cudaStream_t s)
{
    KPOOL_CUDA_CHECK(cudaMemsetAsync(a.workspace, 0, 256, s));
    Params p{a, static_cast<int *>(a.workspace) + 1};
    check_kernel<<<1, 256, 0, s>>>(a.cu_q, a.B, a.Tq, p.status);
    KPOOL_CUDA_CHECK(cudaGetLastError());
    if (a.Tq == 0) return KPOOL_OK;
    paged_mla_kernel<<<static_cast<unsigned>(a.Tq), 256, 0, s>>>(p);
    KPOOL_CUDA_CHECK(cudaGetLastError());
    return KPOOL_OK;
}

}  // namespace kpool

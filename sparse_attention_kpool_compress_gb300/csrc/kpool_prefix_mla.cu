// Attention of a batch whose sequences share prefixes, over a paged latent
// cache (absorbed form: latent rows are keys and values).  include/kpool.h
// states the contract.  For query row (t, h) of sequence b, over the tokens
// j < vis(t) that it sees:
//
//   s_j = scale * q[t, h, :] . c_b[j, :]
//   o[t, h, :] = sum_j softmax_j(s) c_b[j, :],   lse[t, h] = ln sum_j exp(s_j)
//
// One warp per row: a lane holds 16 of the 512 columns, the scores are warp
// sums, and the softmax runs on a reference maximum that follows the largest
// score seen.
#include <cuda_bf16.h>

#include <algorithm>

#include "kpool_internal.h"
#include "kpool_ptx.cuh"

namespace kpool {
namespace {

constexpr int kDc = 512;
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ bool in_range(int i, int n) { return i >= 0 && i < n; }

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

__global__ void __launch_bounds__(1024) check_kernel(const PrefixMlaArgs a, int *ws)
{
    bool bad = false;
    for (int i = threadIdx.x; i <= a.B; i += blockDim.x)
        bad |= i == 0 ? a.cu_q[0] != 0 : a.cu_q[i] < a.cu_q[i - 1];
    for (int i = threadIdx.x; i <= a.G; i += blockDim.x)
        bad |= i == 0 ? a.cu_groups[0] != 0 : a.cu_groups[i] < a.cu_groups[i - 1];
    bad |= a.cu_q[a.B] != a.Tq || a.cu_groups[a.G] != a.B;
    bad = __syncthreads_or(bad) != 0;
    if (threadIdx.x == 0) ws[1] = bad ? KPOOL_STATUS_BAD_SEQLENS : 0;
}

__device__ __forceinline__ void load16(const uint16_t *row, int lane, float (&v)[16])
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + 256 * k + 8 * lane);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
            v[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__global__ void __launch_bounds__(256) rows_kernel(const PrefixMlaArgs a, int *ws)
{
    if (ws[1] & KPOOL_STATUS_BAD_SEQLENS) return;
    const int lane = threadIdx.x & 31;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
    if (row >= a.Tq * a.H) return;
    const int t = static_cast<int>(row / a.H);
    const int b = segment_of(a.cu_q, a.B, t), g = segment_of(a.cu_groups, a.G, b);
    auto table_row = [&](int seq) { return a.seq_ids != nullptr ? a.seq_ids[seq] : seq; };
    auto length = [&](int r) {
        const int64_t n = in_range(r, a.n_rows) ? a.seq_lens[r] : -1;
        const int64_t room = static_cast<int64_t>(a.max_pages) * a.page_size;
        if (n < 0 || n > room) {
            if (lane == 0) atomicOr(ws + 1, KPOOL_STATUS_BAD_PAGE);
            return static_cast<int>(n < 0 ? 0 : room);
        }
        return static_cast<int>(n);
    };
    const int first = table_row(a.cu_groups[g]), own = table_row(b);
    const int len = length(own);
    const int shared = min(max(a.prefix_lens[g], 0), length(first));
    const int vis = min(len, max(0, len - (a.cu_q[b + 1] - 1 - t)));
    const uint16_t *kv = static_cast<const uint16_t *>(a.kv);
    float q[16], acc[16], v[16];
    load16(static_cast<const uint16_t *>(a.q) + row * kDc, lane, q);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float c = a.scale * 1.44269504088896341f;
    for (int j = 0; j < vis; ++j) {
        const int r = j < shared ? first : own;
        const int page = a.page_table[static_cast<int64_t>(r) * a.max_pages + j / a.page_size];
        if (!in_range(page, a.n_pages)) {
            if (lane == 0) atomicOr(ws + 1, KPOOL_STATUS_BAD_PAGE);
            continue;
        }
        load16(kv + page * a.kv_page_stride + (j % a.page_size) * kDc, lane, v);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s = fmaf(q[i], v[i], s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        s *= c;
        if (s > m) {
            const float f = ptx::ex2_approx(m - s);
            l *= f;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] *= f;
            m = s;
        }
        const float p = ptx::ex2_approx(s - m);
        l += p;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmaf(p, v[i], acc[i]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t *o = static_cast<uint16_t *>(a.o) + row * kDc;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(acc[8 * k + 2 * i] * inv, acc[8 * k + 2 * i + 1] * inv);
            w[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
        *reinterpret_cast<uint4 *>(o + 256 * k + 8 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t prefix_mla_workspace_bytes(int64_t, int, int, int) { return 256; }

int run_prefix_mla(const PrefixMlaArgs &a, cudaStream_t s)
{
    int *ws = static_cast<int *>(a.workspace);
    check_kernel<<<1, 1024, 0, s>>>(a, ws);
    KPOOL_CUDA_CHECK(cudaGetLastError());
    const int64_t rows = a.Tq * a.H;
    if (rows > 0) rows_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(a, ws);
    KPOOL_CUDA_CHECK(cudaGetLastError());
    return KPOOL_OK;
}

}  // namespace kpool

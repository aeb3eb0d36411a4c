// Backward pass of the sparse attention over the selection (kpool_mla.cu): the
// gradients of the queries and of the latent rows, which are keys and values.
// For query row t and head h, over the row's token list J(t), with the log-sum
// lse and the output o that the forward pass left and their gradients:
//
//   p_j     = exp(scale * q[t, h, :] . c[j, :] - lse[t, h])
//   delta   = sum_d do[t, h, d] o[t, h, d] - dlse[t, h]
//   ds_j    = scale * p_j * (do[t, h, :] . c[j, :] - delta)
//   dq[t, h, :]  = sum_j ds_j c[j, :]
//   dc[j, :]    += ds_j q[t, h, :] + p_j do[t, h, :]
//
// First form: a block per row, a warp per eight heads, lanes over the columns.
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
    RowLists rows;
    const uint16_t *q, *kv, *o, *d_o;
    const float *lse, *d_lse;
    uint16_t *dq;
    float *acc;                 // [Tk, 512]: the latent rows' gradients
    float scale;
};

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

__device__ __forceinline__ float warp_dot(const float (&a)[16], const float (&b)[16])
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    return s;
}

__global__ void __launch_bounds__(256) sparse_mla_bwd_kernel(const Params p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    const RowMsg m = row_msg(p.rows, t, lane);
    const int64_t base = (static_cast<int64_t>(t) * kH + 8 * warp) * kDc;
    float dq[8][16], lse[8], delta[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        float a[16], b[16];
        load16(p.o + base + h * kDc, lane, a);
        load16(p.d_o + base + h * kDc, lane, b);
        const int64_t at = static_cast<int64_t>(t) * kH + 8 * warp + h;
        delta[h] = warp_dot(a, b) - (p.d_lse != nullptr ? p.d_lse[at] : 0.f);
        lse[h] = p.lse[at];
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[h][i] = 0.f;
    }
    for (int j = 0; j < m.n_slots; ++j) {
        const int tok = token_of(p.rows, m, j);
        if (tok < 0) continue;
        float c[16], dc[16];
        load16(p.kv + static_cast<int64_t>(tok) * kDc, lane, c);
#pragma unroll
        for (int i = 0; i < 16; ++i) dc[i] = 0.f;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            float a[16], b[16];
            load16(p.q + base + h * kDc, lane, a);
            load16(p.d_o + base + h * kDc, lane, b);
            const float s = warp_dot(a, c) * p.scale, dp = warp_dot(b, c);
            const float w = lse[h] == -INFINITY ? 0.f : expf(s - lse[h]);
            const float ds = w * (dp - delta[h]) * p.scale;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                dq[h][i] = fmaf(ds, c[i], dq[h][i]);
                dc[i] = fmaf(ds, a[i], fmaf(w, b[i], dc[i]));
            }
        }
        float *to = p.acc + static_cast<int64_t>(tok) * kDc + 8 * lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) atomicAdd(to + (i >> 3) * 256 + (i & 7), dc[i]);
    }
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __nv_bfloat16 v = __float2bfloat16_rn(dq[h][i]);
            p.dq[base + h * kDc + (i >> 3) * 256 + 8 * lane + (i & 7)] = *reinterpret_cast<const uint16_t *>(&v);
        }
}

// The sums of the latent rows' gradients, rounded to BF16: eight a thread.
__global__ void __launch_bounds__(256) round_kernel(const float4 *acc, uint4 *out, int64_t n)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n; i += step) {
        const float4 a = acc[2 * i], b = acc[2 * i + 1];
        const float2 v[4] = {{a.x, a.y}, {a.z, a.w}, {b.x, b.y}, {b.z, b.w}};
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[k].x, v[k].y);
            w[k] = *reinterpret_cast<const uint32_t *>(&x);
        }
        out[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

size_t sparse_mla_bwd_workspace_bytes(int64_t T, int64_t Tk)
{
    (void)T;
    return 256 + static_cast<size_t>(Tk) * kDc * 4;
}

int run_sparse_mla_bwd(const SparseMlaArgs &a, const SparseMlaGrad &g, cudaStream_t s)
{
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    KPOOL_CUDA_CHECK(cudaMemsetAsync(ws, 0, sparse_mla_bwd_workspace_bytes(a.T, a.Tk), s));
    Params p{};
    p.rows = row_lists(a);
    p.q = static_cast<const uint16_t *>(a.q);
    p.kv = static_cast<const uint16_t *>(a.kv);
    p.o = static_cast<const uint16_t *>(a.o);
    p.d_o = static_cast<const uint16_t *>(g.d_o);
    p.lse = a.lse;
    p.d_lse = g.d_lse;
    p.dq = static_cast<uint16_t *>(g.dq);
    p.acc = reinterpret_cast<float *>(ws + 256);
    p.scale = a.scale;
    if (a.T > 0) {
        sparse_mla_bwd_kernel<<<static_cast<unsigned>(a.T), 256, 0, s>>>(p);
        KPOOL_CUDA_CHECK(cudaGetLastError());
    }
    const int64_t n = a.Tk * (kDc / 8);
    if (n > 0) {
        round_kernel<<<static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 8 * num_sms())), 256, 0, s>>>(
            reinterpret_cast<const float4 *>(p.acc), static_cast<uint4 *>(g.dkv), n);
        KPOOL_CUDA_CHECK(cudaGetLastError());
    }
    return KPOOL_OK;
}

}  // namespace kpool

// C ABI of libkpool.so: host-side argument checks, then one or two kernel
// launches per call on the caller's stream.  See include/kpool.h for the
// contract of every entry point.
#include <cstdarg>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include <cmath>

#include "kpool_internal.h"

namespace kpool {

namespace {
thread_local std::string g_last_error;
}

void set_error(const std::string &msg) { g_last_error = msg; }
void clear_error() { g_last_error.clear(); }
const char *last_error_cstr() { return g_last_error.c_str(); }

int fail(int code, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error(buf);
    return code;
}

int num_sms()
{
    static std::mutex mu;
    static std::vector<int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    std::lock_guard<std::mutex> lk(mu);
    if (static_cast<int>(cache.size()) <= dev) cache.resize(dev + 1, 0);
    if (cache[dev] == 0) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        cache[dev] = n > 0 ? n : 1;
    }
    return cache[dev];
}

int check_docs(const int32_t *cu_seqlens, const int32_t *cu_pools, int n_docs, int64_t T,
               int kpool, int64_t P_total)
{
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1 (got %d)", n_docs);
    if ((cu_seqlens == nullptr) != (cu_pools == nullptr))
        return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens and cu_pools must both be NULL or both set");
    if (cu_seqlens == nullptr) {
        if (n_docs != 1)
            return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be 1 when cu_seqlens is NULL");
        if (P_total >= 0 && P_total != T / kpool)
            return fail(KPOOL_ERR_INVALID_ARG, "P_total must be T / kpool for one sequence");
    } else {
        if (!aligned(cu_seqlens, 4) || !aligned(cu_pools, 4))
            return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens / cu_pools must be 4-byte aligned");
    }
    if (P_total > T) return fail(KPOOL_ERR_INVALID_ARG, "P_total exceeds T");
    return KPOOL_OK;
}

}  // namespace kpool

using namespace kpool;

namespace {

int check_common(int64_t T, int kpool)
{
    if (T < 0 || T > 0x7FFFFFFFLL) return fail(KPOOL_ERR_INVALID_ARG, "T out of range");
    if (kpool < 1 || kpool > 64)
        return fail(KPOOL_ERR_UNSUPPORTED, "kpool must be in [1, 64] (got %d)", kpool);
    return KPOOL_OK;
}

// Shared checks of the sparse-attention entry points.
int check_mla_args(const void *q, const void *kv, int64_t T, int64_t Tk, int H, int Dc,
                   float scale, const void *o_out, const float *lse_out, const void *workspace,
                   size_t workspace_bytes)
{
    if (T < 0 || T > 0x7FFFFFFFLL) return fail(KPOOL_ERR_INVALID_ARG, "T out of range");
    if (Tk < 0 || Tk > 0x7FFFFFFFLL) return fail(KPOOL_ERR_INVALID_ARG, "Tk out of range");
    if (H != 64 || Dc != 512)
        return fail(KPOOL_ERR_UNSUPPORTED, "the sparse attention is built for H = 64, Dc = 512 "
                    "(got H = %d, Dc = %d)", H, Dc);
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(KPOOL_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
    if (T > 0 && (!q || !o_out || !lse_out))
        return fail(KPOOL_ERR_INVALID_ARG, "q, o_out and lse_out are required");
    if (T > 0 && !kv) return fail(KPOOL_ERR_INVALID_ARG, "kv is required");
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(o_out, 16) || !aligned(lse_out, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "q, kv and o_out must be 16-byte aligned");
    if (!workspace || workspace_bytes < sparse_mla_workspace_bytes() || !aligned(workspace, 256))
        return fail(KPOOL_ERR_WORKSPACE, "workspace of at least %zu bytes, 256-byte aligned, needed",
                    sparse_mla_workspace_bytes());
    return KPOOL_OK;
}

// What the backward calls add to the forward calls' arguments (o and lse are
// checked there, as its outputs).
int check_mla_grad(const void *d_o, const float *d_lse, int64_t T, int64_t Tk, const void *dq_out,
                   const void *dkv_out, const void *workspace, size_t workspace_bytes)
{
    if (T > 0 && (!d_o || !dq_out)) return fail(KPOOL_ERR_INVALID_ARG, "d_o and dq_out are required");
    if (Tk > 0 && !dkv_out) return fail(KPOOL_ERR_INVALID_ARG, "dkv_out is required");
    if (!aligned(d_o, 16) || !aligned(dq_out, 16) || !aligned(dkv_out, 16) || !aligned(d_lse, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "d_o, dq_out and dkv_out must be 16-byte aligned");
    const size_t need = sparse_mla_bwd_workspace_need(T, Tk);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
        return fail(KPOOL_ERR_WORKSPACE, "workspace of at least %zu bytes, 256-byte aligned, needed", need);
    return KPOOL_OK;
}

// The selection's sizes.
int check_selection(int64_t T, int kpool, int index_topk, const int32_t *pool_idx)
{
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    if (T > 0 && !pool_idx) return fail(KPOOL_ERR_INVALID_ARG, "pool_idx is required");
    if (!aligned(pool_idx, 4)) return fail(KPOOL_ERR_INVALID_ARG, "pool_idx must be 4-byte aligned");
    return KPOOL_OK;
}

// ---- paged cache -----------------------------------------------------------
int check_pool(const kpool_page_pool *p)
{
    if (!p) return fail(KPOOL_ERR_INVALID_ARG, "pool is required");
    if (p->n_seqs < 1 || p->n_pages < 1 || p->max_pages < 1 || p->page_size < 1)
        return fail(KPOOL_ERR_INVALID_ARG, "n_seqs, n_pages, max_pages and page_size must be >= 1");
    if ((static_cast<int64_t>(p->max_pages) + 1) * p->page_size > 0x7FFFFFFFLL || p->max_pages > (1 << 20))
        return fail(KPOOL_ERR_INVALID_ARG, "max_pages must be <= 2^20 and (max_pages + 1) * page_size < 2^31");
    if (p->n_pages > (1 << 28) || p->n_seqs > (1 << 28))
        return fail(KPOOL_ERR_INVALID_ARG, "n_pages and n_seqs must be <= 2^28");
    if (!p->page_table || !p->seq_lens || !p->ref_count || !p->free_list || !p->free_count)
        return fail(KPOOL_ERR_INVALID_ARG, "the pool's five arrays are required");
    if (!aligned(p->page_table, 4) || !aligned(p->seq_lens, 4) || !aligned(p->ref_count, 4) ||
        !aligned(p->free_list, 4) || !aligned(p->free_count, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "the pool's arrays must be 4-byte aligned");
    return KPOOL_OK;
}

// page_size 0: not known to the call.
int check_stores(const kpool_page_store *st, int n, int n_pages, int page_size)
{
    if (n < 0 || n > KPOOL_MAX_STORES)
        return fail(KPOOL_ERR_INVALID_ARG, "n_stores must be 0 .. %d", KPOOL_MAX_STORES);
    if (n > 0 && !st) return fail(KPOOL_ERR_INVALID_ARG, "stores are required");
    for (int i = 0; i < n; ++i) {
        const kpool_page_store &g = st[i];
        if (!g.data) return fail(KPOOL_ERR_INVALID_ARG, "store %d has no data", i);
        if (g.n_layers < 1 || g.rows_per_page < 1 || g.row_bytes < 16)
            return fail(KPOOL_ERR_INVALID_ARG, "store %d: n_layers, rows_per_page >= 1 and row_bytes >= 16 needed", i);
        if (page_size > 0 && (g.rows_per_page > page_size || page_size % g.rows_per_page != 0))
            return fail(KPOOL_ERR_INVALID_ARG, "store %d: rows_per_page must divide page_size", i);
        if (!aligned(g.data, 16) || g.layer_stride % 16 != 0 || g.page_stride % 16 != 0 || g.row_bytes % 16 != 0)
            return fail(KPOOL_ERR_INVALID_ARG, "store %d: address, strides and row_bytes must be multiples of 16", i);
        const int64_t page = static_cast<int64_t>(g.rows_per_page) * g.row_bytes;
        if (page > (int64_t(1) << 30) || g.n_layers > 4096)
            return fail(KPOOL_ERR_INVALID_ARG, "store %d: pages of at most 2^30 bytes in at most 4096 layers", i);
        if (g.layer_stride < 0 || g.page_stride < 0 || g.layer_stride > (int64_t(1) << 46) ||
            g.page_stride > (int64_t(1) << 40))
            return fail(KPOOL_ERR_INVALID_ARG, "store %d: strides out of range", i);
        // pages within layers, or layers within pages; no two pages overlap
        const bool pages_in = (n_pages == 1 || g.page_stride >= page) &&
                              (g.n_layers == 1 || g.layer_stride >= (n_pages - 1) * g.page_stride + page);
        const bool layers_in = (g.n_layers == 1 || g.layer_stride >= page) &&
                               (n_pages == 1 || g.page_stride >= (g.n_layers - 1) * g.layer_stride + page);
        if (!pages_in && !layers_in) return fail(KPOOL_ERR_INVALID_ARG, "store %d: its pages overlap", i);
    }
    return KPOOL_OK;
}

int check_pages_workspace(const void *ws, size_t bytes, int64_t n, int n_seqs, int n_pages)
{
    const size_t need = pages_workspace_bytes(n, n_seqs, n_pages);
    if (!ws || bytes < need || !aligned(ws, 256))
        return fail(KPOOL_ERR_WORKSPACE, "workspace of at least %zu bytes, 256-byte aligned, needed", need);
    return KPOOL_OK;
}

// The list arguments of a call over n items, which are all int32 arrays.
int check_items(int64_t n, std::initializer_list<const int32_t *> arrays)
{
    if (n < 0 || n > (1 << 28)) return fail(KPOOL_ERR_INVALID_ARG, "n out of range");
    for (const int32_t *a : arrays) {
        if (n > 0 && !a) return fail(KPOOL_ERR_INVALID_ARG, "a list of the call is missing");
        if (!aligned(a, 4)) return fail(KPOOL_ERR_INVALID_ARG, "the lists must be 4-byte aligned");
    }
    return KPOOL_OK;
}

// Does out[0, n) share memory with one of the pool's arrays?
bool in_pool(const int32_t *out, int64_t n, const kpool_page_pool &p)
{
    const uintptr_t o0 = reinterpret_cast<uintptr_t>(out), o1 = o0 + 4 * n;
    auto meets = [&](const int32_t *a, int64_t len) {
        const uintptr_t a0 = reinterpret_cast<uintptr_t>(a);
        return o0 < a0 + 4 * len && a0 < o1;
    };
    return meets(p.page_table, static_cast<int64_t>(p.n_seqs) * p.max_pages) || meets(p.seq_lens, p.n_seqs) ||
           meets(p.ref_count, p.n_pages) || meets(p.free_list, p.n_pages) || meets(p.free_count, 1);
}

// A call without items: a clean status word and nothing else.
int nothing_listed(void *ws, kpool_stream_t stream)
{
    KPOOL_CUDA_CHECK(cudaMemsetAsync(ws, 0, 16, reinterpret_cast<cudaStream_t>(stream)));
    return KPOOL_OK;
}

int check_h(int H)
{
    if (H != 4 && H != 8 && H != 16 && H != 32 && H != 64 && H != 128)
        return fail(KPOOL_ERR_UNSUPPORTED, "H must be one of 4, 8, 16, 32, 64, 128 (got %d)", H);
    return KPOOL_OK;
}

int check_score_args(const void *q, const float *q_scale, const float *w, const void *pk,
                     const float *pk_scale, const int32_t *cu_seqlens, const int32_t *cu_pools,
                     int n_docs, int64_t T, int64_t P_total, int H, int D, int kpool, int fp8,
                     void *workspace, size_t workspace_bytes)
{
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if ((rc = check_h(H))) return rc;
    if (fp8) {
        if (D != 128) return fail(KPOOL_ERR_UNSUPPORTED, "FP8 mode needs D = 128 (got %d)", D);
        if (!q_scale || !pk_scale)
            return fail(KPOOL_ERR_INVALID_ARG, "FP8 mode needs q_scale and pk_scale");
        if (!aligned(q_scale, 16) || !aligned(pk_scale, 4))
            return fail(KPOOL_ERR_INVALID_ARG, "q_scale must be 16-byte aligned");
    } else {
        if (D != 32 && D != 64 && D != 128)
            return fail(KPOOL_ERR_UNSUPPORTED, "D must be 32, 64 or 128 (got %d)", D);
        if (q_scale || pk_scale)
            return fail(KPOOL_ERR_INVALID_ARG, "q_scale / pk_scale must be NULL in bf16 mode");
    }
    if (T > 0 && (!q || !w)) return fail(KPOOL_ERR_INVALID_ARG, "q and w must be non-NULL");
    if (P_total > 0 && !pk) return fail(KPOOL_ERR_INVALID_ARG, "pk must be non-NULL");
    if (!aligned(q, 16) || !aligned(pk, 16) || !aligned(w, 16))
        return fail(KPOOL_ERR_INVALID_ARG, "q, pk and w must be 16-byte aligned");
    if (P_total < 0) return fail(KPOOL_ERR_INVALID_ARG, "P_total < 0");
    if (static_cast<int64_t>(T) * H > 0x7FFFFFFFLL)
        return fail(KPOOL_ERR_UNSUPPORTED, "T * H exceeds 2^31 - 1");
    if ((rc = check_docs(cu_seqlens, cu_pools, n_docs, T, kpool, P_total))) return rc;
    const size_t need = score_workspace_bytes(T, H, n_docs);
    if (!workspace || workspace_bytes < need)
        return fail(KPOOL_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu)", need,
                    workspace ? workspace_bytes : static_cast<size_t>(0));
    if (!aligned(workspace, 256))
        return fail(KPOOL_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return KPOOL_OK;
}

}  // namespace

extern "C" {

const char *kpool_last_error(void) { return last_error_cstr(); }

int kpool_version(void) { return 10000; }

int kpool_num_pools(const int32_t *cu_seqlens_host, int n_docs, int64_t T, int kpool,
                    int32_t *cu_pools_host_out, int64_t *total_pools_out)
{
    clear_error();
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if (!cu_seqlens_host || !cu_pools_host_out || !total_pools_out)
        return fail(KPOOL_ERR_INVALID_ARG, "NULL pointer");
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1");
    if (cu_seqlens_host[0] != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens[0] must be 0 (got %d)", cu_seqlens_host[0]);
    if (cu_seqlens_host[n_docs] != T)
        return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens[n_docs] must equal T");
    int64_t acc = 0;
    cu_pools_host_out[0] = 0;
    for (int d = 0; d < n_docs; ++d) {
        const int64_t L = static_cast<int64_t>(cu_seqlens_host[d + 1]) - cu_seqlens_host[d];
        if (L < 0) return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens decreases at document %d", d);
        acc += L / kpool;
        cu_pools_host_out[d + 1] = static_cast<int32_t>(acc);
    }
    *total_pools_out = acc;
    return KPOOL_OK;
}

int kpool_cu_pools(const int32_t *cu_seqlens, int n_docs, int kpool, int32_t *cu_pools_out,
                   kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_cu_pools");
    if (kpool < 1 || kpool > 64) return fail(KPOOL_ERR_UNSUPPORTED, "kpool must be in [1, 64]");
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1");
    if (!cu_seqlens || !cu_pools_out) return fail(KPOOL_ERR_INVALID_ARG, "NULL pointer");
    KPOOL_CUDA_CHECK(launch_cu_pools(cu_seqlens, n_docs, kpool, cu_pools_out,
                                     reinterpret_cast<cudaStream_t>(stream)));
    return KPOOL_OK;
}

int kpool_compress(const void *k, const void *gate, const float *ape,
                   const int32_t *cu_seqlens, const int32_t *cu_pools, int n_docs,
                   int64_t T, int D, int kpool, int64_t P_total, void *pk_out,
                   uint8_t *pk_fp8_out, float *pk_scale_out, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_compress");
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if (D != 32 && D != 64 && D != 128)
        return fail(KPOOL_ERR_UNSUPPORTED, "D must be 32, 64 or 128 (got %d)", D);
    if (P_total < 0) return fail(KPOOL_ERR_INVALID_ARG, "P_total < 0");
    if ((rc = check_docs(cu_seqlens, cu_pools, n_docs, T, kpool, P_total))) return rc;
    if (P_total > 0 && (!k || !gate || !ape || !pk_out))
        return fail(KPOOL_ERR_INVALID_ARG, "k, gate, ape and pk_out must be non-NULL");
    if (!aligned(k, 16) || !aligned(gate, 16) || !aligned(pk_out, 16) || !aligned(ape, 16))
        return fail(KPOOL_ERR_INVALID_ARG, "k, gate, ape and pk_out must be 16-byte aligned");
    if ((pk_fp8_out == nullptr) != (pk_scale_out == nullptr))
        return fail(KPOOL_ERR_INVALID_ARG, "pk_fp8_out and pk_scale_out go together");
    if (pk_fp8_out) {
        if (D != 128) return fail(KPOOL_ERR_UNSUPPORTED, "FP8 pooled keys need D = 128");
        if (!aligned(pk_fp8_out, 16) || !aligned(pk_scale_out, 4))
            return fail(KPOOL_ERR_INVALID_ARG, "pk_fp8_out must be 16-byte aligned");
    }
    KPOOL_CUDA_CHECK(launch_compress(k, gate, ape, cu_seqlens, cu_pools, n_docs, T, D, kpool,
                                     P_total, pk_out, pk_fp8_out, pk_scale_out,
                                     reinterpret_cast<cudaStream_t>(stream)));
    return KPOOL_OK;
}

int kpool_quantize_fp8(const void *x, int64_t rows, int D, uint8_t *x_fp8_out, float *scale_out,
                       kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_quantize_fp8");
    if (D != 128) return fail(KPOOL_ERR_UNSUPPORTED, "FP8 rows need D = 128 (got %d)", D);
    if (rows < 0) return fail(KPOOL_ERR_INVALID_ARG, "rows < 0");
    if (rows > 0 && (!x || !x_fp8_out || !scale_out))
        return fail(KPOOL_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(x, 16) || !aligned(x_fp8_out, 16) || !aligned(scale_out, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "x and x_fp8_out must be 16-byte aligned");
    KPOOL_CUDA_CHECK(launch_quantize_fp8(x, rows, x_fp8_out, scale_out,
                                         reinterpret_cast<cudaStream_t>(stream)));
    return KPOOL_OK;
}

size_t kpool_score_topk_workspace_size(int64_t T, int H, int n_docs)
{
    if (T < 0 || n_docs < 1 || check_h(H) != KPOOL_OK) return 0;
    return score_workspace_bytes(T, H, n_docs);
}

size_t kpool_score_topk_workspace_size_split(int64_t T, int H, int n_docs, int kpool,
                                             int index_topk)
{
    if (T < 0 || n_docs < 1 || check_h(H) != KPOOL_OK) return 0;
    if (kpool < 1 || index_topk < 1 || index_topk % kpool != 0) return 0;
    return score_workspace_split_bytes(T, H, n_docs, index_topk / kpool);
}

int kpool_score_topk(const void *q, const float *q_scale, const float *w, const void *pk,
                     const float *pk_scale, const int32_t *cu_seqlens, const int32_t *cu_pools,
                     int n_docs, int64_t T, int64_t P_total, int H, int D, int kpool,
                     int index_topk, int fp8, int32_t *pool_idx_out, float *pool_score_out,
                     void *workspace, size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_score_topk");
    int rc = check_score_args(q, q_scale, w, pk, pk_scale, cu_seqlens, cu_pools, n_docs, T,
                              P_total, H, D, kpool, fp8, workspace, workspace_bytes);
    if (rc) return rc;
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    const int Kp = index_topk / kpool;
    const int cap = score_capacity(H, D, fp8);
    int kp2 = 1;
    while (kp2 < Kp) kp2 <<= 1;
    if (Kp + 128 > cap || kp2 > cap)
        return fail(KPOOL_ERR_UNSUPPORTED,
                    "index_topk / kpool = %d exceeds the per-query candidate capacity %d for H=%d "
                    "(needs Kp + 128 and the next power of two of Kp to fit)",
                    Kp, cap, H);
    if (T > 0 && (!pool_idx_out || !pool_score_out))
        return fail(KPOOL_ERR_INVALID_ARG, "pool_idx_out and pool_score_out must be non-NULL");
    ScoreArgs a{};
    a.q = q; a.q_scale = q_scale; a.w = w; a.pk = pk; a.pk_scale = pk_scale;
    a.cu_seqlens = cu_seqlens; a.cu_pools = cu_pools; a.n_docs = n_docs;
    a.T = T; a.P_total = P_total; a.H = H; a.D = D; a.kpool = kpool; a.Kp = Kp;
    a.fp8 = fp8 ? 1 : 0; a.mode = 0;
    a.pool_idx = pool_idx_out; a.pool_score = pool_score_out; a.scores = nullptr;
    a.ws = static_cast<int *>(workspace); a.ws_bytes = workspace_bytes;
    return run_score(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_score_topk_noalloc(const void *q, const float *q_scale, const float *w, const void *pk,
                             const float *pk_scale, const int32_t *cu_seqlens,
                             const int32_t *cu_pools, int n_docs, int64_t T, int64_t P_total,
                             int H, int D, int kpool, int index_topk, int fp8,
                             int32_t *pool_idx_out, float *pool_score_out, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_score_topk_noalloc");
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if ((rc = check_h(H))) return rc;
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1 (got %d)", n_docs);
    int *scratch = nullptr;
    size_t scratch_bytes = 0;
    int64_t max_tiles = 0;
    const int64_t QT = 256 / H;
    const int64_t need_tiles = (T + QT - 1) / QT + n_docs;
    // the capacity is a compile-time constant: reject before touching the device
    if (need_tiles > kNoAllocMaxTiles)
        return fail(KPOOL_ERR_UNSUPPORTED,
                    "kpool_score_topk_noalloc: T=%lld with H=%d and %d documents needs %lld "
                    "query tiles; its fixed scratch holds at most %d (use kpool_score_topk "
                    "with a caller-provided workspace)",
                    static_cast<long long>(T), H, n_docs, static_cast<long long>(need_tiles),
                    kNoAllocMaxTiles);
    if ((rc = noalloc_scratch(&scratch, &scratch_bytes, &max_tiles))) return rc;
    if (need_tiles > max_tiles)
        return fail(KPOOL_ERR_UNSUPPORTED, "no-alloc scratch too small (%lld tiles needed)",
                    static_cast<long long>(need_tiles));
    return kpool_score_topk(q, q_scale, w, pk, pk_scale, cu_seqlens, cu_pools, n_docs, T, P_total,
                            H, D, kpool, index_topk, fp8, pool_idx_out, pool_score_out, scratch,
                            scratch_bytes, stream);
}

int kpool_score_topk_at(const void *q, const float *q_scale, const float *w, const void *pk,
                        const float *pk_scale, const int32_t *cu_seqlens_q,
                        const int32_t *q_start_pos, const int32_t *cu_pools, int n_docs,
                        int64_t Tq, int64_t P_total, int H, int D, int kpool, int index_topk,
                        int fp8, int32_t *pool_idx_out, float *pool_score_out, void *workspace,
                        size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_score_topk_at");
    if (!cu_seqlens_q || !q_start_pos || !cu_pools)
        return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens_q, q_start_pos and cu_pools are required");
    if (!aligned(q_start_pos, 4)) return fail(KPOOL_ERR_INVALID_ARG, "q_start_pos misaligned");
    // the key-side pool count is independent of the number of query rows
    int rc = check_score_args(q, q_scale, w, pk, pk_scale, cu_seqlens_q, cu_pools, n_docs, Tq, 0,
                              H, D, kpool, fp8, workspace, workspace_bytes);
    if (rc) return rc;
    if (P_total < 0) return fail(KPOOL_ERR_INVALID_ARG, "P_total < 0");
    if (P_total > 0 && !pk) return fail(KPOOL_ERR_INVALID_ARG, "pk must be non-NULL");
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    const int Kp = index_topk / kpool;
    const int cap = score_capacity(H, D, fp8);
    int kp2 = 1;
    while (kp2 < Kp) kp2 <<= 1;
    if (Kp + 128 > cap || kp2 > cap)
        return fail(KPOOL_ERR_UNSUPPORTED,
                    "index_topk / kpool = %d exceeds the per-query candidate capacity %d for H=%d",
                    Kp, cap, H);
    if (Tq > 0 && (!pool_idx_out || !pool_score_out))
        return fail(KPOOL_ERR_INVALID_ARG, "pool_idx_out and pool_score_out must be non-NULL");
    ScoreArgs a{};
    a.q = q; a.q_scale = q_scale; a.w = w; a.pk = pk; a.pk_scale = pk_scale;
    a.cu_seqlens = cu_seqlens_q; a.cu_pools = cu_pools; a.q_pos = q_start_pos; a.n_docs = n_docs;
    a.T = Tq; a.P_total = P_total; a.H = H; a.D = D; a.kpool = kpool; a.Kp = Kp;
    a.fp8 = fp8 ? 1 : 0; a.mode = 0;
    a.pool_idx = pool_idx_out; a.pool_score = pool_score_out; a.scores = nullptr;
    a.ws = static_cast<int *>(workspace); a.ws_bytes = workspace_bytes;
    return run_score(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_expand_indices_at(const int32_t *pool_idx, const int32_t *cu_seqlens_q,
                            const int32_t *q_start_pos, const int32_t *cu_seqlens_k,
                            const int32_t *cu_pools, int n_docs, int64_t Tq, int kpool,
                            int index_topk, int always_select_tail, int32_t *tok_idx_out,
                            kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_expand_indices_at");
    int rc = check_common(Tq, kpool);
    if (rc) return rc;
    if (!cu_seqlens_q || !q_start_pos || !cu_seqlens_k || !cu_pools)
        return fail(KPOOL_ERR_INVALID_ARG,
                    "cu_seqlens_q, q_start_pos, cu_seqlens_k and cu_pools are required");
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1");
    if (!aligned(cu_seqlens_q, 4) || !aligned(q_start_pos, 4) || !aligned(cu_seqlens_k, 4) ||
        !aligned(cu_pools, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    if (Tq > 0 && (!pool_idx || !tok_idx_out))
        return fail(KPOOL_ERR_INVALID_ARG, "pool_idx and tok_idx_out must be non-NULL");
    if (!aligned(pool_idx, 4) || !aligned(tok_idx_out, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "pool_idx and tok_idx_out must be 4-byte aligned");
    const int Kp = index_topk / kpool;
    KPOOL_CUDA_CHECK(launch_expand(pool_idx, cu_seqlens_q, q_start_pos, cu_seqlens_k, cu_pools,
                                   n_docs, Tq, kpool, Kp, always_select_tail ? 1 : 0, tok_idx_out,
                                   reinterpret_cast<cudaStream_t>(stream)));
    return KPOOL_OK;
}

int kpool_score_dense(const void *q, const float *q_scale, const float *w, const void *pk,
                      const float *pk_scale, const int32_t *cu_seqlens, const int32_t *cu_pools,
                      int n_docs, int64_t T, int64_t P_total, int H, int D, int kpool, int fp8,
                      float *scores_out, void *workspace, size_t workspace_bytes,
                      kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_score_dense");
    int rc = check_score_args(q, q_scale, w, pk, pk_scale, cu_seqlens, cu_pools, n_docs, T,
                              P_total, H, D, kpool, fp8, workspace, workspace_bytes);
    if (rc) return rc;
    if (T > 0 && P_total > 0 && !scores_out)
        return fail(KPOOL_ERR_INVALID_ARG, "scores_out must be non-NULL");
    if (static_cast<double>(T) * static_cast<double>(P_total) > 4.0e9)
        return fail(KPOOL_ERR_UNSUPPORTED, "dense scores are meant for small T");
    ScoreArgs a{};
    a.q = q; a.q_scale = q_scale; a.w = w; a.pk = pk; a.pk_scale = pk_scale;
    a.cu_seqlens = cu_seqlens; a.cu_pools = cu_pools; a.n_docs = n_docs;
    a.T = T; a.P_total = P_total; a.H = H; a.D = D; a.kpool = kpool; a.Kp = 1;
    a.fp8 = fp8 ? 1 : 0; a.mode = 1;
    a.pool_idx = nullptr; a.pool_score = nullptr; a.scores = scores_out;
    a.ws = static_cast<int *>(workspace); a.ws_bytes = workspace_bytes;
    return run_score(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_expand_indices(const int32_t *pool_idx, const int32_t *cu_seqlens,
                         const int32_t *cu_pools, int n_docs, int64_t T, int kpool,
                         int index_topk, int always_select_tail, int32_t *tok_idx_out,
                         kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_expand_indices");
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    if ((rc = check_docs(cu_seqlens, cu_pools, n_docs, T, kpool, -1))) return rc;
    if (T > 0 && (!pool_idx || !tok_idx_out))
        return fail(KPOOL_ERR_INVALID_ARG, "pool_idx and tok_idx_out must be non-NULL");
    if (!aligned(pool_idx, 4) || !aligned(tok_idx_out, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "pool_idx and tok_idx_out must be 4-byte aligned");
    const int Kp = index_topk / kpool;
    if (static_cast<int64_t>(Kp) * kpool + kpool > 0x7FFFFFFF)
        return fail(KPOOL_ERR_UNSUPPORTED, "row width overflows");
    KPOOL_CUDA_CHECK(launch_expand(pool_idx, cu_seqlens, nullptr, nullptr, cu_pools, n_docs, T,
                                   kpool, Kp, always_select_tail ? 1 : 0, tok_idx_out,
                                   reinterpret_cast<cudaStream_t>(stream)));
    return KPOOL_OK;
}

}  // extern "C"

namespace {

// Host-side layout check of a host cu_seqlens; fills *P_total.
int host_layout(const int32_t *cu_host, int n_docs, int64_t T, int kpool, int64_t *P_total)
{
    if (!cu_host) {
        *P_total = T / kpool;
        return KPOOL_OK;
    }
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1 (got %d)", n_docs);
    if (cu_host[0] != 0 || cu_host[n_docs] != T)
        return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens must run from 0 to T");
    int64_t P = 0;
    for (int d = 0; d < n_docs; ++d) {
        const int64_t L = static_cast<int64_t>(cu_host[d + 1]) - cu_host[d];
        if (L < 0) return fail(KPOOL_ERR_INVALID_ARG, "cu_seqlens must be non-decreasing");
        P += L / kpool;
    }
    *P_total = P;
    return KPOOL_OK;
}

int check_forward_shapes(int64_t T, int H, int D, int kpool, int index_topk, int fp8)
{
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if ((rc = check_h(H))) return rc;
    if (fp8 ? D != 128 : (D != 32 && D != 64 && D != 128))
        return fail(KPOOL_ERR_UNSUPPORTED, "D must be 32, 64 or 128 (128 in FP8 mode)");
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    const int Kp = index_topk / kpool;
    const int cap = score_capacity(H, D, fp8);
    int kp2 = 1;
    while (kp2 < Kp) kp2 <<= 1;
    if (Kp + 128 > cap || kp2 > cap)
        return fail(KPOOL_ERR_UNSUPPORTED,
                    "index_topk / kpool = %d exceeds the per-query candidate capacity %d", Kp,
                    cap);
    if (T * H > 0x7FFFFFFFLL) return fail(KPOOL_ERR_UNSUPPORTED, "T * H exceeds 2^31 - 1");
    return KPOOL_OK;
}

}  // namespace

extern "C" {

size_t kpool_indexer_forward_host_scratch_size(const int32_t *cu_seqlens_host, int n_docs,
                                               int64_t T, int H, int D, int kpool,
                                               int index_topk, int fp8, int64_t chunk_rows)
{
    if (chunk_rows < 0 || check_forward_shapes(T, H, D, kpool, index_topk, fp8)) return 0;
    int64_t P = 0;
    if (host_layout(cu_seqlens_host, cu_seqlens_host ? n_docs : 1, T, kpool, &P)) return 0;
    return pipeline_scratch_bytes(T, H, D, cu_seqlens_host ? n_docs : 1, kpool, index_topk, fp8,
                                  chunk_rows, P);
}

int kpool_indexer_forward_host(const void *q, const void *k, const void *gate, const float *ape,
                               const float *w, const int32_t *cu_seqlens_host, int n_docs,
                               int64_t T, int H, int D, int kpool, int index_topk,
                               int always_select_tail, int fp8, int64_t chunk_rows,
                               int32_t *tok_idx_out, void *scratch, size_t scratch_bytes,
                               kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_indexer_forward_host");
    int rc = check_forward_shapes(T, H, D, kpool, index_topk, fp8);
    if (rc) return rc;
    if (chunk_rows < 0) return fail(KPOOL_ERR_INVALID_ARG, "chunk_rows < 0");
    if (!cu_seqlens_host) n_docs = 1;
    int64_t P = 0;
    if ((rc = host_layout(cu_seqlens_host, n_docs, T, kpool, &P))) return rc;
    if (T == 0) return KPOOL_OK;
    if (!q || !k || !gate || !ape || !w || !tok_idx_out)
        return fail(KPOOL_ERR_INVALID_ARG, "NULL host pointer");
    if (!scratch) return fail(KPOOL_ERR_WORKSPACE, "scratch is NULL");
    if (!aligned(scratch, 256))
        return fail(KPOOL_ERR_INVALID_ARG, "scratch must be 256-byte aligned");
    PipelineArgs a{};
    a.q = q;
    a.k = k;
    a.gate = gate;
    a.ape = ape;
    a.w = w;
    a.cu_seqlens_host = cu_seqlens_host;   // NULL: one sequence
    a.n_docs = n_docs;
    a.T = T;
    a.P_total = P;
    a.chunk_rows = chunk_rows;
    a.H = H;
    a.D = D;
    a.kpool = kpool;
    a.index_topk = index_topk;
    a.tail = always_select_tail ? 1 : 0;
    a.fp8 = fp8 ? 1 : 0;
    a.tok_out = tok_idx_out;
    a.scratch = scratch;
    a.scratch_bytes = scratch_bytes;
    return run_pipeline(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_read_status(const void *workspace, int *status_out)
{
    clear_error();
    if (!workspace || !status_out) return fail(KPOOL_ERR_INVALID_ARG, "NULL pointer");
    KPOOL_CUDA_CHECK(cudaDeviceSynchronize());
    int v = 0;
    KPOOL_CUDA_CHECK(cudaMemcpy(&v, static_cast<const int *>(workspace) + 1, sizeof(int),
                                cudaMemcpyDeviceToHost));
    *status_out = v;
    return KPOOL_OK;
}

int kpool_project_compress(const void *x, const void *w_kg, const float *k_norm_weight,
                           const float *k_norm_bias, float k_norm_eps, const float *ape,
                           const int32_t *cu_seqlens, const int32_t *cu_pools, int n_docs,
                           int64_t T, int hidden, int D, int kpool, int64_t P_total, void *pk_out,
                           void *k_out, void *gate_out, void *workspace, size_t workspace_bytes,
                           kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_project_compress");
    int rc = check_common(T, kpool);
    if (rc) return rc;
    if (D != 128) return fail(KPOOL_ERR_UNSUPPORTED, "the fused projection needs D = 128 (got %d)", D);
    if (32 % kpool != 0)
        return fail(KPOOL_ERR_UNSUPPORTED, "the fused projection needs kpool dividing 32 (got %d)",
                    kpool);
    if (hidden < 64 || hidden % 64 != 0 || hidden > 65536)
        return fail(KPOOL_ERR_UNSUPPORTED, "hidden must be a multiple of 64 in [64, 65536] (got %d)",
                    hidden);
    if (T * static_cast<int64_t>(hidden) > (int64_t(1) << 40))
        return fail(KPOOL_ERR_UNSUPPORTED, "T * hidden too large");
    if (P_total < 0) return fail(KPOOL_ERR_INVALID_ARG, "P_total < 0");
    if ((rc = check_docs(cu_seqlens, cu_pools, n_docs, T, kpool, P_total))) return rc;
    if (T > 0 && (!x || !w_kg || !k_norm_weight || !k_norm_bias || !ape))
        return fail(KPOOL_ERR_INVALID_ARG, "x, w_kg, k_norm_weight, k_norm_bias and ape are required");
    if (P_total > 0 && !pk_out) return fail(KPOOL_ERR_INVALID_ARG, "pk_out is required");
    if (!aligned(x, 16) || !aligned(w_kg, 16) || !aligned(pk_out, 16) || !aligned(k_out, 16) ||
        !aligned(gate_out, 16) || !aligned(ape, 4) || !aligned(k_norm_weight, 4) ||
        !aligned(k_norm_bias, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "x, w_kg, pk_out, k_out and gate_out must be 16-byte aligned");
    if (!(k_norm_eps >= 0.f)) return fail(KPOOL_ERR_INVALID_ARG, "k_norm_eps must be >= 0");
    if (!workspace || workspace_bytes < 256 || !aligned(workspace, 256))
        return fail(KPOOL_ERR_WORKSPACE, "workspace of at least 256 bytes, 256-byte aligned, needed");
    ProjectArgs a{};
    a.x = x; a.w = w_kg; a.gamma = k_norm_weight; a.beta = k_norm_bias; a.ape = ape;
    a.eps = k_norm_eps; a.cu_seqlens = cu_seqlens; a.cu_pools = cu_pools; a.n_docs = n_docs;
    a.T = T; a.P_total = P_total; a.hidden = hidden; a.kpool = kpool;
    a.pk_out = pk_out; a.k_out = k_out; a.gate_out = gate_out;
    a.status = static_cast<int *>(workspace) + 1;
    return run_project_compress(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_score_topk_noalloc_status(int *status_out)
{
    clear_error();
    if (!status_out) return fail(KPOOL_ERR_INVALID_ARG, "NULL pointer");
    int *scratch = nullptr;
    size_t scratch_bytes = 0;
    int64_t max_tiles = 0;
    const int rc = noalloc_scratch(&scratch, &scratch_bytes, &max_tiles);
    if (rc) return rc;
    return kpool_read_status(scratch, status_out);
}

uint64_t kpool_debug_set_wait_limit_ns(uint64_t ns) { return set_wait_limit_ns(ns); }

size_t kpool_sparse_mla_workspace_size(void) { return sparse_mla_workspace_bytes(); }

int kpool_sparse_mla_fwd(const void *q, const void *kv, const int32_t *tok_idx, int64_t T,
                         int64_t Tk, int W, int H, int Dc, float softmax_scale, void *o_out,
                         float *lse_out, void *workspace, size_t workspace_bytes,
                         kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_fwd");
    int rc = check_mla_args(q, kv, T, Tk, H, Dc, softmax_scale, o_out, lse_out, workspace,
                            workspace_bytes);
    if (rc) return rc;
    if (W < 0 || W > (1 << 20)) return fail(KPOOL_ERR_INVALID_ARG, "W out of range");
    if (T > 0 && W > 0 && !tok_idx) return fail(KPOOL_ERR_INVALID_ARG, "tok_idx is required");
    if (!aligned(tok_idx, 4)) return fail(KPOOL_ERR_INVALID_ARG, "tok_idx must be 4-byte aligned");
    SparseMlaArgs a{};
    a.q = q; a.kv = kv; a.tok_idx = tok_idx; a.T = T; a.Tk = Tk; a.W = W; a.n_docs = 1;
    a.kpool = 1; a.scale = softmax_scale; a.o = o_out; a.lse = lse_out; a.workspace = workspace;
    // a zero-width list still runs the kernel (every row gets o = 0 and
    // lse = -inf); the kernel never reads a row of width 0
    if (W == 0) a.tok_idx = static_cast<const int32_t *>(workspace);
    return run_sparse_mla(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_sparse_mla_fwd_pools(const void *q, const void *kv, const int32_t *pool_idx,
                               const int32_t *cu_seqlens, const int32_t *cu_pools, int n_docs,
                               int64_t T, int H, int Dc, int kpool, int index_topk,
                               int always_select_tail, float softmax_scale, void *o_out,
                               float *lse_out, void *workspace, size_t workspace_bytes,
                               kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_fwd_pools");
    int rc = check_mla_args(q, kv, T, T, H, Dc, softmax_scale, o_out, lse_out, workspace,
                            workspace_bytes);
    if (rc) return rc;
    if ((rc = check_common(T, kpool))) return rc;
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    if ((rc = check_docs(cu_seqlens, cu_pools, n_docs, T, kpool, -1))) return rc;
    if (T > 0 && !pool_idx) return fail(KPOOL_ERR_INVALID_ARG, "pool_idx is required");
    if (!aligned(pool_idx, 4)) return fail(KPOOL_ERR_INVALID_ARG, "pool_idx must be 4-byte aligned");
    SparseMlaArgs a{};
    a.q = q; a.kv = kv; a.pool_idx = pool_idx; a.cu_seqlens = cu_seqlens; a.cu_pools = cu_pools;
    a.n_docs = n_docs; a.T = T; a.Tk = T; a.kpool = kpool; a.Kp = index_topk / kpool;
    a.tail = always_select_tail ? 1 : 0; a.scale = softmax_scale; a.o = o_out; a.lse = lse_out;
    a.workspace = workspace;
    return run_sparse_mla(a, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_sparse_mla_fwd_pools_at(const void *q, const void *kv, const int32_t *pool_idx,
                                  const int32_t *cu_seqlens_q, const int32_t *q_start_pos,
                                  const int32_t *cu_seqlens_k, const int32_t *cu_pools, int n_docs,
                                  int64_t Tq, int64_t Tk, int H, int Dc, int kpool, int index_topk,
                                  int always_select_tail, float softmax_scale, void *o_out,
                                  float *lse_out, void *workspace, size_t workspace_bytes,
                                  kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_fwd_pools_at");
    int rc = check_mla_args(q, kv, Tq, Tk, H, Dc, softmax_scale, o_out, lse_out, workspace,
                            workspace_bytes);
    if (rc) return rc;
    if ((rc = check_common(Tq, kpool))) return rc;
    if (!cu_seqlens_q || !q_start_pos || !cu_seqlens_k || !cu_pools)
        return fail(KPOOL_ERR_INVALID_ARG,
                    "cu_seqlens_q, q_start_pos, cu_seqlens_k and cu_pools are required");
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1");
    if (!aligned(cu_seqlens_q, 4) || !aligned(q_start_pos, 4) || !aligned(cu_seqlens_k, 4) ||
        !aligned(cu_pools, 4) || !aligned(pool_idx, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
    if (index_topk < 1 || index_topk % kpool != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "index_topk must be a positive multiple of kpool");
    if (Tq > 0 && !pool_idx) return fail(KPOOL_ERR_INVALID_ARG, "pool_idx is required");
    SparseMlaArgs a{};
    a.q = q; a.kv = kv; a.pool_idx = pool_idx; a.cu_seqlens = cu_seqlens_q; a.q_pos = q_start_pos;
    a.cu_k = cu_seqlens_k; a.cu_pools = cu_pools; a.n_docs = n_docs; a.T = Tq; a.Tk = Tk;
    a.kpool = kpool; a.Kp = index_topk / kpool; a.tail = always_select_tail ? 1 : 0;
    a.scale = softmax_scale; a.o = o_out; a.lse = lse_out; a.workspace = workspace;
    return run_sparse_mla(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t kpool_sparse_mla_bwd_workspace_size(int64_t T, int64_t Tk)
{
    if (T < 0 || T > 0x7FFFFFFFLL || Tk < 0 || Tk > 0x7FFFFFFFLL) return 0;
    return sparse_mla_bwd_workspace_bytes(T, Tk);
}

int kpool_sparse_mla_bwd(const void *q, const void *kv, const int32_t *tok_idx, const void *o, const float *lse,
                         const void *d_o, const float *d_lse, int64_t T, int64_t Tk, int W, int H, int Dc,
                         float softmax_scale, void *dq_out, void *dkv_out, void *workspace, size_t workspace_bytes,
                         kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_bwd");
    int rc = check_mla_args(q, kv, T, Tk, H, Dc, softmax_scale, o, lse, workspace, workspace_bytes);
    if (rc) return rc;
    if ((rc = check_mla_grad(d_o, d_lse, T, Tk, dq_out, dkv_out, workspace, workspace_bytes))) return rc;
    if (W < 0 || W > (1 << 20)) return fail(KPOOL_ERR_INVALID_ARG, "W out of range");
    if (T > 0 && W > 0 && !tok_idx) return fail(KPOOL_ERR_INVALID_ARG, "tok_idx is required");
    if (!aligned(tok_idx, 4)) return fail(KPOOL_ERR_INVALID_ARG, "tok_idx must be 4-byte aligned");
    SparseMlaArgs a{};
    a.q = q; a.kv = kv; a.tok_idx = tok_idx; a.T = T; a.Tk = Tk; a.W = W; a.n_docs = 1;
    a.kpool = 1; a.scale = softmax_scale; a.o = const_cast<void *>(o); a.lse = const_cast<float *>(lse);
    a.workspace = workspace;
    // (a row of width 0 is never read)
    if (W == 0) a.tok_idx = static_cast<const int32_t *>(workspace);
    const SparseMlaGrad g{d_o, d_lse, dq_out, dkv_out};
    return run_sparse_mla_bwd(a, g, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_sparse_mla_bwd_pools(const void *q, const void *kv, const int32_t *pool_idx, const int32_t *cu_seqlens,
                               const int32_t *cu_pools, int n_docs, const void *o, const float *lse, const void *d_o,
                               const float *d_lse, int64_t T, int H, int Dc, int kpool, int index_topk,
                               int always_select_tail, float softmax_scale, void *dq_out, void *dkv_out,
                               void *workspace, size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_bwd_pools");
    int rc = check_mla_args(q, kv, T, T, H, Dc, softmax_scale, o, lse, workspace, workspace_bytes);
    if (rc) return rc;
    if ((rc = check_mla_grad(d_o, d_lse, T, T, dq_out, dkv_out, workspace, workspace_bytes))) return rc;
    if ((rc = check_selection(T, kpool, index_topk, pool_idx))) return rc;
    if ((rc = check_docs(cu_seqlens, cu_pools, n_docs, T, kpool, -1))) return rc;
    SparseMlaArgs a{};
    a.q = q; a.kv = kv; a.pool_idx = pool_idx; a.cu_seqlens = cu_seqlens; a.cu_pools = cu_pools;
    a.n_docs = n_docs; a.T = T; a.Tk = T; a.kpool = kpool; a.Kp = index_topk / kpool;
    a.tail = always_select_tail ? 1 : 0; a.scale = softmax_scale; a.o = const_cast<void *>(o);
    a.lse = const_cast<float *>(lse); a.workspace = workspace;
    const SparseMlaGrad g{d_o, d_lse, dq_out, dkv_out};
    return run_sparse_mla_bwd(a, g, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_sparse_mla_bwd_pools_at(const void *q, const void *kv, const int32_t *pool_idx,
                                  const int32_t *cu_seqlens_q, const int32_t *q_start_pos,
                                  const int32_t *cu_seqlens_k, const int32_t *cu_pools, int n_docs, const void *o,
                                  const float *lse, const void *d_o, const float *d_lse, int64_t Tq, int64_t Tk, int H,
                                  int Dc, int kpool, int index_topk, int always_select_tail, float softmax_scale,
                                  void *dq_out, void *dkv_out, void *workspace, size_t workspace_bytes,
                                  kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_bwd_pools_at");
    int rc = check_mla_args(q, kv, Tq, Tk, H, Dc, softmax_scale, o, lse, workspace, workspace_bytes);
    if (rc) return rc;
    if ((rc = check_mla_grad(d_o, d_lse, Tq, Tk, dq_out, dkv_out, workspace, workspace_bytes))) return rc;
    if ((rc = check_selection(Tq, kpool, index_topk, pool_idx))) return rc;
    if (!cu_seqlens_q || !q_start_pos || !cu_seqlens_k || !cu_pools)
        return fail(KPOOL_ERR_INVALID_ARG,
                    "cu_seqlens_q, q_start_pos, cu_seqlens_k and cu_pools are required");
    if (n_docs < 1) return fail(KPOOL_ERR_INVALID_ARG, "n_docs must be >= 1");
    if (!aligned(cu_seqlens_q, 4) || !aligned(q_start_pos, 4) || !aligned(cu_seqlens_k, 4) || !aligned(cu_pools, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
    SparseMlaArgs a{};
    a.q = q; a.kv = kv; a.pool_idx = pool_idx; a.cu_seqlens = cu_seqlens_q; a.q_pos = q_start_pos;
    a.cu_k = cu_seqlens_k; a.cu_pools = cu_pools; a.n_docs = n_docs; a.T = Tq; a.Tk = Tk;
    a.kpool = kpool; a.Kp = index_topk / kpool; a.tail = always_select_tail ? 1 : 0;
    a.scale = softmax_scale; a.o = const_cast<void *>(o); a.lse = const_cast<float *>(lse); a.workspace = workspace;
    const SparseMlaGrad g{d_o, d_lse, dq_out, dkv_out};
    return run_sparse_mla_bwd(a, g, reinterpret_cast<cudaStream_t>(stream));
}

size_t kpool_sparse_mla_paged_workspace_size(int64_t Tq, int kpool, int index_topk)
{
    if (Tq < 0 || Tq > 0x7FFFFFFFLL || kpool < 1 || kpool > 64 || index_topk < 1 || index_topk % kpool != 0) return 0;
    return paged_mla_workspace_bytes(Tq, index_topk / kpool, kpool);
}

int kpool_sparse_mla_fwd_pools_paged(const void *q, const void *kv, int64_t kv_page_stride, int n_pages, int page_size,
                                     const int32_t *page_table, const int32_t *seq_lens, int n_rows, int max_pages,
                                     const int32_t *seq_ids, const int32_t *pool_idx, const int32_t *cu_seqlens_q,
                                     const int32_t *q_start_pos, const int32_t *cu_pools, int B, int64_t Tq, int H,
                                     int Dc, int kpool, int index_topk, int always_select_tail, float softmax_scale,
                                     void *o_out, float *lse_out, void *workspace, size_t workspace_bytes,
                                     kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_sparse_mla_fwd_pools_paged");
    int rc = check_mla_args(q, kv, Tq, 0, H, Dc, softmax_scale, o_out, lse_out, workspace, workspace_bytes);
    if (rc) return rc;
    if ((rc = check_selection(Tq, kpool, index_topk, pool_idx))) return rc;
    if (B < 1 || B > (1 << 24)) return fail(KPOOL_ERR_INVALID_ARG, "B must be 1 .. 2^24");
    if (n_rows < 1 || max_pages < 1 || max_pages > (1 << 20) || page_size < 1 ||
        static_cast<int64_t>(max_pages) * page_size > 0x7FFFFFFFLL)
        return fail(KPOOL_ERR_INVALID_ARG,
                    "n_rows and page_size must be >= 1, max_pages 1 .. 2^20, max_pages * page_size < 2^31");
    if (!seq_ids && n_rows < B) return fail(KPOOL_ERR_INVALID_ARG, "without seq_ids, n_rows must be >= B");
    if (n_pages < 1 || n_pages > (1 << 28)) return fail(KPOOL_ERR_INVALID_ARG, "n_pages out of range");
    if (kv_page_stride < static_cast<int64_t>(page_size) * Dc || kv_page_stride % 8 != 0 ||
        kv_page_stride >= (int64_t(1) << 34))
        return fail(KPOOL_ERR_INVALID_ARG, "kv_page_stride must be a multiple of 8 of at least a page's elements");
    if (!kv || !page_table || !seq_lens || !cu_seqlens_q || !q_start_pos || !cu_pools)
        return fail(KPOOL_ERR_INVALID_ARG,
                    "kv, page_table, seq_lens, cu_seqlens_q, q_start_pos and cu_pools are required");
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(seq_ids, 4) || !aligned(cu_seqlens_q, 4) ||
        !aligned(q_start_pos, 4) || !aligned(cu_pools, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
    const size_t need = paged_mla_workspace_need(Tq, index_topk / kpool, kpool);
    if (workspace_bytes < need)
        return fail(KPOOL_ERR_WORKSPACE, "workspace of at least %zu bytes, 256-byte aligned, needed", need);
    PagedMlaArgs a{};
    a.q = q; a.kv = kv; a.kv_page_stride = kv_page_stride; a.n_pages = n_pages; a.page_size = page_size;
    a.page_table = page_table; a.seq_lens = seq_lens; a.n_rows = n_rows; a.max_pages = max_pages;
    a.seq_ids = seq_ids; a.pool_idx = pool_idx; a.cu_q = cu_seqlens_q; a.q_pos = q_start_pos; a.cu_pools = cu_pools;
    a.B = B; a.Tq = Tq; a.kpool = kpool; a.Kp = index_topk / kpool; a.tail = always_select_tail ? 1 : 0;
    a.scale = softmax_scale; a.o = o_out; a.lse = lse_out; a.workspace = workspace;
    return run_paged_mla(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t kpool_pages_workspace_size(int64_t n, int n_seqs, int n_pages)
{
    if (n < 0 || n > (1 << 28) || n_seqs < 0 || n_seqs > (1 << 28) || n_pages < 1 || n_pages > (1 << 28)) return 0;
    return pages_workspace_bytes(n, n_seqs, n_pages);
}

int kpool_pages_copy(const int32_t *src, const int32_t *dst, int64_t n, int n_pages,
                     const kpool_page_store *stores, int n_stores, void *workspace,
                     size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_pages_copy");
    if (n_pages < 1 || n_pages > (1 << 28)) return fail(KPOOL_ERR_INVALID_ARG, "n_pages out of range");
    int rc = check_items(n, {src, dst});
    if (rc) return rc;
    if ((rc = check_stores(stores, n_stores, n_pages, 0))) return rc;
    if (n <= kPagesFusedCopy) {
        if (!workspace || workspace_bytes < 256 || !aligned(workspace, 256))
            return fail(KPOOL_ERR_WORKSPACE, "workspace of at least 256 bytes, 256-byte aligned, needed");
    } else if ((rc = check_pages_workspace(workspace, workspace_bytes, n, 0, n_pages))) {
        return rc;
    }
    if (n == 0) return nothing_listed(workspace, stream);
    return run_pages_copy(src, dst, static_cast<int>(n), n_pages, stores, n_stores, workspace,
                          reinterpret_cast<cudaStream_t>(stream));
}

int kpool_pages_fork(const kpool_page_pool *pool, const int32_t *parents, const int32_t *children, int64_t n,
                     const kpool_page_store *stores, int n_stores, void *workspace, size_t workspace_bytes,
                     kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_pages_fork");
    int rc = check_pool(pool);
    if (rc) return rc;
    if ((rc = check_items(n, {parents, children}))) return rc;
    if ((rc = check_stores(stores, n_stores, pool->n_pages, pool->page_size))) return rc;
    if ((rc = check_pages_workspace(workspace, workspace_bytes, n, pool->n_seqs, pool->n_pages))) return rc;
    if (n == 0) return nothing_listed(workspace, stream);
    return run_pages_fork(*pool, parents, children, static_cast<int>(n), stores, n_stores, workspace,
                          reinterpret_cast<cudaStream_t>(stream));
}

int kpool_pages_extend(const kpool_page_pool *pool, const int32_t *seqs, const int32_t *n_new, int64_t n,
                       int32_t *begin_out, void *workspace, size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_pages_extend");
    int rc = check_pool(pool);
    if (rc) return rc;
    if ((rc = check_items(n, {seqs, n_new, begin_out}))) return rc;
    if ((begin_out < seqs + n && seqs < begin_out + n) || (begin_out < n_new + n && n_new < begin_out + n))
        return fail(KPOOL_ERR_INVALID_ARG, "begin_out overlaps a list of the call");
    if ((rc = check_pages_workspace(workspace, workspace_bytes, n, pool->n_seqs, pool->n_pages))) return rc;
    if (n > 0 && in_pool(begin_out, n, *pool)) return fail(KPOOL_ERR_INVALID_ARG, "begin_out overlaps the pool's arrays");
    if (n == 0) return nothing_listed(workspace, stream);
    return run_pages_extend(*pool, seqs, n_new, static_cast<int>(n), begin_out, workspace,
                            reinterpret_cast<cudaStream_t>(stream));
}

int kpool_pages_write(const kpool_page_pool *pool, const int32_t *seqs, const int32_t *begin,
                      const int32_t *cu_rows, int64_t n, int64_t total, const void *rows,
                      int64_t rows_layer_stride, const kpool_page_store *store, void *workspace,
                      size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_pages_write");
    int rc = check_pool(pool);
    if (rc) return rc;
    if ((rc = check_items(n, {seqs, begin, cu_rows}))) return rc;
    if ((rc = check_stores(store, 1, pool->n_pages, pool->page_size))) return rc;
    if (total < 0 || total > 0x7FFFFFFFLL) return fail(KPOOL_ERR_INVALID_ARG, "total out of range");
    if (total > 0 && n == 0) return fail(KPOOL_ERR_INVALID_ARG, "rows without a sequence");
    if (total > 0 && !rows) return fail(KPOOL_ERR_INVALID_ARG, "rows are required");
    if (!aligned(rows, 16) || rows_layer_stride % 16 != 0)
        return fail(KPOOL_ERR_INVALID_ARG, "rows must be 16-byte aligned in every layer");
    if (rows_layer_stride < 0 || (store->n_layers > 1 && rows_layer_stride < total * store->row_bytes))
        return fail(KPOOL_ERR_INVALID_ARG, "rows_layer_stride is less than a layer's rows");
    if ((rc = check_pages_workspace(workspace, workspace_bytes, n, pool->n_seqs, pool->n_pages))) return rc;
    return run_pages_write(*pool, seqs, begin, cu_rows, static_cast<int>(n), total, rows, rows_layer_stride, *store,
                           workspace, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_pages_free(const kpool_page_pool *pool, const int32_t *seqs, int64_t n, void *workspace,
                     size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_pages_free");
    int rc = check_pool(pool);
    if (rc) return rc;
    if ((rc = check_items(n, {seqs}))) return rc;
    if ((rc = check_pages_workspace(workspace, workspace_bytes, n, pool->n_seqs, pool->n_pages))) return rc;
    if (n == 0) return nothing_listed(workspace, stream);
    return run_pages_free(*pool, seqs, static_cast<int>(n), workspace, reinterpret_cast<cudaStream_t>(stream));
}

int kpool_pages_compact(const kpool_page_pool *pool, const kpool_page_store *stores, int n_stores, void *workspace,
                        size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_pages_compact");
    int rc = check_pool(pool);
    if (rc) return rc;
    if ((rc = check_stores(stores, n_stores, pool->n_pages, pool->page_size))) return rc;
    if ((rc = check_pages_workspace(workspace, workspace_bytes, 0, pool->n_seqs, pool->n_pages))) return rc;
    return run_pages_compact(*pool, stores, n_stores, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t kpool_shared_prefix_mla_workspace_size(int64_t Tq, int H, int B, int G)
{
    if (Tq < 0 || H < 1 || H > 128 || Tq * H > 0x7FFFFFFFLL || B < 0 || B > (1 << 24) || G < 0 || G > (1 << 24))
        return 0;
    return prefix_mla_workspace_bytes(Tq, H, B, G);
}

int kpool_shared_prefix_mla_fwd(const void *q, const void *kv, int64_t kv_page_stride, int n_pages, int page_size,
                                const int32_t *page_table, const int32_t *seq_lens, int n_rows, int max_pages,
                                const int32_t *seq_ids, const int32_t *cu_seqlens_q, int B,
                                const int32_t *cu_groups, const int32_t *prefix_lens, int G, int64_t Tq, int H,
                                int Dc, float softmax_scale, void *o_out, float *lse_out, void *workspace,
                                size_t workspace_bytes, kpool_stream_t stream)
{
    clear_error();
    KPOOL_NVTX_RANGE("kpool_shared_prefix_mla_fwd");
    if (H < 1 || H > 128 || Dc != 512)
        return fail(KPOOL_ERR_UNSUPPORTED, "built for 1 <= H <= 128, Dc = 512 (got H = %d, Dc = %d)", H, Dc);
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return fail(KPOOL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128 (got %d)", page_size);
    if (Tq < 0 || Tq * H > 0x7FFFFFFFLL) return fail(KPOOL_ERR_INVALID_ARG, "Tq out of range");
    if (B < 1 || B > (1 << 24) || G < 1 || G > (1 << 24))
        return fail(KPOOL_ERR_INVALID_ARG, "B and G must be 1 .. 2^24");
    if (n_rows < 1 || max_pages < 1 || max_pages > (1 << 20))
        return fail(KPOOL_ERR_INVALID_ARG, "n_rows must be >= 1 and max_pages 1 .. 2^20");
    if (!seq_ids && n_rows < B) return fail(KPOOL_ERR_INVALID_ARG, "without seq_ids, n_rows must be >= B");
    if (n_pages < 1 || n_pages > (1 << 28)) return fail(KPOOL_ERR_INVALID_ARG, "n_pages out of range");
    if (kv_page_stride < static_cast<int64_t>(page_size) * Dc || kv_page_stride % 8 != 0 ||
        kv_page_stride >= (int64_t(1) << 39))
        return fail(KPOOL_ERR_INVALID_ARG, "kv_page_stride must be a multiple of 8 of at least a page's elements");
    if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
        return fail(KPOOL_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
    if (Tq > 0 && (!q || !o_out || !lse_out))
        return fail(KPOOL_ERR_INVALID_ARG, "q, o_out and lse_out are required");
    if (!kv || !page_table || !seq_lens || !cu_seqlens_q || !cu_groups || !prefix_lens)
        return fail(KPOOL_ERR_INVALID_ARG,
                    "kv, page_table, seq_lens, cu_seqlens_q, cu_groups and prefix_lens are required");
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(o_out, 16) || !aligned(lse_out, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "q, kv and o_out must be 16-byte aligned");
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(seq_ids, 4) || !aligned(cu_seqlens_q, 4) ||
        !aligned(cu_groups, 4) || !aligned(prefix_lens, 4))
        return fail(KPOOL_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
    const size_t need = prefix_mla_workspace_bytes(Tq, H, B, G);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
        return fail(KPOOL_ERR_WORKSPACE, "workspace of at least %zu bytes, 256-byte aligned, needed", need);
    PrefixMlaArgs a{};
    a.q = q; a.kv = kv; a.kv_page_stride = kv_page_stride; a.n_pages = n_pages; a.page_size = page_size;
    a.page_table = page_table; a.seq_lens = seq_lens; a.n_rows = n_rows; a.max_pages = max_pages;
    a.seq_ids = seq_ids; a.cu_q = cu_seqlens_q; a.B = B; a.cu_groups = cu_groups; a.prefix_lens = prefix_lens;
    a.G = G; a.Tq = Tq; a.H = H; a.scale = softmax_scale; a.o = o_out; a.lse = lse_out; a.workspace = workspace;
    return run_prefix_mla(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

"""Python binding of libkpool.so (the GB300-native KPool DSA indexer).

Thin ctypes marshalling over the C ABI declared in ``include/kpool.h``: each
function checks dtypes/devices, allocates outputs with torch (device memory
and streams are torch's job here), and calls the C entry point of the same
name on the current CUDA stream.  Every step of the computation runs in the
library's CUDA kernels; there is no fallback of any kind -- importing this
module fails loudly if ``libkpool.so`` has not been built.

Sources (page titles and sections): Megatron-LM PR "GLM5.3 Flash (KDA + mHC +
KPool DSA) support + FP8", Changes section 3 "KPool DSA indexer + NoPE";
SkyRL PR "GLM-5.3-Flash (glm5_next) Megatron support", commit "k-pool
indexer"; xtuner PR "GLM-5.3-Flash F5: NoPE DSA + KPool indexer".
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkpool.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libkpool.so is not built (expected at %s); run "
        "`python -c \"import __graft_entry__ as g; g.build()\"` or "
        "`python sparse_attention_kpool_compress_gb300/build.py`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_SZ = ctypes.c_size_t

_SIGS = {
    "kpool_last_error": (ctypes.c_char_p, []),
    "kpool_version": (_I, []),
    "kpool_num_pools": (_I, [_P, _I, _L, _I, _P, _P]),
    "kpool_cu_pools": (_I, [_P, _I, _I, _P, _P]),
    "kpool_compress": (_I, [_P, _P, _P, _P, _P, _I, _L, _I, _I, _L, _P, _P, _P, _P]),
    "kpool_quantize_fp8": (_I, [_P, _L, _I, _P, _P, _P]),
    "kpool_project_compress": (_I, [_P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _I, _L, _I, _I,
                                    _I, _L, _P, _P, _P, _P, _SZ, _P]),
    "kpool_score_topk_workspace_size": (_SZ, [_L, _I, _I]),
    "kpool_score_topk_workspace_size_split": (_SZ, [_L, _I, _I, _I, _I]),
    "kpool_score_topk": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _L, _L, _I, _I, _I, _I, _I,
                              _P, _P, _P, _SZ, _P]),
    "kpool_score_topk_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _L, _L, _I, _I, _I, _I,
                                      _I, _P, _P, _P]),
    "kpool_score_dense": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _L, _L, _I, _I, _I, _I,
                               _P, _P, _SZ, _P]),
    "kpool_expand_indices": (_I, [_P, _P, _P, _I, _L, _I, _I, _I, _P, _P]),
    "kpool_score_topk_at": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _L, _L, _I, _I, _I, _I, _I,
                                 _P, _P, _P, _SZ, _P]),
    "kpool_expand_indices_at": (_I, [_P, _P, _P, _P, _P, _I, _L, _I, _I, _I, _P, _P]),
    "kpool_sparse_mla_workspace_size": (_SZ, []),
    "kpool_sparse_mla_fwd": (_I, [_P, _P, _P, _L, _L, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                  _SZ, _P]),
    "kpool_sparse_mla_fwd_pools": (_I, [_P, _P, _P, _P, _P, _I, _L, _I, _I, _I, _I, _I,
                                        ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "kpool_sparse_mla_fwd_pools_at": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _L, _L, _I, _I, _I,
                                           _I, _I, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "kpool_sparse_mla_bwd_workspace_size": (_SZ, [_L, _L]),
    "kpool_sparse_mla_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _L, _L, _I, _I, _I, ctypes.c_float,
                                  _P, _P, _P, _SZ, _P]),
    "kpool_sparse_mla_bwd_pools": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _L, _I, _I, _I,
                                        _I, _I, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "kpool_sparse_mla_bwd_pools_at": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _L, _L,
                                           _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P, _SZ,
                                           _P]),
    "kpool_sparse_mla_paged_workspace_size": (_SZ, [_L, _I, _I]),
    "kpool_sparse_mla_fwd_pools_paged": (_I, [_P, _P, _L, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P,
                                              _P, _I, _L, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                                              _P, _P, _SZ, _P]),
    "kpool_pages_workspace_size": (_SZ, [_L, _I, _I]),
    "kpool_pages_copy": (_I, [_P, _P, _L, _I, _P, _I, _P, _SZ, _P]),
    "kpool_pages_fork": (_I, [_P, _P, _P, _L, _P, _I, _P, _SZ, _P]),
    "kpool_pages_extend": (_I, [_P, _P, _P, _L, _P, _P, _SZ, _P]),
    "kpool_pages_write": (_I, [_P, _P, _P, _P, _L, _L, _P, _L, _P, _P, _SZ, _P]),
    "kpool_pages_free": (_I, [_P, _P, _L, _P, _SZ, _P]),
    "kpool_pages_compact": (_I, [_P, _P, _I, _P, _SZ, _P]),
    "kpool_shared_prefix_mla_workspace_size": (_SZ, [_L, _I, _I, _I]),
    "kpool_shared_prefix_mla_fwd": (_I, [_P, _P, _L, _I, _I, _P, _P, _I, _I, _P, _P, _I, _P, _P,
                                         _I, _L, _I, _I, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "kpool_read_status": (_I, [_P, _P]),
    "kpool_score_topk_noalloc_status": (_I, [_P]),
    "kpool_debug_set_wait_limit_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
    "kpool_indexer_forward_host_scratch_size": (_SZ, [_P, _I, _L, _I, _I, _I, _I, _I, _L]),
    "kpool_indexer_forward_host": (_I, [_P, _P, _P, _P, _P, _P, _I, _L, _I, _I, _I, _I, _I, _I,
                                        _L, _P, _P, _SZ, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

STATUS_TIMEOUT = 1
STATUS_BAD_SEQLENS = 2
STATUS_BAD_PAGE = 4
STATUS_NO_PAGES = 8


class KPoolError(RuntimeError):
    def __init__(self, code, fn):
        msg = _lib.kpool_last_error().decode(errors="replace")
        super().__init__("%s failed (%d): %s" % (fn, code, msg))
        self.code = code


def _check(rc, fn):
    if rc != 0:
        raise KPoolError(rc, fn)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype=None, device=True):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if device and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)


def _as_u8(t):
    if t is None:
        return None
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


def _docs(cu_seqlens, cu_pools):
    if cu_seqlens is None:
        if cu_pools is not None:
            raise ValueError("cu_pools given without cu_seqlens")
        return 1
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    _need(cu_pools, "cu_pools", torch.int32)
    return cu_seqlens.numel() - 1


# ---------------------------------------------------------------------------

def kpool_version() -> int:
    return int(_lib.kpool_version())


def kpool_num_pools(cu_seqlens_host, T: int, kpool: int):
    """Host helper: (cu_pools int32 CPU tensor, total pools) from a host
    cu_seqlens (list or CPU int32 tensor).  Validates the layout."""
    cs = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous().cpu()
    out = torch.empty_like(cs)
    total = ctypes.c_int64(0)
    _check(_lib.kpool_num_pools(_ptr(cs), cs.numel() - 1, T, kpool, _ptr(out),
                                ctypes.byref(total)), "kpool_num_pools")
    return out, int(total.value)


def kpool_cu_pools(cu_seqlens: torch.Tensor, kpool: int) -> torch.Tensor:
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    out = torch.empty_like(cu_seqlens)
    _check(_lib.kpool_cu_pools(_ptr(cu_seqlens), cu_seqlens.numel() - 1, kpool, _ptr(out),
                               _stream(cu_seqlens.device)), "kpool_cu_pools")
    return out


def kpool_compress(k, gate, ape, kpool: int, cu_seqlens=None, cu_pools=None, P_total=None,
                   fp8: bool = False, out=None):
    """Pooled keys pk [P_total, D] bf16 (plus E4M3 codes and scales when
    fp8).  For packed documents pass device cu_seqlens/cu_pools and P_total."""
    _need(k, "k", torch.bfloat16)
    _need(gate, "gate", torch.bfloat16)
    _need(ape, "ape", torch.float32)
    n_docs = _docs(cu_seqlens, cu_pools)
    T, D = k.shape
    if P_total is None:
        if cu_seqlens is not None:
            raise ValueError("P_total is required with cu_seqlens")
        P_total = T // kpool
    pk = out if out is not None else torch.empty(P_total, D, dtype=torch.bfloat16,
                                                 device=k.device)
    pk8 = sc = None
    if fp8:
        pk8 = torch.empty(P_total, D, dtype=torch.uint8, device=k.device)
        sc = torch.empty(P_total, dtype=torch.float32, device=k.device)
    _check(_lib.kpool_compress(_ptr(k), _ptr(gate), _ptr(ape), _ptr(cu_seqlens), _ptr(cu_pools),
                               n_docs, T, D, kpool, P_total, _ptr(pk), _ptr(pk8), _ptr(sc),
                               _stream(k.device)), "kpool_compress")
    return (pk, pk8, sc) if fp8 else pk


def kpool_project_compress(x, w_kg, k_norm_weight, k_norm_bias, k_norm_eps: float, ape,
                           kpool: int, cu_seqlens=None, cu_pools=None, P_total=None,
                           want_k_gate: bool = False, workspace=None):
    """Pooled keys pk [P_total, 128] bf16 straight from hidden states x [T,
    hidden] (key projection, k_norm, gate projection and compression in one
    kernel); with want_k_gate also the projected keys and gate [T, 128]."""
    _need(x, "x", torch.bfloat16)
    _need(w_kg, "w_kg", torch.bfloat16)
    for t_, n_ in ((k_norm_weight, "k_norm_weight"), (k_norm_bias, "k_norm_bias"), (ape, "ape")):
        _need(t_, n_, torch.float32)
    n_docs = _docs(cu_seqlens, cu_pools)
    T, hidden = x.shape
    D = w_kg.shape[0] // 2
    if P_total is None:
        if cu_seqlens is not None:
            raise ValueError("P_total is required with cu_seqlens")
        P_total = T // kpool
    pk = torch.empty(P_total, D, dtype=torch.bfloat16, device=x.device)
    k_out = g_out = None
    if want_k_gate:
        k_out = torch.empty(T, D, dtype=torch.bfloat16, device=x.device)
        g_out = torch.empty(T, D, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=x.device)
    _check(_lib.kpool_project_compress(_ptr(x), _ptr(w_kg), _ptr(k_norm_weight),
                                       _ptr(k_norm_bias), float(k_norm_eps), _ptr(ape),
                                       _ptr(cu_seqlens), _ptr(cu_pools), n_docs, T, hidden, D,
                                       kpool, P_total, _ptr(pk), _ptr(k_out), _ptr(g_out),
                                       _ptr(workspace), workspace.numel(), _stream(x.device)),
           "kpool_project_compress")
    return (pk, k_out, g_out) if want_k_gate else pk


def kpool_quantize_fp8(x):
    """x bf16 [..., 128] -> (E4M3 codes uint8 [..., 128], fp32 scales [...])."""
    _need(x, "x", torch.bfloat16)
    D = x.shape[-1]
    rows = x.numel() // D
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check(_lib.kpool_quantize_fp8(_ptr(x), rows, D, _ptr(codes), _ptr(sc), _stream(x.device)),
           "kpool_quantize_fp8")
    return codes, sc


def kpool_score_topk_workspace_size(T: int, H: int, n_docs: int = 1) -> int:
    return int(_lib.kpool_score_topk_workspace_size(T, H, n_docs))


def kpool_score_topk_workspace_size_split(T: int, H: int, n_docs: int, kpool: int,
                                          index_topk: int) -> int:
    return int(_lib.kpool_score_topk_workspace_size_split(T, H, n_docs, kpool, index_topk))


def new_workspace(T: int, H: int, n_docs: int = 1, device="cuda", kpool: int | None = None,
                  index_topk: int | None = None) -> torch.Tensor:
    """Workspace for kpool_score_topk[_at]; with kpool and index_topk it is
    large enough for the split-pool schedule of calls with few query tiles."""
    if kpool is not None and index_topk is not None:
        n = kpool_score_topk_workspace_size_split(T, H, n_docs, kpool, index_topk)
    else:
        n = kpool_score_topk_workspace_size(T, H, n_docs)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _score_common(q, w, pk, q_scale, pk_scale, cu_seqlens, cu_pools):
    fp8 = q_scale is not None
    if fp8:
        _need(q, "q", (torch.uint8, torch.float8_e4m3fn))
        _need(pk, "pk", (torch.uint8, torch.float8_e4m3fn))
        _need(q_scale, "q_scale", torch.float32)
        _need(pk_scale, "pk_scale", torch.float32)
    else:
        _need(q, "q", torch.bfloat16)
        _need(pk, "pk", torch.bfloat16)
    _need(w, "w", torch.float32)
    n_docs = _docs(cu_seqlens, cu_pools)
    T, H, D = q.shape
    return fp8, n_docs, T, H, D, pk.shape[0]


def kpool_score_topk(q, w, pk, kpool: int, index_topk: int, cu_seqlens=None, cu_pools=None,
                     q_scale=None, pk_scale=None, workspace=None, out=None):
    """(pool_idx int32 [T, Kp], pool_score fp32 [T, Kp]) -- ascending pools,
    -1 / -inf padded."""
    fp8, n_docs, T, H, D, P = _score_common(q, w, pk, q_scale, pk_scale, cu_seqlens, cu_pools)
    Kp = index_topk // kpool
    if workspace is None:
        workspace = new_workspace(T, H, n_docs, q.device, kpool, index_topk)
    if out is None:
        idx = torch.empty(T, Kp, dtype=torch.int32, device=q.device)
        sc = torch.empty(T, Kp, dtype=torch.float32, device=q.device)
    else:
        idx, sc = out
    _check(_lib.kpool_score_topk(_ptr(_as_u8(q)) if fp8 else _ptr(q), _ptr(q_scale), _ptr(w),
                                 _ptr(_as_u8(pk)) if fp8 else _ptr(pk), _ptr(pk_scale),
                                 _ptr(cu_seqlens), _ptr(cu_pools), n_docs, T, P, H, D, kpool,
                                 index_topk, int(fp8), _ptr(idx), _ptr(sc), _ptr(workspace),
                                 workspace.numel(), _stream(q.device)), "kpool_score_topk")
    return idx, sc


def kpool_score_topk_noalloc(q, w, pk, kpool: int, index_topk: int, cu_seqlens=None,
                             cu_pools=None, q_scale=None, pk_scale=None, out=None):
    """kpool_score_topk without a workspace: the library's fixed scratch
    array stands in for it (see include/kpool.h for its limits)."""
    fp8, n_docs, T, H, D, P = _score_common(q, w, pk, q_scale, pk_scale, cu_seqlens, cu_pools)
    Kp = index_topk // kpool
    if out is None:
        idx = torch.empty(T, Kp, dtype=torch.int32, device=q.device)
        sc = torch.empty(T, Kp, dtype=torch.float32, device=q.device)
    else:
        idx, sc = out
    _check(_lib.kpool_score_topk_noalloc(_ptr(_as_u8(q)) if fp8 else _ptr(q), _ptr(q_scale),
                                         _ptr(w), _ptr(_as_u8(pk)) if fp8 else _ptr(pk),
                                         _ptr(pk_scale), _ptr(cu_seqlens), _ptr(cu_pools), n_docs,
                                         T, P, H, D, kpool, index_topk, int(fp8), _ptr(idx),
                                         _ptr(sc), _stream(q.device)),
           "kpool_score_topk_noalloc")
    return idx, sc


def kpool_score_dense(q, w, pk, kpool: int, cu_seqlens=None, cu_pools=None, q_scale=None,
                      pk_scale=None, workspace=None):
    """Test/debug: full fp32 [T, P] scores (-inf where not a causal pool)."""
    fp8, n_docs, T, H, D, P = _score_common(q, w, pk, q_scale, pk_scale, cu_seqlens, cu_pools)
    if workspace is None:
        workspace = new_workspace(T, H, n_docs, q.device)
    out = torch.empty(T, P, dtype=torch.float32, device=q.device)
    _check(_lib.kpool_score_dense(_ptr(_as_u8(q)) if fp8 else _ptr(q), _ptr(q_scale), _ptr(w),
                                  _ptr(_as_u8(pk)) if fp8 else _ptr(pk), _ptr(pk_scale),
                                  _ptr(cu_seqlens), _ptr(cu_pools), n_docs, T, P, H, D, kpool,
                                  int(fp8), _ptr(out), _ptr(workspace), workspace.numel(),
                                  _stream(q.device)), "kpool_score_dense")
    return out


def kpool_expand_indices(pool_idx, kpool: int, index_topk: int, always_select_tail: bool = True,
                         cu_seqlens=None, cu_pools=None, out=None):
    """Token indices int32 [T, Kp*kpool + kpool - 1], ascending, -1 padded."""
    _need(pool_idx, "pool_idx", torch.int32)
    n_docs = _docs(cu_seqlens, cu_pools)
    T = pool_idx.shape[0]
    Kp = index_topk // kpool
    W = Kp * kpool + kpool - 1
    tok = out if out is not None else torch.empty(T, W, dtype=torch.int32, device=pool_idx.device)
    _check(_lib.kpool_expand_indices(_ptr(pool_idx), _ptr(cu_seqlens), _ptr(cu_pools), n_docs, T,
                                     kpool, index_topk, int(bool(always_select_tail)), _ptr(tok),
                                     _stream(pool_idx.device)), "kpool_expand_indices")
    return tok


def kpool_score_topk_at(q, w, pk, kpool: int, index_topk: int, cu_seqlens_q, q_start_pos,
                        cu_pools, q_scale=None, pk_scale=None, workspace=None, out=None):
    """Positioned queries (decode / chunked prefill): document d's query rows
    [cu_seqlens_q[d], cu_seqlens_q[d+1]) sit at positions q_start_pos[d] + i."""
    fp8, n_docs, T, H, D, P = _score_common(q, w, pk, q_scale, pk_scale, cu_seqlens_q, cu_pools)
    _need(q_start_pos, "q_start_pos", torch.int32)
    Kp = index_topk // kpool
    if workspace is None:
        workspace = new_workspace(T, H, n_docs, q.device, kpool, index_topk)
    if out is None:
        idx = torch.empty(T, Kp, dtype=torch.int32, device=q.device)
        sc = torch.empty(T, Kp, dtype=torch.float32, device=q.device)
    else:
        idx, sc = out
    _check(_lib.kpool_score_topk_at(_ptr(_as_u8(q)) if fp8 else _ptr(q), _ptr(q_scale), _ptr(w),
                                    _ptr(_as_u8(pk)) if fp8 else _ptr(pk), _ptr(pk_scale),
                                    _ptr(cu_seqlens_q), _ptr(q_start_pos), _ptr(cu_pools), n_docs,
                                    T, P, H, D, kpool, index_topk, int(fp8), _ptr(idx), _ptr(sc),
                                    _ptr(workspace), workspace.numel(), _stream(q.device)),
           "kpool_score_topk_at")
    return idx, sc


def kpool_expand_indices_at(pool_idx, kpool: int, index_topk: int, cu_seqlens_q, q_start_pos,
                            cu_seqlens_k, cu_pools, always_select_tail: bool = True, out=None):
    """Key-token indices for positioned queries [Tq, Kp*kpool + kpool - 1]."""
    _need(pool_idx, "pool_idx", torch.int32)
    for t_, n_ in ((cu_seqlens_q, "cu_seqlens_q"), (q_start_pos, "q_start_pos"),
                   (cu_seqlens_k, "cu_seqlens_k"), (cu_pools, "cu_pools")):
        _need(t_, n_, torch.int32)
    T = pool_idx.shape[0]
    Kp = index_topk // kpool
    W = Kp * kpool + kpool - 1
    tok = out if out is not None else torch.empty(T, W, dtype=torch.int32, device=pool_idx.device)
    _check(_lib.kpool_expand_indices_at(_ptr(pool_idx), _ptr(cu_seqlens_q), _ptr(q_start_pos),
                                        _ptr(cu_seqlens_k), _ptr(cu_pools), cu_seqlens_q.numel() - 1,
                                        T, kpool, index_topk, int(bool(always_select_tail)),
                                        _ptr(tok), _stream(pool_idx.device)),
           "kpool_expand_indices_at")
    return tok


def kpool_sparse_mla_workspace_size() -> int:
    return int(_lib.kpool_sparse_mla_workspace_size())


def _mla_outputs(q, workspace, o, lse):
    T, H, Dc = q.shape
    if o is None:
        o = torch.empty(T, H, Dc, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(T, H, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(kpool_sparse_mla_workspace_size(), dtype=torch.uint8,
                                device=q.device)
    return o, lse, workspace


def kpool_sparse_mla_fwd(q, kv, tok_idx, softmax_scale: float, workspace=None, o=None, lse=None):
    """Sparse attention over explicit token lists: q bf16 [T, 64, 512], kv bf16
    [Tk, 512], tok_idx int32 [T, W] (-1 = none) -> (o bf16 [T, 64, 512], lse
    fp32 [T, 64])."""
    _need(q, "q", torch.bfloat16)
    _need(kv, "kv", torch.bfloat16)
    _need(tok_idx, "tok_idx", torch.int32)
    T, H, Dc = q.shape
    o, lse, workspace = _mla_outputs(q, workspace, o, lse)
    _check(_lib.kpool_sparse_mla_fwd(_ptr(q), _ptr(kv), _ptr(tok_idx), T, kv.shape[0],
                                     tok_idx.shape[1], H, Dc, float(softmax_scale), _ptr(o),
                                     _ptr(lse), _ptr(workspace), workspace.numel(),
                                     _stream(q.device)), "kpool_sparse_mla_fwd")
    return o, lse


def kpool_sparse_mla_fwd_pools(q, kv, pool_idx, kpool: int, index_topk: int,
                               softmax_scale: float, cu_seqlens=None, cu_pools=None,
                               always_select_tail: bool = True, workspace=None, o=None, lse=None):
    """Sparse attention fused with the expansion of pool_idx [T, index_topk //
    kpool] (keys = the query tokens, kv bf16 [T, 512])."""
    _need(q, "q", torch.bfloat16)
    _need(kv, "kv", torch.bfloat16)
    _need(pool_idx, "pool_idx", torch.int32)
    n_docs = _docs(cu_seqlens, cu_pools)
    T, H, Dc = q.shape
    o, lse, workspace = _mla_outputs(q, workspace, o, lse)
    _check(_lib.kpool_sparse_mla_fwd_pools(_ptr(q), _ptr(kv), _ptr(pool_idx), _ptr(cu_seqlens),
                                           _ptr(cu_pools), n_docs, T, H, Dc, kpool, index_topk,
                                           int(bool(always_select_tail)), float(softmax_scale),
                                           _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                           _stream(q.device)), "kpool_sparse_mla_fwd_pools")
    return o, lse


def kpool_sparse_mla_fwd_pools_at(q, kv, pool_idx, kpool: int, index_topk: int,
                                  softmax_scale: float, cu_seqlens_q, q_start_pos, cu_seqlens_k,
                                  cu_pools, always_select_tail: bool = True, workspace=None,
                                  o=None, lse=None):
    """kpool_sparse_mla_fwd_pools for positioned queries (keys kv [Tk, 512])."""
    _need(q, "q", torch.bfloat16)
    _need(kv, "kv", torch.bfloat16)
    _need(pool_idx, "pool_idx", torch.int32)
    for t_, n_ in ((cu_seqlens_q, "cu_seqlens_q"), (q_start_pos, "q_start_pos"),
                   (cu_seqlens_k, "cu_seqlens_k"), (cu_pools, "cu_pools")):
        _need(t_, n_, torch.int32)
    T, H, Dc = q.shape
    o, lse, workspace = _mla_outputs(q, workspace, o, lse)
    _check(_lib.kpool_sparse_mla_fwd_pools_at(
        _ptr(q), _ptr(kv), _ptr(pool_idx), _ptr(cu_seqlens_q), _ptr(q_start_pos),
        _ptr(cu_seqlens_k), _ptr(cu_pools), cu_seqlens_q.numel() - 1, T, kv.shape[0], H, Dc,
        kpool, index_topk, int(bool(always_select_tail)), float(softmax_scale), _ptr(o),
        _ptr(lse), _ptr(workspace), workspace.numel(), _stream(q.device)),
        "kpool_sparse_mla_fwd_pools_at")
    return o, lse


# ---- paged cache ------------------------------------------------------------

class _Pool(ctypes.Structure):
    _fields_ = [("page_table", _P), ("seq_lens", _P), ("ref_count", _P), ("free_list", _P),
                ("free_count", _P), ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


# The calls below are short on the GPU, so the host's part is kept short as well:
# one combined test per tensor (the messages are made only when it fails), raw
# pointers and streams, structures packed in one go.
# (a CPU build of torch has no streams; the host-only calls work there)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_pack_store = struct.Struct("@Pqqiiii").pack
_I32 = torch.int32


def _same_device(index, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s is on %s, not on cuda:%d" % (name, t.device, index))


def _ints(t, name, n, index):
    """Address of a contiguous int32 tensor of n entries on CUDA device `index`."""
    if not (t.dtype is _I32 and t.is_cuda and t.get_device() == index and t.numel() == n
            and t.is_contiguous()):
        _need(t, name, _I32)
        _same_device(index, **{name: t})
        raise ValueError("%s must have %d entries (got %d)" % (name, n, t.numel()))
    return t.data_ptr()


def _device_of(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.get_device()


def _call(index, name, fn, *args):
    """fn(*args, stream) on device `index` and its current stream."""
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        raise KPoolError(rc, name)


@functools.lru_cache(maxsize=None)
def _devices(index):
    return torch.device("cuda", index)


def _bytes(workspace, size, index):
    """(tensor, address, size) of a call's workspace: the caller's, or a new one."""
    if workspace is None:
        workspace = torch.empty(max(256, size), dtype=torch.uint8, device=_devices(index))
    elif not (workspace.is_cuda and workspace.get_device() == index
              and workspace.dtype is torch.uint8 and workspace.is_contiguous()):
        _need(workspace, "workspace", torch.uint8)
        _same_device(index, workspace=workspace)
    return workspace, workspace.data_ptr(), workspace.numel()


class KPoolPages:
    """Which pages the sequences of a paged cache hold: page_table int32
    [n_seqs, max_pages], seq_lens [n_seqs], ref_count [n_pages], free_list
    [n_pages] and free_count [1], CUDA tensors of one device that the
    kpool_pages_* calls read and change in place (include/kpool.h,
    kpool_page_pool).  kpool_pages_new makes an empty one.  `workspace` is the
    one that calls on this pool use unless they are given another (calls on a
    pool are ordered anyway); kpool_read_status(pages.workspace) tells how the
    last of them went.  (kpool_pages_copy is a call on stores, not on a pool.)
    Calls may run on another stream than the one that the pool was made on: the
    first there waits until the workspace is made (in a capture, what begins it
    has to; torch.cuda.graph does), and its memory goes to nobody else before
    they have ended."""

    __slots__ = ("page_table", "seq_lens", "ref_count", "free_list", "free_count", "page_size",
                 "n_seqs", "n_pages", "workspace", "_index", "_c", "_at", "_ws", "_most",
                 "_streams", "_made")

    def __init__(self, page_table, seq_lens, ref_count, free_list, free_count, page_size: int):
        arrays = dict(page_table=page_table, seq_lens=seq_lens, ref_count=ref_count,
                      free_list=free_list, free_count=free_count)
        for name, t in arrays.items():
            _need(t, name, torch.int32)
        _same_device(page_table.get_device(), **arrays)
        if page_table.dim() != 2 or seq_lens.numel() != page_table.shape[0]:
            raise ValueError("page_table must be [n_seqs, max_pages] and seq_lens [n_seqs]")
        if ref_count.numel() != free_list.numel() or free_count.numel() != 1:
            raise ValueError("ref_count and free_list must be [n_pages] and free_count [1]")
        page_size = int(page_size)
        if page_size < 1:
            raise ValueError("page_size must be >= 1")
        put = super().__setattr__
        for name, t in arrays.items():
            put(name, t)
        put("page_size", page_size)
        put("n_seqs", page_table.shape[0])
        put("n_pages", ref_count.numel())
        put("_index", page_table.get_device())
        put("_c", _Pool(page_table.data_ptr(), seq_lens.data_ptr(), ref_count.data_ptr(),
                        free_list.data_ptr(), free_count.data_ptr(), page_table.shape[0],
                        page_table.shape[1], ref_count.numel(), page_size))
        put("_at", ctypes.addressof(self._c))
        # (enough for every list that names each sequence once)
        put("_most", max(self.n_pages, self.n_seqs))
        put("workspace", torch.zeros(
            max(256, _lib.kpool_pages_workspace_size(self._most, self.n_seqs, self.n_pages)),
            dtype=torch.uint8, device=page_table.device))
        put("_ws", (self.workspace, self.workspace.data_ptr(), self.workspace.numel()))
        put("_streams", {_raw_stream(self._index)})
        with torch.cuda.device(self._index):
            put("_made", None if torch.cuda.is_current_stream_capturing() else
                torch.cuda.current_stream().record_event())

    def __setattr__(self, name, value):
        raise AttributeError("a KPoolPages keeps its tensors: make another one")


def kpool_pages_new(n_seqs: int, n_pages: int, max_pages: int, page_size: int,
                    device="cuda") -> KPoolPages:
    """An empty pool: every page free (page 0 is taken first), no sequence
    holding any."""
    kw = dict(dtype=torch.int32, device=device)
    return KPoolPages(torch.full((n_seqs, max_pages), -1, **kw), torch.zeros(n_seqs, **kw),
                      torch.zeros(n_pages, **kw), torch.arange(n_pages - 1, -1, -1, **kw),
                      torch.full((1,), n_pages, **kw), page_size)


def _store(t, n_pages, index):
    """A kpool_page_store, packed."""
    shape, stride = t.shape, t.stride()
    dim = len(shape)
    if dim != 3 and dim != 4:
        raise ValueError("a store is [layers, n_pages, rows, width] or [n_pages, rows, width]")
    rows, width = shape[-2], shape[-1]
    if not t.is_cuda:
        raise ValueError("a store must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError("a store is on %s, not on cuda:%d" % (t.device, index))
    if shape[-3] != n_pages:
        raise ValueError("a store has %d pages, not %d" % (shape[-3], n_pages))
    if (width > 1 and stride[-1] != 1) or (rows > 1 and stride[-2] != width):
        raise ValueError("the rows of a store's page must be contiguous")
    size = t.element_size()
    return _pack_store(t.data_ptr(), stride[0] * size if dim == 4 else 0, stride[-3] * size,
                       shape[0] if dim == 4 else 1, rows, width * size, 0)


def _stores(stores, n_pages, index):
    """(packed array, count) of stores: tensors [layers, n_pages, rows, width] or
    [n_pages, rows, width] whose pages are contiguous, with layers and pages in
    either order of memory."""
    if isinstance(stores, torch.Tensor):
        return _store(stores, n_pages, index), 1
    return b"".join([_store(t, n_pages, index) for t in stores]), len(stores)


def kpool_pages_workspace_size(n: int, n_seqs: int, n_pages: int) -> int:
    return int(_lib.kpool_pages_workspace_size(n, n_seqs, n_pages))


def kpool_pages_copy(src, dst, stores, workspace=None):
    """Page dst[i] becomes a copy of page src[i] in every store and layer.  A
    list that is refused is told by the workspace alone (kpool_read_status): give
    one (256 bytes of uint8 up to 1024 pairs, else kpool_pages_workspace_size(n,
    0, n_pages)) to see whether it was."""
    first = stores if isinstance(stores, torch.Tensor) else stores[0] if len(stores) else None
    if first is None:
        raise ValueError("a store is required")
    index, n, n_pages = _device_of(src, "src"), src.numel(), first.shape[-3]
    a, b = _ints(src, "src", n, index), _ints(dst, "dst", n, index)
    st, n_stores = _stores(stores, n_pages, index)
    if workspace is None and n <= 1024:
        keep, ws, size = _status_words(index)
    else:
        keep, ws, size = _bytes(workspace, 0 if workspace is not None else
                                _lib.kpool_pages_workspace_size(n, 0, n_pages), index)
    _call(index, "kpool_pages_copy", _lib.kpool_pages_copy, a, b, n, n_pages, st, n_stores, ws,
          size)


@functools.lru_cache(maxsize=None)
def _status_words(index):
    """Workspace of calls that write a status word only, which nobody reads."""
    t = torch.zeros(256, dtype=torch.uint8, device=_devices(index))
    return t, t.data_ptr(), 256


def _join(pages):
    """The pool's own workspace is used on a stream that it was not made on."""
    with torch.cuda.device(pages._index):
        stream = torch.cuda.current_stream()
        pages.workspace.record_stream(stream)
        if not torch.cuda.is_current_stream_capturing():
            if pages._made is not None:
                stream.wait_event(pages._made)
            pages._streams.add(stream.cuda_stream)


def _pool_call(pages, workspace, n, name, fn, *args):
    """fn(*args, workspace, size, stream) over n items, in the pool's own workspace
    unless the caller gives one."""
    index = pages._index
    if workspace is None:
        stream = _raw_stream(index)
        if stream not in pages._streams:
            _join(pages)
        if n <= pages._most:
            _, ws, size = pages._ws
            if _current_device() != index:
                return _call(index, name, fn, *args, ws, size)
            rc = fn(*args, ws, size, stream)
            if rc:
                raise KPoolError(rc, name)
            return
    keep, ws, size = _bytes(workspace, 0 if workspace is not None else
                            _lib.kpool_pages_workspace_size(n, pages.n_seqs, pages.n_pages), index)
    _call(index, name, fn, *args, ws, size)
    if workspace is None:
        # a list with repetitions: how it went is told where the pool's calls tell it
        with torch.inference_mode():               # (the pool may have been made in it)
            pages.workspace[:16].copy_(keep[:16])


def kpool_pages_fork(pages: KPoolPages, parents, children, stores=(), workspace=None):
    """Sequence children[i], which holds nothing, becomes a copy of sequence
    parents[i]: whole pages are shared, a partial last page is copied."""
    index, n = pages._index, parents.numel()
    a, b = _ints(parents, "parents", n, index), _ints(children, "children", n, index)
    st, n_stores = _stores(stores, pages.n_pages, index)
    _pool_call(pages, workspace, n, "kpool_pages_fork",
               _lib.kpool_pages_fork, pages._at, a, b, n, st, n_stores)


def kpool_pages_extend(pages: KPoolPages, seqs, n_new, workspace=None, out=None):
    """Sequence seqs[i] grows by n_new[i] tokens -> its length before, int32
    [n] (-1 everywhere when the call is refused)."""
    index, n = pages._index, seqs.numel()
    a, b = _ints(seqs, "seqs", n, index), _ints(n_new, "n_new", n, index)
    if out is None:
        out = torch.empty(n, dtype=_I32, device=_devices(index))
    c = _ints(out, "out", n, index)
    _pool_call(pages, workspace, n, "kpool_pages_extend",
               _lib.kpool_pages_extend, pages._at, a, b, n, c)
    return out


def kpool_pages_write(pages: KPoolPages, seqs, begin, cu_rows, rows, store, workspace=None):
    """Rows cu_rows[i] .. cu_rows[i+1] - 1 of `rows` ([layers, total, width], or
    [total, width] for one layer) go to the rows begin[i], begin[i] + 1, ... of
    sequence seqs[i] in `store`."""
    index, n = pages._index, seqs.numel()
    a, b = _ints(seqs, "seqs", n, index), _ints(begin, "begin", n, index)
    c = _ints(cu_rows, "cu_rows", n + 1, index)
    if not (rows.dtype is store.dtype and rows.is_contiguous() and rows.get_device() == index):
        _need(rows, "rows", store.dtype)
        _same_device(index, rows=rows)
    st = _store(store, pages.n_pages, index)
    layers, width = store.shape[0] if store.dim() == 4 else 1, store.shape[-1]
    shape = rows.shape
    if len(shape) not in (2, 3) or (shape[0] if len(shape) == 3 else 1) != layers:
        raise ValueError("rows must be [layers, total, width] of the store's %d layers" % layers)
    if shape[-1] != width:
        raise ValueError("rows are %d wide, the store's %d" % (shape[-1], width))
    total = shape[-2]
    _pool_call(pages, workspace, n, "kpool_pages_write", _lib.kpool_pages_write, pages._at, a, b, c, n,
               total, rows.data_ptr(), total * width * rows.element_size(), st)


def kpool_pages_free(pages: KPoolPages, seqs, workspace=None):
    """The listed sequences give up their pages."""
    index, n = pages._index, seqs.numel()
    a = _ints(seqs, "seqs", n, index)
    _pool_call(pages, workspace, n, "kpool_pages_free", _lib.kpool_pages_free, pages._at, a, n)


def kpool_pages_compact(pages: KPoolPages, stores=(), workspace=None):
    """The k referenced pages move to the pages 0 .. k - 1, in every store."""
    index = pages._index
    st, n_stores = _stores(stores, pages.n_pages, index)
    _pool_call(pages, workspace, 0, "kpool_pages_compact",
               _lib.kpool_pages_compact, pages._at, st, n_stores)


def kpool_shared_prefix_mla_workspace_size(Tq: int, H: int, B: int, G: int) -> int:
    return int(_lib.kpool_shared_prefix_mla_workspace_size(Tq, H, B, G))


def kpool_shared_prefix_mla_fwd(q, kv, page_table, seq_lens, cu_seqlens_q, cu_groups, prefix_lens,
                                softmax_scale: float, seq_ids=None, workspace=None, o=None,
                                lse=None):
    """Attention over a paged latent cache for groups of sequences that share
    a prefix, read and multiplied once per group: q bf16 [Tq, H, 512], kv bf16
    [n_pages, page_size, 512] (one layer of a store) -> (o bf16 [Tq, H, 512],
    lse fp32 [Tq, H]).  A sequence's queries are its last tokens."""
    index, bf16 = _device_of(q, "q"), torch.bfloat16
    if not (q.dtype is bf16 and q.is_contiguous()):
        _need(q, "q", bf16)
    if kv.dtype is not bf16:
        raise TypeError("kv must be %s (got %s)" % (bf16, kv.dtype))
    n_pages, page_size, Dc = kv.shape
    stride = kv.stride()
    if kv.get_device() != index or stride[2] != 1 or stride[1] != Dc:
        _same_device(index, kv=kv)
        raise ValueError("the rows of a page of kv must be contiguous")
    Tq, H, D = q.shape
    if D != Dc:
        raise ValueError("q is %d wide, kv %d" % (D, Dc))
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_rows, max_pages]")
    n_rows, max_pages = page_table.shape
    B, G = cu_seqlens_q.numel() - 1, cu_groups.numel() - 1
    lists = (_ints(page_table, "page_table", n_rows * max_pages, index),
             _ints(seq_lens, "seq_lens", n_rows, index), n_rows, max_pages,
             None if seq_ids is None else _ints(seq_ids, "seq_ids", B, index),
             _ints(cu_seqlens_q, "cu_seqlens_q", B + 1, index), B,
             _ints(cu_groups, "cu_groups", G + 1, index),
             _ints(prefix_lens, "prefix_lens", G, index), G)
    if o is None:
        o = torch.empty_like(q)
    elif (o.shape != q.shape or o.dtype is not bf16 or not o.is_contiguous()
          or o.get_device() != index):
        _need(o, "o", bf16)
        _same_device(index, o=o)
        raise ValueError("o must be shaped like q")
    if lse is None:
        lse = torch.empty(Tq, H, dtype=torch.float32, device=_devices(index))
    elif (lse.numel() != Tq * H or lse.dtype is not torch.float32 or not lse.is_contiguous()
          or lse.get_device() != index):
        _need(lse, "lse", torch.float32)
        _same_device(index, lse=lse)
        raise ValueError("lse must be [Tq, H]")
    keep, ws, size = _bytes(workspace, 0 if workspace is not None else
                            _lib.kpool_shared_prefix_mla_workspace_size(Tq, H, B, G), index)
    # (the stride of a single page says nothing)
    _call(index, "kpool_shared_prefix_mla_fwd", _lib.kpool_shared_prefix_mla_fwd, q.data_ptr(),
          kv.data_ptr(), stride[0] if n_pages > 1 else page_size * Dc, n_pages, page_size, *lists,
          Tq, H, Dc, float(softmax_scale), o.data_ptr(), lse.data_ptr(), ws, size)
    return o, lse


# ---- sparse attention: backward pass, paged form --------------------------------

def _fits(t, shape, dtype, index):
    return t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous()


def _refuse(t, name, shape, dtype, index):
    """Says why `t` does not fit, if it does not."""
    if not _fits(t, shape, dtype, index):
        _need(t, name, dtype)
        _same_device(index, **{name: t})
        raise ValueError("%s must be %s (got %s)" % (name, tuple(shape), tuple(t.shape)))


def _output(t, name, shape, dtype, index):
    """`t`, checked, or a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=_devices(index))
    _refuse(t, name, shape, dtype, index)
    return t


def _list_rows(t, name, T, width, index):
    """Address of the lists int32 [T, width] (width None: any), and their width."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != T or (width is not None and shape[1] != width):
        raise ValueError("%s must be [%d, %s] (got %s)" % (name, T, "W" if width is None else width, tuple(shape)))
    return _ints(t, name, T * shape[1], index), shape[1]


def kpool_sparse_mla_bwd_workspace_size(T: int, Tk: int) -> int:
    return int(_lib.kpool_sparse_mla_bwd_workspace_size(T, Tk))


def _mla_sizes(q, kv):
    """(device index, T, Tk, H, Dc) of q [T, H, Dc] and kv [Tk, Dc]."""
    shape, rows = q.shape, kv.shape
    if len(shape) != 3 or len(rows) != 2 or rows[1] != shape[2]:
        raise ValueError("q must be [T, H, Dc] and kv [Tk, Dc] (got %s and %s)" % (tuple(shape), tuple(rows)))
    return _device_of(q, "q"), shape[0], rows[0], shape[1], shape[2]


def _mla_bwd(name, fn, index, q, kv, lists, o, lse, d_o, d_lse, sizes, softmax_scale, workspace, dq, dkv):
    """fn(q, kv, *lists, o, lse, d_o, d_lse, *sizes, scale, dq, dkv, workspace) -> (dq, dkv)"""
    bf16, f32, shape, rows = torch.bfloat16, torch.float32, q.shape, kv.shape
    T, heads = shape[0], shape[:2]
    if not (q.dtype is bf16 and kv.dtype is bf16 and o.dtype is bf16 and d_o.dtype is bf16 and lse.dtype is f32
            and q.is_contiguous() and kv.is_contiguous() and o.is_contiguous() and d_o.is_contiguous()
            and lse.is_contiguous() and o.shape == shape and d_o.shape == shape and lse.shape == heads
            and kv.get_device() == index and o.get_device() == index and d_o.get_device() == index
            and lse.get_device() == index and (d_lse is None or _fits(d_lse, heads, f32, index))):
        for t, n, want, dtype in ((q, "q", shape, bf16), (kv, "kv", rows, bf16), (o, "o", shape, bf16),
                                  (d_o, "d_o", shape, bf16), (lse, "lse", heads, f32),
                                  (lse if d_lse is None else d_lse, "d_lse", heads, f32)):
            _refuse(t, n, want, dtype, index)
    dq = torch.empty_like(q) if dq is None else _output(dq, "dq", shape, bf16, index)
    dkv = torch.empty_like(kv) if dkv is None else _output(dkv, "dkv", rows, bf16, index)
    keep, ws, size = _bytes(workspace, 0 if workspace is not None else
                            _lib.kpool_sparse_mla_bwd_workspace_size(T, rows[0]), index)
    _call(index, name, fn, q.data_ptr(), kv.data_ptr(), *lists, o.data_ptr(), lse.data_ptr(), d_o.data_ptr(),
          None if d_lse is None else d_lse.data_ptr(), *sizes, float(softmax_scale), dq.data_ptr(), dkv.data_ptr(), ws,
          size)
    return dq, dkv


def kpool_sparse_mla_bwd(q, kv, tok_idx, o, lse, d_o, softmax_scale: float, d_lse=None, workspace=None, dq=None,
                         dkv=None):
    """Gradients of kpool_sparse_mla_fwd: from d_o bf16 [T, 64, 512] (and d_lse
    fp32 [T, 64], if lse is used) and the o and lse that it wrote -> (dq bf16
    [T, 64, 512], dkv bf16 [Tk, 512])."""
    index, T, Tk, H, Dc = _mla_sizes(q, kv)
    at, width = _list_rows(tok_idx, "tok_idx", T, None, index)
    return _mla_bwd("kpool_sparse_mla_bwd", _lib.kpool_sparse_mla_bwd, index, q, kv, (at,), o, lse, d_o, d_lse,
                    (T, Tk, width, H, Dc), softmax_scale, workspace, dq, dkv)


def kpool_sparse_mla_bwd_pools(q, kv, pool_idx, o, lse, d_o, kpool: int, index_topk: int, softmax_scale: float,
                               cu_seqlens=None, cu_pools=None, always_select_tail: bool = True, d_lse=None,
                               workspace=None, dq=None, dkv=None):
    """Gradients of kpool_sparse_mla_fwd_pools (kv [T, 512]) -> (dq, dkv)."""
    index, T, Tk, H, Dc = _mla_sizes(q, kv)
    if (cu_seqlens is None) != (cu_pools is None):
        raise ValueError("cu_seqlens and cu_pools go together")
    if Tk != T:
        raise ValueError("kv must have the %d rows of q (got %d)" % (T, Tk))
    at, n_docs = _list_rows(pool_idx, "pool_idx", T, index_topk // kpool, index)[0], 1
    docs = (None, None)
    if cu_seqlens is not None:
        n_docs = cu_seqlens.numel() - 1
        docs = (_ints(cu_seqlens, "cu_seqlens", n_docs + 1, index), _ints(cu_pools, "cu_pools", n_docs + 1, index))
    return _mla_bwd("kpool_sparse_mla_bwd_pools", _lib.kpool_sparse_mla_bwd_pools, index, q, kv, (at, *docs, n_docs), o,
                    lse, d_o, d_lse, (T, H, Dc, kpool, index_topk, 1 if always_select_tail else 0), softmax_scale,
                    workspace, dq, dkv)


def kpool_sparse_mla_bwd_pools_at(q, kv, pool_idx, o, lse, d_o, kpool: int, index_topk: int, softmax_scale: float,
                                  cu_seqlens_q, q_start_pos, cu_seqlens_k, cu_pools, always_select_tail: bool = True,
                                  d_lse=None, workspace=None, dq=None, dkv=None):
    """Gradients of kpool_sparse_mla_fwd_pools_at (keys kv [Tk, 512]) -> (dq, dkv)."""
    index, T, Tk, H, Dc = _mla_sizes(q, kv)
    n = cu_seqlens_q.numel() - 1
    lists = (_list_rows(pool_idx, "pool_idx", T, index_topk // kpool, index)[0],
             _ints(cu_seqlens_q, "cu_seqlens_q", n + 1, index), _ints(q_start_pos, "q_start_pos", n, index),
             _ints(cu_seqlens_k, "cu_seqlens_k", n + 1, index), _ints(cu_pools, "cu_pools", n + 1, index), n)
    return _mla_bwd("kpool_sparse_mla_bwd_pools_at", _lib.kpool_sparse_mla_bwd_pools_at, index, q, kv, lists, o, lse, d_o,
                    d_lse, (T, Tk, H, Dc, kpool, index_topk, 1 if always_select_tail else 0), softmax_scale, workspace,
                    dq, dkv)


def kpool_sparse_mla_paged_workspace_size(Tq: int, kpool: int, index_topk: int) -> int:
    return int(_lib.kpool_sparse_mla_paged_workspace_size(Tq, kpool, index_topk))


def kpool_sparse_mla_fwd_pools_paged(q, kv, page_table, seq_lens, pool_idx, kpool: int, index_topk: int,
                                     softmax_scale: float, cu_seqlens_q, q_start_pos, cu_pools, seq_ids=None,
                                     always_select_tail: bool = True, workspace=None, o=None, lse=None):
    """kpool_sparse_mla_fwd_pools_at over a paged cache: kv bf16 [n_pages,
    page_size, 512] (one layer of a store), page_table and seq_lens as in
    KPoolPages -> (o bf16 [Tq, 64, 512], lse fp32 [Tq, 64]).  q_start_pos is
    what kpool_pages_extend returned for the new tokens."""
    index, bf16 = _device_of(q, "q"), torch.bfloat16
    if kv.dtype is not bf16:
        raise TypeError("kv must be %s (got %s)" % (bf16, kv.dtype))
    shape, pages = q.shape, kv.shape
    if len(shape) != 3 or len(pages) != 3 or pages[2] != shape[2]:
        raise ValueError("q must be [Tq, H, Dc] and kv [n_pages, page_size, Dc] (got %s and %s)"
                         % (tuple(shape), tuple(pages)))
    Tq, H, Dc = shape
    n_pages, page_size, _ = pages
    stride = kv.stride()
    if kv.get_device() != index or stride[2] != 1 or (stride[1] != Dc and page_size > 1):
        _same_device(index, kv=kv)
        raise ValueError("the rows of a page of kv must be contiguous")
    _refuse(q, "q", shape, bf16, index)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_rows, max_pages]")
    n_rows, max_pages = page_table.shape
    B = cu_seqlens_q.numel() - 1
    lists = (_ints(page_table, "page_table", n_rows * max_pages, index), _ints(seq_lens, "seq_lens", n_rows, index),
             n_rows, max_pages, None if seq_ids is None else _ints(seq_ids, "seq_ids", B, index),
             _list_rows(pool_idx, "pool_idx", Tq, index_topk // kpool, index)[0],
             _ints(cu_seqlens_q, "cu_seqlens_q", B + 1, index), _ints(q_start_pos, "q_start_pos", B, index),
             _ints(cu_pools, "cu_pools", B + 1, index), B)
    o = torch.empty_like(q) if o is None else _output(o, "o", shape, bf16, index)
    lse = _output(lse, "lse", shape[:2], torch.float32, index)
    keep, ws, size = _bytes(workspace, 0 if workspace is not None else
                            _lib.kpool_sparse_mla_paged_workspace_size(Tq, kpool, index_topk), index)
    # (the stride of a single page says nothing)
    _call(index, "kpool_sparse_mla_fwd_pools_paged", _lib.kpool_sparse_mla_fwd_pools_paged, q.data_ptr(),
          kv.data_ptr(), stride[0] if n_pages > 1 else page_size * Dc, n_pages, page_size, *lists, Tq, H, Dc, kpool,
          index_topk, 1 if always_select_tail else 0, float(softmax_scale), o.data_ptr(), lse.data_ptr(), ws, size)
    return o, lse


def _host_cu(cu_seqlens_host):
    if cu_seqlens_host is None:
        return None, 1
    _need(cu_seqlens_host, "cu_seqlens_host", torch.int32, device=False)
    if cu_seqlens_host.is_cuda:
        raise ValueError("cu_seqlens_host must be a CPU tensor")
    return cu_seqlens_host, cu_seqlens_host.numel() - 1


def kpool_indexer_forward_host_scratch_size(T: int, H: int, D: int, kpool: int, index_topk: int,
                                            cu_seqlens_host=None, fp8: bool = False,
                                            chunk_rows: int = 0) -> int:
    cu, n_docs = _host_cu(cu_seqlens_host)
    return int(_lib.kpool_indexer_forward_host_scratch_size(_ptr(cu), n_docs, T, H, D, kpool,
                                                            index_topk, int(fp8), chunk_rows))


def kpool_indexer_forward_host(q, k, gate, ape, w, kpool: int, index_topk: int,
                               always_select_tail: bool = True, cu_seqlens_host=None,
                               fp8: bool = False, chunk_rows: int = 0, scratch=None, out=None,
                               device=None):
    """The whole pass from host (CPU, ideally pinned) tensors to host token
    indices int32 [T, Kp*kpool + kpool - 1], copies overlapped with the
    kernels.  Enqueued on the current CUDA stream of `device`; synchronize it
    before reading the result.  Without `scratch`, a device scratch of
    kpool_indexer_forward_host_scratch_size bytes (about 0.9 GB at T=131072)
    is allocated for the call: pass one to reuse it across calls."""
    for t_, n_, dt in ((q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                       (gate, "gate", torch.bfloat16), (ape, "ape", torch.float32),
                       (w, "w", torch.float32)):
        _need(t_, n_, dt, device=False)
        if t_.is_cuda:
            raise ValueError("%s must be a host tensor" % n_)
    cu, n_docs = _host_cu(cu_seqlens_host)
    T, H, D = q.shape
    dev = torch.device("cuda") if device is None else torch.device(device)
    W = (index_topk // kpool) * kpool + kpool - 1
    if out is None:
        out = torch.empty(T, W, dtype=torch.int32, pin_memory=True)
    if scratch is None:
        n = kpool_indexer_forward_host_scratch_size(T, H, D, kpool, index_topk, cu, fp8,
                                                    chunk_rows)
        scratch = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    _check(_lib.kpool_indexer_forward_host(_ptr(q), _ptr(k), _ptr(gate), _ptr(ape), _ptr(w),
                                           _ptr(cu), n_docs, T, H, D, kpool, index_topk,
                                           int(bool(always_select_tail)), int(fp8), chunk_rows,
                                           _ptr(out), _ptr(scratch), scratch.numel(),
                                           _stream(dev)), "kpool_indexer_forward_host")
    return out


def kpool_read_status(workspace) -> int:
    """Status word of the last call that used `workspace` (waits for its device)."""
    v = ctypes.c_int(0)
    with torch.cuda.device(-1 if workspace is None else workspace.get_device()):
        _check(_lib.kpool_read_status(_ptr(workspace), ctypes.byref(v)), "kpool_read_status")
    return int(v.value)


def kpool_score_topk_noalloc_status() -> int:
    """Status word of the last kpool_score_topk_noalloc on the current device."""
    v = ctypes.c_int(0)
    _check(_lib.kpool_score_topk_noalloc_status(ctypes.byref(v)),
           "kpool_score_topk_noalloc_status")
    return int(v.value)


def kpool_debug_set_wait_limit_ns(ns: int) -> int:
    """Test entry: limit of each scoring-kernel wait (0 = the 2 s default);
    returns the previous limit."""
    return int(_lib.kpool_debug_set_wait_limit_ns(int(ns)))


def kpool_indexer_forward(q, k, gate, ape, w, kpool: int, index_topk: int,
                          always_select_tail: bool = True, cu_seqlens=None, cu_pools=None,
                          P_total=None, fp8: bool = False, workspace=None):
    """The whole indexer path on the current stream: compress -> (FP8 cast of
    q and pooled keys) -> score + top-k -> expand.  Returns
    (tok_idx, pool_idx, pool_score)."""
    if fp8:
        pk, pk8, pks = kpool_compress(k, gate, ape, kpool, cu_seqlens, cu_pools, P_total, fp8=True)
        q8, qs = kpool_quantize_fp8(q)
        idx, sc = kpool_score_topk(q8, w, pk8, kpool, index_topk, cu_seqlens, cu_pools,
                                   q_scale=qs, pk_scale=pks, workspace=workspace)
    else:
        pk = kpool_compress(k, gate, ape, kpool, cu_seqlens, cu_pools, P_total)
        idx, sc = kpool_score_topk(q, w, pk, kpool, index_topk, cu_seqlens, cu_pools,
                                   workspace=workspace)
    tok = kpool_expand_indices(idx, kpool, index_topk, always_select_tail, cu_seqlens, cu_pools)
    return tok, idx, sc


__all__ = [n for n in dir() if n.startswith("kpool_")] + ["KPoolError", "KPoolPages",
                                                           "new_workspace", "LIB_PATH"]

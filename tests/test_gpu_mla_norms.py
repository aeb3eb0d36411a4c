"""The sparse attention's gradients and its paged form against the definition as a whole: 2-norms
of the errors over all rows and row by row (mla_norm_checks), where many rows list a token."""
import numpy as np
import pytest
import torch

from mla_grad_checks import H, check_forward
from mla_norm_checks import GradNorms, check_outputs
from sparse_attention_kpool_compress_gb300 import workloads as W
from test_gpu_mla_bwd import _dev, _inputs, _lists, _pools, _rows_of
from test_gpu_paged_mla import Case

pytestmark = pytest.mark.gpu
SCALE = W.MLA_SCALE


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


@pytest.mark.parametrize("T,Tk,sizes,scale,with_lse", [
    (400, 64, [64, 40], SCALE, False), (400, 64, [64, 40], SCALE, True), (400, 64, [64, 40], 0.3, True),
    (1500, 7, [333, 0, 100], SCALE, False), (76, 500, [333, 65, 128], SCALE, True), (9, 40, [333, 200], SCALE, False)])
def test_lists(K, T, Tk, sizes, scale, with_lse):
    """Each token in most of the rows; lists that name a token many times; whole rows and rows that are cut."""
    q, kv, d_o, d_lse = _inputs(T, Tk, 51)
    tok = _lists(np.random.default_rng(T), T, Tk, 333, sizes)
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, scale)
    grad_lse = d_lse if with_lse else None
    want = GradNorms(q, kv, _rows_of(tok, Tk), o, lse, d_o, scale, grad_lse)
    for _ in range(2):
        want.check(*K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, scale, d_lse=grad_lse))


@pytest.mark.parametrize("kp,budget,lens", [(4, 512, (4099,)), (8, 64, (1200, 1, 700, 0, 555)), (1, 300, (333, 900))])
def test_pools(K, kp, budget, lens):
    """All rows of sequences over and under the budget."""
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    sel, cu_pools = _pools(np.random.default_rng(kp), cu, kp, budget)
    q, kv, d_o, _ = _inputs(T, T, 53)
    cu_d, cp_d = _dev(cu), _dev(cu_pools)
    tok = K.kpool_expand_indices(sel, kp, budget * kp, True, cu_d, cp_d)
    lists = _rows_of(tok, T)
    o, lse = K.kpool_sparse_mla_fwd_pools(q, kv, sel, kp, budget * kp, SCALE, cu_d, cp_d)
    dq, dkv = K.kpool_sparse_mla_bwd_pools(q, kv, sel, o, lse, d_o, kp, budget * kp, SCALE, cu_d, cp_d)
    GradNorms(q, kv, lists, o, lse, d_o, SCALE).check(dq, dkv)


@pytest.mark.parametrize("lens,queries", [([1500, 3100, 77, 2048], [100, 140, 20, 60]), ([2500, 2049, 90], [3, 2, 4])])
def test_paged_and_flat(K, lens, queries):
    """Every row of the paged call and of the flat call on the same tokens, whole rows and rows that are cut: each
    within the rounding of p of the definition (the two take blocks of different lengths)."""
    lens, queries, kp, budget = np.array(lens), np.array(queries), 4, 512
    c = Case(3, lens, queries, kp, budget, 32)
    cu_k = np.concatenate([[0], np.cumsum(lens)])
    flat = torch.cat(c.flat)
    rows = [torch.from_numpy(toks + cu_k[b]).cuda() for b, toks in c.lists]
    paged = c.call(K)
    at = K.kpool_sparse_mla_fwd_pools_at(c.q, flat, c.sel, kp, kp * budget, SCALE, c.cu_q, c.pos, _dev(cu_k), c.cu_pools)
    for what, (o, lse) in (("paged", paged), ("flat", at)):
        assert o.shape == (len(rows), H, 512)
        check_outputs(o, c.q, flat, rows, SCALE, what)
        for t, j in enumerate(rows):
            check_forward(o[t], lse[t], c.q[t], flat[j], SCALE, (what, t))

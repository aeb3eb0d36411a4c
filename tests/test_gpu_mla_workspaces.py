"""One workspace, sized for the largest batch, in calls of fewer and fewer rows (a rollout
whose sequences end one by one): the sparse attention's backward pass and its paged form."""
import numpy as np
import pytest
import torch

from mla_grad_checks import Grads
from sparse_attention_kpool_compress_gb300 import workloads as W
from test_gpu_mla_bwd import _inputs, _lists, _rows_of
from test_gpu_paged_mla import Case

pytestmark = pytest.mark.gpu
SCALE = W.MLA_SCALE


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


@pytest.mark.parametrize("most", [81, 200, 8192])
def test_backward(K, most):
    Tk, rng = 150, np.random.default_rng(most)
    ws = torch.full((K.kpool_sparse_mla_bwd_workspace_size(most, Tk),), 0x7F, dtype=torch.uint8, device="cuda")
    for T in (200, 81, 80, 77, 76, 5, 3, 1):
        if T > most:
            continue
        q, kv, d_o, _ = _inputs(T, Tk, T)
        tok = _lists(rng, T, Tk, 200, [200, 90, 0, 130] if T > 1 else [200])
        o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, SCALE)
        dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
        assert K.kpool_read_status(ws) == 0
        Grads(q, kv, _rows_of(tok, Tk), o, lse, d_o, SCALE).check(dq, dkv, T)


@pytest.mark.parametrize("most", [81, 200, 8192])
def test_paged(K, most):
    ws = torch.full((K.kpool_sparse_mla_paged_workspace_size(most, 4, 1024),), 0x7F, dtype=torch.uint8, device="cuda")
    for T in (200, 81, 80, 77, 76, 5, 3, 1):
        if T > most:
            continue
        c = Case(T, [1100 + t % 7 for t in range(T)], [1] * T, 4, 256, 64)
        o, lse = c.call(K, workspace=ws)
        assert K.kpool_read_status(ws) == 0
        c.check(o, lse, T, rows=set(range(0, T, max(1, T // 9))) | {T - 1})

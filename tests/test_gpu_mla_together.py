"""The sparse attention's calls at the same time: the backward pass, the paged form (whole rows and rows that
are cut) and the flat form on streams of their own, each with its own workspace."""
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


def test_calls_on_several_streams(K):
    cases = [Case(31, [2500, 900], [1, 2], 4, 512, 64), Case(32, [900] * 3, [80, 70, 60], 4, 128, 32)]
    back = []
    for T in (20, 300):
        q, kv, d_o, _ = _inputs(T, 400, T)
        tok = _lists(np.random.default_rng(T), T, 400, 260, [260, 100, 0, 65])
        back.append((q, kv, tok, *K.kpool_sparse_mla_fwd(q, kv, tok, SCALE), d_o))
    spaces = [c.workspace(K) for c in cases] + [
        torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(b[0].shape[0], 400), dtype=torch.uint8, device="cuda") for b in back]
    calls = [lambda c=c, w=w: c.call(K, workspace=w) for c, w in zip(cases, spaces)]
    calls += [lambda b=b, w=w: K.kpool_sparse_mla_bwd(*b, SCALE, workspace=w) for b, w in zip(back, spaces[2:])]
    calls += [lambda b=b: K.kpool_sparse_mla_fwd(*b[:3], SCALE) for b in back]
    alone = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(8):
        for f, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    assert [K.kpool_read_status(w) for w in spaces] == [0] * len(spaces)
    want = [Grads(b[0], b[1], _rows_of(b[2], 400), *b[3:], SCALE) for b in back]
    for i, g in enumerate(got):
        i %= len(calls)
        # (dkv's sums have no fixed order)
        assert torch.equal(g[0], alone[i][0]), i
        if i in (2, 3):
            want[i - 2].check(*g)
        else:
            assert torch.equal(g[1], alone[i][1]), i

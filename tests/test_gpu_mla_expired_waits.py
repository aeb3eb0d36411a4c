"""Expired waits of the sparse attention's backward pass and of its paged form: the status
word tells of them, and the next call in the same workspace is clean and right."""
import numpy as np
import pytest
import torch

from mla_grad_checks import Grads, check_forward
from sparse_attention_kpool_compress_gb300 import workloads as W
from test_gpu_mla_bwd import DC, H, _inputs, _lists, _rows_of
from test_gpu_paged_mla import Case

pytestmark = pytest.mark.gpu
SCALE = W.MLA_SCALE


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


@pytest.mark.parametrize("rows", [1, 7, 20, 76, 77, 400])
def test_backward_reports_an_expired_wait(K, rows):
    """Rows that are cut into runs (up to half as many as there are SMs) and whole ones, at a limit that the
    first wait passes."""
    Tk = 300
    q, kv, d_o, _ = _inputs(rows, Tk, 43)
    tok = _lists(np.random.default_rng(rows), rows, Tk, 2051, [2051, 700, 1500, 65])
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, SCALE)
    ws = torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(rows, Tk), dtype=torch.uint8, device="cuda")
    status = []
    for _ in range(8):
        K.kpool_debug_set_wait_limit_ns(1)
        try:
            K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
            status.append(K.kpool_read_status(ws))
        finally:
            assert K.kpool_debug_set_wait_limit_ns(0) == 1
        dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
        assert K.kpool_read_status(ws) == 0
    assert status == [K.STATUS_TIMEOUT] * len(status)
    Grads(q, kv, _rows_of(tok, Tk), o, lse, d_o, SCALE).check(dq, dkv)


def test_backward_wait_that_suspends(K):
    """A limit of 1 ms, at which probes suspend the thread as at the default.  The roles wait for a row's first
    block while its list of 2^20 entries is looked through, which takes longer."""
    T, Tk, width = 77, 40, 1 << 20
    q, kv, d_o, _ = _inputs(T, Tk, 47)
    tok = torch.full((T, width), -1, dtype=torch.int32, device="cuda")
    tok[:, 5] = torch.arange(T, device="cuda") % Tk
    lists = [r[r >= 0].long() for r in tok[:, :6]]
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok[:, :6].contiguous(), SCALE)
    ws = torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(T, Tk), dtype=torch.uint8, device="cuda")

    def call():
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        got = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
        end.record()
        return got, K.kpool_read_status(ws), begin.elapsed_time(end)

    for _ in range(2):
        (dq, dkv), status, ms = call()
        assert status == 0
        Grads(q, kv, lists, o, lse, d_o, SCALE).check(dq, dkv)
        assert ms > 1.5, ms                      # (the look alone: a row has one block)
        K.kpool_debug_set_wait_limit_ns(1000000)
        try:
            assert call()[1] == K.STATUS_TIMEOUT
        finally:
            assert K.kpool_debug_set_wait_limit_ns(0) == 1000000


def test_paged_wait_that_suspends(K):
    """The same: the roles wait for the first block while rows that see nothing are passed over, 600 for each
    SM."""
    T = 600 * torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(21, [3, 700], [1, 1], 4, 8, 16, tail=False, shuffled=False)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(T + 1, H, DC, dtype=torch.bfloat16, device="cuda")
    q[T] = c.q[1]
    sel = torch.full((T + 1, 8), -1, **i32)
    sel[T] = c.sel[1]
    # T queries of the first sequence, all at positions without a whole pool: as many sequences of one row
    ids = torch.zeros(T + 1, **i32)
    ids[T] = 1
    cu = torch.arange(T + 2, **i32)
    pos = torch.full((T + 1,), 2, **i32)
    pos[T] = 699
    pools = torch.zeros(T + 2, **i32)
    pools[T + 1] = 700 // 4
    ws = torch.zeros(K.kpool_sparse_mla_paged_workspace_size(T + 1, 4, 32), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(T + 1, H, device="cuda")

    def call():
        o.fill_(7.0)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        K.kpool_sparse_mla_fwd_pools_paged(q, c.kv, c.table, c.row_lens, sel, 4, 32, SCALE, cu, pos, pools, seq_ids=ids,
                                           always_select_tail=False, workspace=ws, o=o, lse=lse)
        end.record()
        return K.kpool_read_status(ws), begin.elapsed_time(end)

    for _ in range(2):
        status, ms = call()
        assert status == 0
        assert torch.all(o[:T] == 0) and torch.isneginf(lse[:T]).all()
        check_forward(o[T], lse[T], q[T], c.flat[1][torch.from_numpy(c.lists[1][1]).cuda()], SCALE)
        assert ms > 1.5, ms                      # (passing over the rows)
        K.kpool_debug_set_wait_limit_ns(1000000)
        try:
            assert call()[0] == K.STATUS_TIMEOUT
        finally:
            assert K.kpool_debug_set_wait_limit_ns(0) == 1000000

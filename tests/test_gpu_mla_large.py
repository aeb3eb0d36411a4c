"""The largest sizes of the sparse attention's backward pass and of its paged form."""
import math

import numpy as np
import pytest
import torch

from mla_grad_checks import DC, E, H, U, Grads, check_forward
from sparse_attention_kpool_compress_gb300 import workloads as W

pytestmark = pytest.mark.gpu
SCALE = W.MLA_SCALE


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


def test_a_row_of_nearly_2_31_tokens(K):
    """The longest sequence that a table can hold, one page in every place of it, every token listed: o is the
    mean of equal rows, lse the log of their number."""
    page, pages = 127 * 113, 149640
    n = page * pages
    assert n == (1 << 31) - 8
    i32 = dict(dtype=torch.int32, device="cuda")
    pools = n // 64
    table = torch.zeros(1, pages, **i32)
    kv = torch.ones(1, page, DC, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, H, DC, dtype=torch.bfloat16, device="cuda")
    sel = torch.arange(pools, **i32).view(1, pools)
    ws = torch.zeros(K.kpool_sparse_mla_paged_workspace_size(1, 64, 64 * pools), dtype=torch.uint8, device="cuda")
    o, lse = K.kpool_sparse_mla_fwd_pools_paged(q, kv, table, torch.tensor([n], **i32), sel, 64, 64 * pools, SCALE,
                                                torch.tensor([0, 1], **i32), torch.tensor([n - 1], **i32),
                                                torch.tensor([0, pools], **i32), workspace=ws)
    assert K.kpool_read_status(ws) == 0
    # sums of ones: exact up to 2^24 a thread, and as multiples of 16 up to 2^28 a run, which has 2^26
    assert torch.all((o.float() - 1).abs() <= U)
    # a few roundings each of the runs' log-sums (26, base 2), of their join and of the whole (31)
    assert torch.all((lse.double() - math.log(n)).abs() <= 16 * E * 31)


def _queries(T, seed):
    """bf16 [T, 64, 512], a piece at a time."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.empty(T, H, DC, dtype=torch.bfloat16, device="cuda")
    for part in x.split(4096):
        part.normal_(generator=g)
    return x


def test_more_than_65536_rows_backward(K):
    """Queries, outputs and their gradients behind 2^32 bytes: rows on both sides of the border, and the sums of
    all rows."""
    T, Tk, width = 65536 + 301, 3000, 5
    rng = np.random.default_rng(61)
    kv = torch.randn(Tk, DC, generator=torch.Generator("cuda").manual_seed(62), device="cuda").to(torch.bfloat16)
    tok = torch.from_numpy(rng.integers(0, Tk, size=(T, width)).astype(np.int32)).cuda()
    tok[::3, 2] = -1
    q, d_o = _queries(T, 63), _queries(T, 64)
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, SCALE)
    ws = torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(T, Tk), dtype=torch.uint8, device="cuda")
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    rows = [0, 1, 2, 32767, 32768, 65534, 65535, 65536, 65537, T - 2, T - 1]
    lists = {t: tok[t][tok[t] >= 0].long() for t in rows}
    for t in rows:
        check_forward(o[t], lse[t], q[t], kv[lists[t]], SCALE, t)
    want = Grads(q, kv, lists, o, lse, d_o, SCALE, rows=rows)
    for t in rows:
        err, tol = (dq[t].double() - want.dq[t]).abs(), want.dq_tol[t] + U * want.dq[t].abs() + 1e-30
        assert torch.all(err <= tol), (t, float((err / tol).max()))
    del want
    # the latent rows' gradients, from all rows
    some = torch.tensor([0, 1, 1500, Tk - 1], device="cuda")
    at = (torch.isin(tok, some).any(1)).nonzero()[:, 0]
    assert (at >= 65536).any() and (at < 65536).any()
    small = [r[r >= 0].long() for r in tok[at]]
    want = Grads(q[at], kv, small, o[at], lse[at], d_o[at], SCALE)
    err, tol = (dkv.double() - want.dkv)[some].abs(), (want.dkv_tol + U * want.dkv.abs())[some] + 1e-30
    assert torch.all(err <= tol), float((err / tol).max())


def test_more_than_65536_rows_paged(K):
    """The paged form with its queries and outputs behind 2^32 bytes, in two sequences."""
    n, page = [40000, 26001], 128
    T, kp, budget = sum(n), 4, 8
    used = [-(-x // page) for x in n]
    ids = torch.randperm(sum(used) + 2, generator=torch.Generator().manual_seed(71)).cuda()
    table = torch.full((2, max(used)), -1, dtype=torch.int32, device="cuda")
    table[0, :used[0]], table[1, :used[1]] = ids[:used[0]].int(), ids[used[0]:sum(used)].int()
    kv = torch.randn(sum(used) + 2, page, DC, generator=torch.Generator("cuda").manual_seed(72), device="cuda").to(torch.bfloat16)
    q = _queries(T, 73)
    i32 = dict(dtype=torch.int32, device="cuda")
    pools = [x // kp for x in n]
    sel = torch.full((T, budget), -1, **i32)
    rows, lists = [8, 39999, 40000, 40050, 65534, 65535, 65536, 65537, T - 1], {}
    rng = np.random.default_rng(74)
    for first, lo, hi, base in ((0, 0, n[0], 0), (n[0], n[0], T, pools[0])):
        tau = torch.arange(lo, hi, device="cuda") - first
        seen = (tau + 1) // kp
        pick = torch.from_numpy(rng.random((hi - lo, budget))).cuda().sort(1).values
        col = torch.arange(budget, device="cuda")
        # ascending and apart where there are more pools than the budget, all pools else
        far = (pick * (seen - budget).clamp(min=0)[:, None]).long() + col
        sel[lo:hi] = torch.where(col < seen[:, None], far + base, -1).int()
    o, lse = K.kpool_sparse_mla_fwd_pools_paged(q, kv, table, torch.tensor(n, **i32), sel, kp, kp * budget, SCALE,
                                                torch.tensor([0, n[0], T], **i32), torch.zeros(2, **i32),
                                                torch.tensor([0, pools[0], sum(pools)], **i32))
    for t in rows:
        b = int(t >= n[0])
        tau = t - b * n[0]
        mine = sel[t][sel[t] >= 0].long() - b * pools[0]
        toks = (mine[:, None] * kp + torch.arange(kp, device="cuda")).view(-1)
        toks = torch.cat([toks, torch.arange((tau + 1) // kp * kp, tau + 1, device="cuda")])
        keys = kv[table[b].long()[toks // page], toks % page]
        check_forward(o[t], lse[t], q[t], keys, SCALE, t)

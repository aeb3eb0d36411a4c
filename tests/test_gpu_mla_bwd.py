"""The sparse attention's backward calls (kpool_sparse_mla_bwd, _pools, _pools_at)
against the definition in 64 bits, against differences of the forward function, and
against one another.  Tolerances: mla_grad_checks."""
import numpy as np
import pytest
import torch

from mla_grad_checks import DC, E, H, U, Grads
from sparse_attention_kpool_compress_gb300 import workloads as W

pytestmark = pytest.mark.gpu
SCALE = W.MLA_SCALE


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


def _inputs(T, Tk, seed, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, s=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    return normal(T, H, DC, s=size), normal(Tk, DC), normal(T, H, DC, s=0.1), torch.randn(T, H, generator=g, device="cuda")


def _lists(rng, T, Tk, width, sizes):
    """Rows of these sizes in turn: repeats, holes anywhere, entries out of range in the holes."""
    tok = np.full((T, width), -1, np.int32)
    tok[:, ::7] = Tk + 3
    tok[:, 3::11] = -2147483648
    for t in range(T):
        n = sizes[t % len(sizes)]
        tok[t, np.sort(rng.choice(width, size=n, replace=False))] = rng.integers(0, Tk, size=n)
    return torch.from_numpy(tok).cuda()


def _rows_of(tok, Tk):
    return [r[(r >= 0) & (r < Tk)].long() for r in tok]


def _forward(q, kv, lists, scale):
    """o (rounded once) and lse of the definition."""
    o, lse = torch.zeros_like(q), torch.full(q.shape[:2], -torch.inf, device="cuda")
    for t, j in enumerate(lists):
        if j.numel():
            s = scale * (q[t].double() @ kv[j].double().T)
            l = torch.logsumexp(s, 1)
            o[t], lse[t] = (torch.exp(s - l[:, None]) @ kv[j].double()).to(torch.bfloat16), l.float()
    return o, lse


def _ulp_close(a, b, tol):
    """BF16 sums in two orders: within `tol`, or a step of each other."""
    a, b = a.double(), b.double()
    return torch.all((a - b).abs() <= tol + 2 * U * torch.maximum(a.abs(), b.abs()))


@pytest.mark.parametrize("scale,with_lse", [(SCALE, False), (SCALE, True), (0.3, True)])
def test_lists_against_the_definition(K, scale, with_lse):
    """Empty rows, one token, every edge of a block, repeats, holes, ids out of range; scale 0.3: one
    token has nearly all of the probability."""
    T, Tk, width = 45, 700, 333
    q, kv, d_o, d_lse = _inputs(T, Tk, 1)
    tok = _lists(np.random.default_rng(2), T, Tk, width, [0, 1, 63, 64, 65, 127, 128, 129, 333, 200])
    lists = _rows_of(tok, Tk)
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, scale)
    ws = torch.full((K.kpool_sparse_mla_bwd_workspace_size(T, Tk),), 0x7F, dtype=torch.uint8, device="cuda")
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, scale, d_lse=d_lse if with_lse else None, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    assert torch.all(dq[0] == 0)
    Grads(q, kv, lists, o, lse, d_o, scale, d_lse if with_lse else None).check(dq, dkv)


@pytest.mark.parametrize("T,width", [(1, 1), (1, 2051), (2, 64), (7, 2000), (76, 700), (77, 130), (153, 70), (305, 5)])
def test_numbers_of_rows(K, T, width):
    """One row, one token; rows that are cut over SMs (up to half as many as there are) and whole ones; one row
    more than the GPU has SMs, and twice as many."""
    Tk = 90
    q, kv, d_o, _ = _inputs(T, Tk, 3)
    tok = _lists(np.random.default_rng(T), T, Tk, width, [width, max(1, width // 3), width // 2])
    lists = _rows_of(tok, Tk)
    o, lse = _forward(q, kv, lists, SCALE)
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE)
    Grads(q, kv, lists, o, lse, d_o, SCALE).check(dq, dkv)


def _pools(rng, cu, kp, budget, q_rows=None):
    """Random selections of the rows of packed documents (q_rows[d]: its last rows), and cu_pools."""
    lens = np.diff(cu)
    cu_pools = np.concatenate([[0], np.cumsum(lens // kp)]).astype(np.int32)
    sel = []
    for d, n in enumerate(lens):
        for tau in range(0 if q_rows is None else n - q_rows[d], n):
            row = np.full(budget, -1, np.int32)
            k = min((tau + 1) // kp, budget)
            row[:k] = np.sort(rng.choice((tau + 1) // kp, size=k, replace=False)) + cu_pools[d]
            sel.append(row)
    return torch.from_numpy(np.array(sel).reshape(-1, budget)).cuda(), cu_pools


def _dev(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("kp,budget,tail,docs", [
    (1, 60, True, None), (4, 16, True, None), (4, 24, False, None), (3, 30, True, (90, 0, 211)),
    (8, 9, True, (100, 1, 199)), (64, 2, True, (150, 150)), (64, 2, False, (63, 237))])
def test_pools(K, kp, budget, tail, docs):
    """The fused expansion lists what kpool_expand_indices writes (dq bit for bit), and both are the
    definition's."""
    lens = docs or (300,)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    sel, cu_pools = _pools(np.random.default_rng(kp), cu, kp, budget)
    q, kv, d_o, _ = _inputs(T, T, 5)
    cu_d, cp_d = (_dev(cu), _dev(cu_pools)) if docs else (None, None)
    tok = K.kpool_expand_indices(sel, kp, budget * kp, tail, cu_d, cp_d)
    o, lse = K.kpool_sparse_mla_fwd_pools(q, kv, sel, kp, budget * kp, SCALE, cu_d, cp_d, tail)
    dq, dkv = K.kpool_sparse_mla_bwd_pools(q, kv, sel, o, lse, d_o, kp, budget * kp, SCALE, cu_d, cp_d, tail)
    dq2, dkv2 = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE)
    want = Grads(q, kv, _rows_of(tok, T), o, lse, d_o, SCALE)
    want.check(dq, dkv)
    assert torch.equal(dq, dq2) and _ulp_close(dkv, dkv2, want.dkv_tol)


def test_positioned(K):
    """Answers behind prompts (_pools_at): the rows' gradients, and those of all keys."""
    kp, budget = 4, 40
    lens, nq = np.array([500, 77, 1300, 4]), np.array([60, 1, 33, 4])
    cu_k, cu_q = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lens, nq))
    sel, cu_pools = _pools(np.random.default_rng(8), cu_k, kp, budget, nq)
    T, Tk = int(cu_q[-1]), int(cu_k[-1])
    q, kv, d_o, d_lse = _inputs(T, Tk, 9)
    where = _dev(cu_q), _dev(lens - nq), _dev(cu_k), _dev(cu_pools)
    o, lse = K.kpool_sparse_mla_fwd_pools_at(q, kv, sel, kp, budget * kp, SCALE, *where)
    tok = K.kpool_expand_indices_at(sel, kp, budget * kp, *where)
    want = Grads(q, kv, _rows_of(tok, Tk), o, lse, d_o, SCALE, d_lse)
    dq, dkv = K.kpool_sparse_mla_bwd_pools_at(q, kv, sel, o, lse, d_o, kp, budget * kp, SCALE, *where, d_lse=d_lse)
    want.check(dq, dkv)
    # outputs of the caller
    out = torch.full_like(dq, 7.0), torch.full_like(dkv, 7.0)
    got = K.kpool_sparse_mla_bwd_pools_at(q, kv, sel, o, lse, d_o, kp, budget * kp, SCALE, *where, d_lse=d_lse,
                                          dq=out[0], dkv=out[1])
    assert got[0] is out[0] and got[1] is out[1] and torch.equal(got[0], dq)
    want.check(*got)


def test_against_differences(K):
    """<o, d_o> + <lse, d_lse> as a function of q and kv, by differences in 64 bits along random
    directions."""
    T, Tk = 6, 150
    q, kv, d_o, d_lse = _inputs(T, Tk, 11)
    tok = _lists(np.random.default_rng(4), T, Tk, 140, [140, 20, 1, 70])
    lists = _rows_of(tok, Tk)
    o, lse = _forward(q, kv, lists, SCALE)
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, d_lse=d_lse)

    def f(qd, kvd):
        total = 0.0
        for t, j in enumerate(lists):
            s = SCALE * (qd[t] @ kvd[j].T)
            l = torch.logsumexp(s, 1)
            total = total + ((torch.exp(s - l[:, None]) @ kvd[j]) * d_o[t].double()).sum() + (l * d_lse[t].double()).sum()
        return float(total)

    want = Grads(q, kv, lists, o, lse, d_o, SCALE, d_lse, o_err=U)
    tol_q, tol_kv = want.dq_tol + U * want.dq.abs(), want.dkv_tol + U * want.dkv.abs()
    g = torch.Generator("cuda").manual_seed(0)
    h = 1e-4
    for k in range(8):
        vq = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64) * (k % 3 != 1)
        vk = torch.randn(kv.shape, generator=g, device="cuda", dtype=torch.float64) * (k % 3 != 2)
        # (the third derivative's part of a central difference: by halving h)
        d1, d2 = ((f(q.double() + x * vq, kv.double() + x * vk) - f(q.double() - x * vq, kv.double() - x * vk)) / (2 * x)
                  for x in (h, h / 2))
        slope = (4 * d2 - d1) / 3
        got = float((dq.double() * vq).sum() + (dkv.double() * vk).sum())
        tol = float((tol_q * vq.abs()).sum() + (tol_kv * vk.abs()).sum()) + abs(d2 - d1) + 1e-6
        assert abs(got - slope) <= tol, (k, got, slope, tol)


def test_degenerate_calls(K):
    """No rows, lists of width 0, rows that list nothing; NaN in what nothing lists and in the gradients
    of rows without tokens reaches no result."""
    q, kv, d_o, _ = _inputs(5, 40, 13)
    lse = torch.zeros(5, H, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    dq, dkv = K.kpool_sparse_mla_bwd(q[:0], kv, torch.zeros(0, 4, **i32), q[:0], lse[:0], q[:0], SCALE)
    assert dq.shape == (0, H, DC) and torch.all(dkv == 0)
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, torch.zeros(5, 0, **i32), q, lse, d_o, SCALE)
    assert torch.all(dq == 0) and torch.all(dkv == 0)
    tok = torch.full((5, 100), -1, **i32)
    tok[1, 3], tok[1, 99], tok[3, 64] = 7, 8, 7
    lists = _rows_of(tok, 40)
    clean = kv.clone()
    kv[0], kv[9:], kv[8, 5] = torch.nan, torch.inf, 3.0
    clean[7:9] = kv[7:9]
    o, lse = _forward(q, clean, lists, SCALE)
    assert torch.isneginf(lse[0]).all()
    d_o[0], d_o[2], q[4] = torch.nan, torch.inf, torch.nan
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE)
    assert torch.all(dq[[0, 2, 4]] == 0)
    keep = torch.tensor([1, 3], device="cuda")
    want = Grads(q, clean, lists, o, lse, d_o, SCALE, rows=[1, 3])
    want.check(dq, dkv)
    assert torch.all(dkv[[0] + list(range(9, 40))] == 0) and keep.numel() == 2


def test_nan_of_a_query_stays_in_its_row(K):
    """A NaN query makes its own gradients NaN and those of the rows that it lists, no others."""
    T, Tk = 4, 300
    q, kv, d_o, _ = _inputs(T, Tk, 17)
    tok = torch.arange(T * 70, dtype=torch.int32, device="cuda").view(T, 70)
    lists = _rows_of(tok, Tk)
    o, lse = _forward(q, kv, lists, SCALE)
    q[2, 5, 9] = torch.nan
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE)
    assert torch.isnan(dq[2, 5]).all() and torch.isnan(dkv[lists[2], 9]).all()
    others = [0, 1, 3]
    assert torch.isfinite(dq[others]).all() and torch.isfinite(dkv[torch.cat([lists[t] for t in others])]).all()
    Grads(q, kv, lists, o, lse, d_o, SCALE, rows=others).check(dq, torch.where(torch.isnan(dkv), 0.0, dkv)
                                                              * (~torch.isin(torch.arange(Tk, device="cuda"), lists[2]))[:, None])


def test_streams_graphs_and_a_shared_workspace(K):
    """Two calls in one workspace, on another stream than the tensors' own, captured into a graph and
    replayed after the inputs changed."""
    T, Tk, width = 70, 500, 150
    q, kv, d_o, _ = _inputs(T, Tk, 19)
    rng = np.random.default_rng(6)
    toks = [_lists(rng, T, Tk, width, s) for s in ([150, 3, 64], [0, 90])]
    outs = [_forward(q, kv, _rows_of(t, Tk), SCALE) for t in toks]
    want = [Grads(q, kv, _rows_of(t, Tk), *f, d_o, SCALE) for t, f in zip(toks, outs)]
    ws = torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(T, Tk), dtype=torch.uint8, device="cuda")

    def both():
        return [K.kpool_sparse_mla_bwd(q, kv, t, *f, d_o, SCALE, workspace=ws) for t, f in zip(toks, outs)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    for w, g in zip(want, got):
        w.check(*g, "stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    keep = d_o.clone()
    d_o.zero_()
    graph.replay()
    assert all(torch.all(x == 0) for g in got for x in g)
    d_o.copy_(keep)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        w.check(*g, "graph")
    assert K.kpool_read_status(ws) == 0


def test_the_same_call_twice(K):
    """dq has a fixed order of sums; dkv differs by the order of FP32 additions at most."""
    T, Tk = 400, 64
    q, kv, d_o, _ = _inputs(T, Tk, 23)
    tok = _lists(np.random.default_rng(9), T, Tk, 64, [64, 40])
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, SCALE)
    a, b = (K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE) for _ in range(2))
    assert torch.equal(a[0], b[0])
    want = Grads(q, kv, _rows_of(tok, Tk), o, lse, d_o, SCALE)
    want.check(*a)
    want.check(*b)


def test_many_latent_rows(K):
    """Latent rows and sums behind 2^32 bytes."""
    Tk = (1 << 22) + 100
    T = 3
    q, _, d_o, _ = _inputs(T, 1, 29)
    kv = torch.zeros(Tk, DC, dtype=torch.bfloat16, device="cuda")
    tok = torch.tensor([[5, Tk - 1, 1 << 22, -1], [Tk - 2, -1, 1 << 21, 5], [Tk, Tk - 1, 0, 1]], dtype=torch.int32, device="cuda")
    used = tok[(tok >= 0) & (tok < Tk)].long().unique()
    kv[used] = torch.randn(used.numel(), DC, device="cuda").to(torch.bfloat16)
    lists = _rows_of(tok, Tk)
    o, lse = _forward(q, kv, lists, SCALE)
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE)
    assert int((dkv != 0).any(1).sum()) == used.numel()
    at = torch.full((Tk,), -1, dtype=torch.long, device="cuda")
    at[used] = torch.arange(used.numel(), device="cuda")
    Grads(q, kv[used], [at[j] for j in lists], o, lse, d_o, SCALE).check(dq, dkv[used])


def test_a_long_sequence_sampled(K):
    """8192 tokens over the indexer's kind of selection: some rows of dq, some of dkv with all their
    queries."""
    T, kp, budget = 8192, 4, 512
    q, kv, d_o, _ = _inputs(T, T, 31)
    g = torch.Generator("cuda").manual_seed(1)
    score = torch.rand(T, T // kp, generator=g, device="cuda")
    seen = (torch.arange(T, device="cuda") + 1) // kp
    col = torch.arange(T // kp, device="cuda")
    score.masked_fill_(col >= seen[:, None], -1.0)
    top, which = score.topk(budget, dim=1)
    sel = torch.where(top >= 0, which, T).sort(1).values
    sel = torch.where(sel < T, sel, -1).int()
    ws = torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(T, T), dtype=torch.uint8, device="cuda")
    o, lse = K.kpool_sparse_mla_fwd_pools(q, kv, sel, kp, budget * kp, SCALE)
    dq, dkv = K.kpool_sparse_mla_bwd_pools(q, kv, sel, o, lse, d_o, kp, budget * kp, SCALE, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    tok = K.kpool_expand_indices(sel, kp, budget * kp)
    rows = [0, 1, 3, 4, 62, 63, 64, 2047, 2051, 5000, 8191]
    lists = {t: tok[t][tok[t] >= 0].long() for t in rows}
    want = Grads(q, kv, lists, o, lse, d_o, SCALE, rows=rows)
    for t in rows:
        err, tol = (dq[t].double() - want.dq[t]).abs(), want.dq_tol[t] + U * want.dq[t].abs() + 1e-30
        assert torch.all(err <= tol), (t, float((err / tol).max()))
    for j in (0, 1, 2, 3, 777, 4096, 8000, 8190, 8191):
        t = ((tok == j).any(1)).nonzero()[:, 0]
        k, qd, do, od = kv[j].double(), q[t].double(), d_o[t].double(), o[t].double()
        s = SCALE * (qd @ k)
        p = torch.exp(s - lse[t].double())
        dp, back = do @ k, (do * od).abs().sum(2)
        ds = SCALE * p * (dp - (do * od).sum(2))
        e_s = 512 * E * SCALE * (qd.abs() @ k.abs()) + 12 * E * (s.abs() + lse[t].abs() + 1)
        e_dp = 512 * E * (do.abs() @ k.abs()) + 530 * E * back + 4 * E * dp.abs()
        e_ds, e_p = ds.abs() * (U + 2 * e_s) + SCALE * p * e_dp * (1 + U), p * (U + 2 * e_s)
        got = torch.einsum("th,thd->d", ds, qd) + torch.einsum("th,thd->d", p, do)
        size = torch.einsum("th,thd->d", ds.abs(), qd.abs()) + torch.einsum("th,thd->d", p, do.abs())
        tol = torch.einsum("th,thd->d", e_ds, qd.abs()) + torch.einsum("th,thd->d", e_p, do.abs())
        tol += (128 + t.numel()) * E * size + U * got.abs() + 1e-30
        err = (dkv[j].double() - got).abs()
        assert torch.all(err <= tol), (j, t.numel(), float((err / tol).max()))


def test_refusals_with_tensors(K):
    q, kv, d_o, lse = _inputs(3, 20, 37)
    tok = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    ok = lambda **kw: K.kpool_sparse_mla_bwd(**{**dict(q=q, kv=kv, tok_idx=tok, o=q, lse=lse, d_o=d_o, softmax_scale=0.1), **kw})  # noqa: E731
    ok()
    for kw in (dict(o=q[:2]), dict(d_o=d_o.transpose(1, 2)), dict(lse=lse[:, :32]), dict(tok_idx=tok[:2]), dict(kv=kv[:, :256]),
               dict(dq=q[:1]), dict(dkv=kv[:3]), dict(d_lse=lse[:1]), dict(kv=kv.cpu())):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(q=q.half()), dict(d_o=d_o.float()), dict(lse=lse.double()), dict(tok_idx=tok.long()), dict(d_lse=lse.half())):
        with pytest.raises(TypeError):
            ok(**kw)
    with pytest.raises(K.KPoolError):
        ok(q=q[:, :32].contiguous(), o=q[:, :32].contiguous(), d_o=d_o[:, :32].contiguous(), lse=lse[:, :32].contiguous())
    pools = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="rows of q"):
        K.kpool_sparse_mla_bwd_pools(q, kv, pools, q, lse, d_o, 4, 8, 0.1)
    with pytest.raises(ValueError, match="go together"):
        K.kpool_sparse_mla_bwd_pools(q, kv[:3], pools, q, lse, d_o, 4, 8, 0.1, cu_seqlens=pools[0])
    with pytest.raises(K.KPoolError):
        ok(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("rows", [400, 20])
@pytest.mark.parametrize("limit_ns", [1, 3000])
def test_expired_waits(K, limit_ns, rows):
    """With the wait limit lowered the call reports KPOOL_STATUS_TIMEOUT (1 ns) or finishes; the next call at
    the default limit is clean and right."""
    T, Tk = rows, 300
    q, kv, d_o, _ = _inputs(T, Tk, 41)
    tok = _lists(np.random.default_rng(1), T, Tk, 260, [260, 100, 0, 65])
    o, lse = K.kpool_sparse_mla_fwd(q, kv, tok, SCALE)
    ws = torch.zeros(K.kpool_sparse_mla_bwd_workspace_size(T, Tk), dtype=torch.uint8, device="cuda")
    K.kpool_debug_set_wait_limit_ns(limit_ns)
    try:
        K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
        status = K.kpool_read_status(ws)
    finally:
        assert K.kpool_debug_set_wait_limit_ns(0) == limit_ns
    if limit_ns == 1 and rows == 400:
        assert status & K.STATUS_TIMEOUT
    dq, dkv = K.kpool_sparse_mla_bwd(q, kv, tok, o, lse, d_o, SCALE, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    Grads(q, kv, _rows_of(tok, Tk), o, lse, d_o, SCALE).check(dq, dkv)

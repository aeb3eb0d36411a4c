"""The sparse attention over a paged cache (kpool_sparse_mla_fwd_pools_paged) against
the definition in 64 bits and against the flat form, and a run of the cache, the
indexer, this attention and the backward pass together.  Tolerances: mla_grad_checks."""
import numpy as np
import pytest
import torch

from mla_grad_checks import DC, H, Grads, check_forward
from sparse_attention_kpool_compress_gb300 import workloads as W

pytestmark = pytest.mark.gpu
SCALE = W.MLA_SCALE


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Case:
    """A batch over a paged store: what is not in a sequence is NaN."""

    def __init__(self, seed, lens, queries, kp, budget, page, tail=True, layers=1, shuffled=True, spare=3, extra_rows=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        lens, queries = np.asarray(lens), np.asarray(queries)
        B = len(lens)
        self.lens, self.queries, self.kp, self.budget, self.page, self.tail = lens, queries, kp, budget, page, tail
        used = -(-lens // page)
        n_pages, wide = int(used.sum()) + spare, int(max(1, used.max())) + 1
        ids = rng.permutation(n_pages)
        rows = B + extra_rows
        where = rng.permutation(rows)[:B] if shuffled else np.arange(B)
        table = np.full((rows, wide), -7, np.int32)
        row_lens = np.full(rows, -5, np.int32)
        store = torch.full((layers, n_pages, page, DC), torch.nan, dtype=torch.bfloat16, device="cuda")
        self.kv = store[layers - 1]
        self.flat, at = [], 0
        for b in range(B):
            table[where[b], :used[b]] = ids[at:at + used[b]]
            row_lens[where[b]] = lens[b]
            at += used[b]
            c = torch.randn(int(lens[b]), DC, generator=g, device="cuda").to(torch.bfloat16)
            self.flat.append(c)
            pages = torch.full((int(used[b]), page, DC), torch.nan, dtype=torch.bfloat16, device="cuda")
            pages.view(-1, DC)[:int(lens[b])] = c
            self.kv[torch.from_numpy(table[where[b], :used[b]].astype(np.int64)).cuda()] = pages
        self.table, self.row_lens = _dev(table), _dev(row_lens)
        self.ids = _dev(where) if shuffled or rows != B else None
        self.cu_q = _dev(np.concatenate([[0], np.cumsum(queries)]))
        self.pos = _dev(lens - queries)
        self.cu_pools_h = np.concatenate([[0], np.cumsum(lens // kp)])
        self.cu_pools = _dev(self.cu_pools_h)
        T = int(queries.sum())
        self.q = (torch.randn(T, H, DC, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        sel, self.lists = [], []
        for b in range(B):
            for tau in range(lens[b] - queries[b], lens[b]):
                n = (tau + 1) // kp
                mine = np.sort(rng.choice(n, size=min(n, budget), replace=False)) if n else np.zeros(0, int)
                row = np.full(budget, -1, np.int32)
                row[:len(mine)] = mine + self.cu_pools_h[b]
                sel.append(row)
                toks = (mine[:, None] * kp + np.arange(kp)).reshape(-1)
                if tail:
                    toks = np.concatenate([toks, np.arange((tau + 1) // kp * kp, tau + 1)])
                self.lists.append((b, toks))
        self.sel = _dev(np.array(sel).reshape(-1, budget))

    def call(self, K, **kw):
        kw = {**dict(seq_ids=self.ids, always_select_tail=self.tail), **kw}
        return K.kpool_sparse_mla_fwd_pools_paged(self.q, self.kv, self.table, self.row_lens, self.sel, self.kp,
                                                  self.kp * self.budget, SCALE, self.cu_q, self.pos, self.cu_pools, **kw)

    def workspace(self, K, fill=0):
        return torch.full((K.kpool_sparse_mla_paged_workspace_size(self.q.shape[0], self.kp, self.kp * self.budget),), fill,
                          dtype=torch.uint8, device="cuda")

    def check(self, o, lse, what="", rows=None):
        for t, (b, toks) in enumerate(self.lists):
            if rows is None or t in rows:
                check_forward(o[t], lse[t], self.q[t], self.flat[b][torch.from_numpy(toks).cuda()], SCALE, (what, t, len(toks)))


@pytest.mark.parametrize("page", [1, 16, 24, 64, 128])
@pytest.mark.parametrize("kp,budget,tail", [(4, 40, True), (8, 3, False), (1, 200, True), (64, 3, True)])
def test_against_the_definition(K, page, kp, budget, tail):
    """Ragged lengths around pages and blocks, one to several queries, sequences without any, rows that see
    nothing (no complete pool, no tail)."""
    c = Case(7 * page + kp, [1, 130, kp * budget, kp * budget + 3, 257, 777, 64], [1, 5, 2, 1, 0, 7, 3], kp, budget, page,
             tail, layers=2, extra_rows=2)
    ws = c.workspace(K, 0x7F)
    o, lse = c.call(K, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    c.check(o, lse)


@pytest.mark.parametrize("lens,queries", [([9001], [1]), ([2500, 2049, 2051], [1, 1, 1]), ([3000] * 20, [1] * 20),
                                          ([2300] * 40, [3] * 40), ([2200] * 152, [1] * 152), ([2100] * 170, [1] * 170),
                                          ([2600, 2222], [200, 190])])
def test_numbers_of_rows(K, lens, queries):
    """One row to more than the GPU has SMs, with the full budget: rows are cut over SMs or not."""
    c = Case(len(lens), lens, queries, 4, 512, 64)
    ws = c.workspace(K, 0x7F)
    o, lse = c.call(K, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    n = c.q.shape[0]
    c.check(o, lse, rows=set(range(0, n, max(1, n // 12))) | {n - 1})
    # nothing that the last call left is seen by the next
    again = c.call(K, workspace=ws)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_equals_the_flat_form(K):
    """Rows that are not cut are the flat call's bit for bit; others within the rounding of p."""
    lens, queries, kp, budget = np.array([1500, 3100, 77, 2048]), np.array([100, 140, 20, 60]), 4, 64
    c = Case(3, lens, queries, kp, budget, 32)
    o, lse = c.call(K)
    cu_k = _dev(np.concatenate([[0], np.cumsum(lens)]))
    o2, lse2 = K.kpool_sparse_mla_fwd_pools_at(c.q, torch.cat(c.flat), c.sel, kp, kp * budget, SCALE, c.cu_q, c.pos, cu_k,
                                               c.cu_pools)
    assert torch.allclose(lse, lse2, rtol=0, atol=2e-5)
    assert torch.allclose(o.float(), o2.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    c.check(o, lse, rows={0, 99, 100, 240, 319})


def test_bad_pages_are_skipped(K):
    """A page id, a table row, a length and a position out of range: told by the status, other rows right,
    nothing out of range followed."""
    c = Case(5, [300, 500, 260, 400, 350], [2, 3, 1, 2, 2], 4, 30, 32)
    ws = c.workspace(K)
    ids = c.ids.clone()
    at = c.ids.long()
    c.call(K, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    good = [t for t, (b, _) in enumerate(c.lists) if b == 0]

    def refused(what, restore, rows=good):
        o, lse = c.call(K, workspace=ws)
        assert K.kpool_read_status(ws) == K.STATUS_BAD_PAGE, what
        c.check(o, lse, what, rows=set(rows))
        restore()

    keep = c.table.clone()
    for bad in (-1, c.kv.shape[0], 2 ** 31 - 1, -2 ** 31):
        c.table[at[1]] = bad
        refused(("page", bad), lambda: c.table.copy_(keep))
    for bad in (-1, c.table.shape[0], 2 ** 31 - 1):
        c.ids[2] = bad
        refused(("row", bad), lambda: c.ids.copy_(ids))
    keep_l = c.row_lens.clone()
    for bad in (-3, 2 ** 31 - 1, 100):
        c.row_lens[at[3]] = bad
        refused(("length", bad), lambda: c.row_lens.copy_(keep_l))
    keep_p = c.pos.clone()
    for bad in (-9, 349, 2 ** 31 - 1):
        c.pos[4] = bad
        refused(("position", bad), lambda: c.pos.copy_(keep_p))
    # pools that are not the sequence's are skipped without a word, as by the expansion
    sel = c.sel.clone()
    c.sel[-1] = -1
    c.sel[-2, 0], c.sel[-2, 1] = 2 ** 31 - 1, 0
    o, lse = c.call(K, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    c.check(o, lse, rows=set(good))
    c.sel.copy_(sel)
    cu = c.cu_q.clone()
    for i, bad in ((0, 1), (5, 3), (2, 9), (3, -4), (5, 2 ** 31 - 1)):
        c.cu_q[i] = bad
        c.call(K, workspace=ws)
        assert K.kpool_read_status(ws) & K.STATUS_BAD_SEQLENS, (i, bad)
        c.cu_q.copy_(cu)
    o, lse = c.call(K, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    c.check(o, lse)


@pytest.mark.parametrize("queries", [[1, 2, 1], [60, 50, 70]])
def test_rows_outside_the_batch_stay(K, queries):
    """A padded q: rows behind the last sequence (and in front of the first) are left as they were, told by
    the status; the others are right.  Cut rows and whole ones."""
    c = Case(19, [700, 400, 550], queries, 4, 100, 64)
    n, pad = c.q.shape[0], 5
    c.q = torch.cat([c.q, torch.full((pad, H, DC), torch.nan, device="cuda", dtype=torch.bfloat16)])
    c.sel = torch.cat([c.sel, torch.full((pad, c.budget), 2 ** 31 - 1, device="cuda", dtype=torch.int32)])
    ws = c.workspace(K)
    o, lse = torch.full_like(c.q, 7.0), torch.full((n + pad, H), 7.0, device="cuda")
    c.call(K, workspace=ws, o=o, lse=lse)
    assert K.kpool_read_status(ws) == K.STATUS_BAD_SEQLENS
    assert torch.all(o[n:] == 7) and torch.all(lse[n:] == 7)
    c.check(o, lse, rows=set(range(0, n, max(1, n // 9))) | {n - 1})
    # and the first sequence's first row taken out
    o.fill_(7.0)
    lse.fill_(7.0)
    c.cu_q[0], c.pos[0] = 1, int(c.pos[0]) + 1
    c.call(K, workspace=ws, o=o, lse=lse)
    assert torch.all(o[0] == 7) and torch.all(lse[0] == 7) and torch.all(o[n:] == 7)
    c.check(o, lse, rows={1, n - 1})


def test_degenerate_batches(K):
    """No query rows, and rows whose masks leave nothing (o = 0, lse = -inf)."""
    c = Case(9, [50, 3], [0, 0], 4, 8, 16)
    o, lse = c.call(K)
    assert o.shape == (0, H, DC) and lse.shape == (0, H)
    c = Case(10, [3, 2, 7], [3, 1, 7], 4, 8, 16, tail=False)
    o, lse = c.call(K)
    c.check(o, lse)
    assert torch.isneginf(lse[0]).all() and torch.all(o[0] == 0)


def test_a_nan_query_stays_in_its_row(K):
    c = Case(11, [2100, 2100], [2, 2], 4, 512, 64)
    c.q[1, 3, 7] = torch.nan
    o, lse = c.call(K)
    assert torch.isnan(o[1, 3]).all() and torch.isnan(lse[1, 3])
    assert torch.isfinite(o[1, :3]).all() and torch.isfinite(o[[0, 2, 3]]).all()
    c.check(o, lse, rows={0, 2, 3})


def test_streams_and_graphs(K):
    """Another stream than the tensors' own; two calls in one workspace captured and replayed after the
    cache changed."""
    c, d = Case(12, [900, 2100, 300], [1, 1, 4], 4, 512, 64), Case(13, [700] * 5, [40] * 5, 4, 100, 16)
    ws = torch.zeros(max(c.workspace(K).numel(), d.workspace(K).numel()), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.call(K, workspace=ws), d.call(K, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    some = set(range(0, 200, 17))
    c.check(*got[0])
    d.check(*got[1], rows=some)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.call(K, workspace=ws), d.call(K, workspace=ws)
    keep = c.kv.clone()
    c.kv.zero_()
    graph.replay()
    assert torch.all(got[0][0] == 0)
    c.kv.copy_(keep)
    for _ in range(3):
        graph.replay()
    c.check(*got[0])
    d.check(*got[1], rows=some)
    assert K.kpool_read_status(ws) == 0


def test_a_cache_of_more_than_4_gib(K):
    """Pages behind 2^32 bytes and 2^31 elements, several layers apart."""
    page, layers, n_pages = 64, 3, 26000
    store = torch.zeros(n_pages, layers, page, DC, dtype=torch.bfloat16, device="cuda")
    c = Case(14, [700, 300], [2, 3], 4, 60, page, shuffled=False)
    n = int((c.table >= 0).sum())
    new = torch.randperm(n_pages - 1, generator=torch.Generator().manual_seed(1))[:n].cuda()
    new[:3] = torch.tensor([n_pages - 1, n_pages - 1 - 64, n_pages // 2], device="cuda")
    new = new.unique()[torch.randperm(new.unique().numel(), generator=torch.Generator().manual_seed(2)).cuda()]
    while new.numel() < n:
        new = torch.cat([new, (new.max() - 7).view(1)]).unique()
    live = c.table >= 0
    old = c.table[live].long()
    store[new, 2] = c.kv[old]
    c.table[live] = new.int()
    c.kv = store[:, 2]
    o, lse = c.call(K)
    c.check(o, lse)


def test_refusals_with_tensors(K):
    c = Case(15, [100, 90], [1, 2], 4, 8, 16, shuffled=False)
    with pytest.raises(ValueError, match="contiguous"):
        c.call(K, o=c.q.transpose(0, 1))
    for kw in (dict(o=c.q[:1]), dict(lse=torch.zeros(3, 32, device="cuda")), dict(seq_ids=c.cu_q)):
        with pytest.raises(ValueError):
            c.call(K, **kw)
    with pytest.raises(K.KPoolError):
        c.call(K, workspace=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    keep = c.kv
    c.kv = keep.float()
    with pytest.raises(TypeError):
        c.call(K)
    c.kv = keep[:, :, :256]
    with pytest.raises(ValueError):
        c.call(K)
    c.kv = keep.transpose(0, 1)
    with pytest.raises(ValueError):
        c.call(K)


def test_rollout_and_training_step(K):
    """A rollout's calls and the training step's, together: a prompt written in pieces and forked, answers
    decoded token by token over the chosen pools, then gradients through the flat form of the same tokens.
    The rollout's outputs and the training forward's are both the definition's, and so are the gradients."""
    kp, topk, page, heads, width = 4, 64, 32, 16, 128
    g = torch.Generator("cuda").manual_seed(3)
    prompt, answers, steps = 205, 3, 5
    total = prompt + steps

    def rnd(*shape, s=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)

    # what the layers in front would give, for every token of each answer (the prompt's are shared)
    def tokens(*shape, **kw):
        x = rnd(answers, total, *shape, **kw)
        x[:, :prompt] = x[:1, :prompt]
        return x

    q, kv = tokens(H, DC), tokens(DC)
    iq, ik, gate, iw = tokens(heads, width), tokens(width), tokens(width), tokens(heads, dtype=torch.float32)
    ape = rnd(kp, width, s=0.1, dtype=torch.float32)
    pages = K.kpool_pages_new(answers, 40, 8, page)
    latents = torch.full((40, page, DC), torch.nan, dtype=torch.bfloat16, device="cuda")
    n_pools = -(-total // kp)
    room = _dev(np.arange(answers + 1) * n_pools)            # pooled keys of each answer, with room to grow
    pooled = torch.zeros(answers * n_pools, width, dtype=torch.bfloat16, device="cuda")
    outs = torch.zeros(answers, total, H, DC, dtype=torch.bfloat16, device="cuda")
    logs = torch.zeros(answers, total, H, device="cuda")

    def step(seqs, lo, hi):
        """Tokens lo..hi of these sequences."""
        n, m = len(seqs), hi - lo
        ids, cu = _dev(seqs), _dev(np.arange(n + 1) * m)
        begin = K.kpool_pages_extend(pages, ids, _dev([m] * n))
        assert begin.tolist() == [lo] * n
        K.kpool_pages_write(pages, ids, begin, cu, kv[seqs, lo:hi].reshape(-1, DC).contiguous(), latents)
        for s in seqs:
            whole = hi // kp
            pooled[s * n_pools:s * n_pools + whole] = K.kpool_compress(ik[s, :hi].contiguous(), gate[s, :hi].contiguous(), ape, kp)
        first = _dev([s * n_pools for s in seqs] + [(seqs[-1] + 1) * n_pools])
        sel, _ = K.kpool_score_topk_at(iq[seqs, lo:hi].reshape(-1, heads, width).contiguous(),
                                       iw[seqs, lo:hi].reshape(-1, heads).contiguous(), pooled, kp, topk, cu, begin, first)
        o, lse = K.kpool_sparse_mla_fwd_pools_paged(q[seqs, lo:hi].reshape(-1, H, DC).contiguous(), latents, pages.page_table,
                                                    pages.seq_lens, sel, kp, topk, SCALE, cu, begin, first, seq_ids=ids)
        outs[seqs, lo:hi], logs[seqs, lo:hi] = o.view(n, m, H, DC), lse.view(n, m, H)
        return sel

    step([0], 0, 130)
    step([0], 130, prompt)
    K.kpool_pages_fork(pages, _dev([0, 0]), _dev([1, 2]), [latents])
    outs[1:, :prompt], logs[1:, :prompt] = outs[:1, :prompt], logs[:1, :prompt]
    for i in range(steps):
        step([0, 1, 2], prompt + i, prompt + i + 1)
    assert K.kpool_read_status(pages.workspace) == 0
    # the training step: the answers packed, the same indexer, flat rows
    T = answers * total
    cu = _dev(np.arange(answers + 1) * total)
    cu_pools, P = K.kpool_num_pools((np.arange(answers + 1) * total).tolist(), T, kp)
    cu_pools = cu_pools.cuda()
    flat = lambda x: x.reshape(T, *x.shape[2:]).contiguous()  # noqa: E731
    tok, sel, _ = K.kpool_indexer_forward(flat(iq), flat(ik), flat(gate), ape, flat(iw), kp, topk, True, cu, cu_pools, P)
    qf, kvf = flat(q), flat(kv)
    o, lse = K.kpool_sparse_mla_fwd_pools(qf, kvf, sel, kp, topk, SCALE, cu, cu_pools)
    lists = [r[r >= 0].long() for r in tok]
    for t in list(range(0, T, 41)) + [prompt, T - 1, total + prompt]:
        check_forward(o[t], lse[t], qf[t], kvf[lists[t]], SCALE, ("train", t))
        check_forward(flat(outs)[t], flat(logs)[t], qf[t], kvf[lists[t]], SCALE, ("rollout", t))
    d_o = rnd(T, H, DC, s=0.1)
    d_o.view(answers, total, H, DC)[:, :prompt] = 0          # the loss is on the answers
    dq, dkv = K.kpool_sparse_mla_bwd_pools(qf, kvf, sel, o, lse, d_o, kp, topk, SCALE, cu, cu_pools)
    Grads(qf, kvf, lists, o, lse, d_o, SCALE).check(dq, dkv)
    # the same gradients from the answers' rows alone, at their positions
    rows = (torch.arange(answers, device="cuda")[:, None] * total + prompt + torch.arange(steps, device="cuda")).view(-1)
    dq2, dkv2 = K.kpool_sparse_mla_bwd_pools_at(qf[rows], kvf, sel[rows], o[rows], lse[rows], d_o[rows], kp, topk, SCALE,
                                                _dev(np.arange(answers + 1) * steps), _dev([prompt] * answers), cu, cu_pools)
    # (few rows are cut into runs, whose sums are joined in FP32)
    assert torch.allclose(dq2.float(), dq[rows].float(), rtol=2.0 ** -7, atol=1e-6) and torch.all(dq.view(answers, total, H, DC)[:, :prompt] == 0)
    assert torch.allclose(dkv2.float(), dkv.float(), rtol=2.0 ** -7, atol=1e-5)


@pytest.mark.parametrize("limit_ns", [1, 3000])
def test_expired_waits(K, limit_ns):
    """With the wait limit lowered the call reports KPOOL_STATUS_TIMEOUT (1 ns) or finishes; the next call at
    the default limit is clean and right, for whole rows and for rows that are cut."""
    for c in (Case(16, [900] * 4, [60] * 4, 4, 100, 64), Case(17, [2500, 2200], [1, 2], 4, 512, 64)):
        ws = c.workspace(K)
        K.kpool_debug_set_wait_limit_ns(limit_ns)
        try:
            c.call(K, workspace=ws)
            status = K.kpool_read_status(ws)
        finally:
            assert K.kpool_debug_set_wait_limit_ns(0) == limit_ns
        if limit_ns == 1:
            assert status & K.STATUS_TIMEOUT
        o, lse = c.call(K, workspace=ws)
        assert K.kpool_read_status(ws) == 0
        c.check(o, lse, rows={0, 1, 2, 77, 239})


def test_rising_scores(K):
    """Scores that rise by more than the headroom (8 in base 2) from block to block: the reference maximum and
    the output so far are rescaled at every block, cut rows and whole ones."""
    for queries in ([1], [60, 60, 60]):
        lens = [1400] * len(queries)
        c = Case(18, lens, queries, 1, 1400, 64)
        g = torch.Generator("cuda").manual_seed(4)
        c.q.zero_()
        c.q[:, :, 0] = torch.linspace(0.5, 1.5, H, device="cuda") / SCALE
        for b in range(len(lens)):
            x = torch.randn(1400, DC, generator=g, device="cuda") * 0.2
            x[:, 0] = torch.arange(1400, device="cuda") * 0.15
            c.flat[b] = x.to(torch.bfloat16)
            row = b if c.ids is None else int(c.ids[b])
            ids = c.table[row, :22].long()
            c.kv[ids] = torch.cat([c.flat[b], torch.full((22 * 64 - 1400, DC), torch.nan, device="cuda",
                                                         dtype=torch.bfloat16)]).view(22, 64, DC)
        o, lse = c.call(K)
        c.check(o, lse, rows={0, 59, 60, 100, 179})

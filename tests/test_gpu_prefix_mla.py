"""Attention over a paged cache for groups of sequences that share a prefix
(kpool_shared_prefix_mla_fwd) against its definition in 64 bits.

Tolerance, derived from the arithmetic.  Scores are exact BF16 products summed
in FP32: with u = 2^-23 for one step of a sum (a tensor core's sums may cut
instead of round), 512 terms of magnitude sum S = scale * sum_d |q_d c_d| give an
error of at most ds = 512 u S.  A softmax weight is then off by a factor within
exp(+-2 ds) (its own score and the normaliser), its rounding to BF16 adds 2^-8
of itself, hardware 2^x and the FP32 sums 2^-20, and the output's rounding 2^-8
of |o|.  With A = sum_j w_j |c_j,d| and w the exact weights:

    |o - exact| <= (2^-8 + 2^-20 + 3 ds) A + 2^-8 |exact|
    |lse - exact| <= ds + 2^-20 (1 + |exact|)
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

W = 512
BAD_SEQLENS, BAD_PAGE = 2, 4


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


class Case:
    """groups: [(prefix, [(length, n_q), ...]), ...]; lengths count the prefix."""

    def __init__(self, groups, H=64, page=64, seed=0, scale=W ** -0.5, spare=3, junk=float("nan"), sharp=2.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.RandomState(seed)
        self.H, self.page, self.scale = H, page, scale
        self.prefix = [p for p, _ in groups]
        self.lens = [l for _, seqs in groups for l, _ in seqs]
        self.nq = [n for _, seqs in groups for _, n in seqs]
        self.cu_g = np.concatenate([[0], np.cumsum([len(s) for _, s in groups])])
        self.cu_q = np.concatenate([[0], np.cumsum(self.nq)])
        B = len(self.lens)
        wide = max(1, max(-(-l // page) for l in self.lens) + 1)
        self.table = np.full((B, wide), -1, np.int32)
        rows, n = [], 0
        for gi, (p, seqs) in enumerate(groups):
            first = self.cu_g[gi]
            p = min(max(p, 0), seqs[0][0]) if seqs else 0
            for b in range(first, self.cu_g[gi + 1]):
                whole = p // page if b > first else 0
                self.table[b, :whole] = self.table[first, :whole]
                for j in range(whole, -(-self.lens[b] // page)):
                    self.table[b, j] = n
                    n += 1
        self.n_pages = n + spare
        perm = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.where(self.table >= 0, perm[self.table], -1).astype(np.int32)
        kv = torch.randn(self.n_pages, page, W, generator=g).to(torch.bfloat16)
        self.q = (sharp * torch.randn(int(self.cu_q[-1]), H, W, generator=g)).to(torch.bfloat16)
        # what lies behind a sequence's end, and in pages that nobody holds, is junk
        held = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for b, l in enumerate(self.lens):
            for j in range(-(-l // page)):
                held[int(self.table[b, j]), :max(0, min(page, l - j * page))] = True
        kv[~held] = junk
        self.kv, self.held = kv, held
        # the shared part of a page that a prefix ends in: every sequence has its copy
        for gi, (p, seqs) in enumerate(groups):
            first = self.cu_g[gi]
            if seqs:
                p = min(max(p, 0), seqs[0][0])
                for b in range(first + 1, self.cu_g[gi + 1]):
                    u = min(p % page, max(0, self.lens[b] - p // page * page))
                    if u and p // page < wide and self.table[b, p // page] >= 0:
                        self.kv[int(self.table[b, p // page]), :u] = self.kv[int(self.table[first, p // page]), :u]

    def args(self, dev="cuda"):
        i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
        return [self.q.to(dev), self.kv.to(dev), i(self.table), i(self.lens), i(self.cu_q), i(self.cu_g),
                i(self.prefix), self.scale]

    def tokens(self, b):
        """[length, 512] of sequence b in 64 bits, each sequence through its own pages."""
        pos = np.arange(self.lens[b])
        return self.kv[torch.from_numpy(self.table[b, pos // self.page].astype(np.int64)),
                       torch.from_numpy(pos % self.page)].double()

    def check(self, o, lse, rows=None, note=""):
        o, lse = o.double().cpu(), lse.double().cpu()
        assert o.shape == self.q.shape and lse.shape == self.q.shape[:2]
        u = 2.0 ** -23
        for b in range(len(self.lens)):
            c = self.tokens(b)
            for i in range(self.nq[b]):
                t = int(self.cu_q[b]) + i
                if rows is not None and t not in rows:
                    continue
                n = max(0, self.lens[b] - self.nq[b] + i + 1)
                q = self.q[t].double()
                if n == 0:
                    assert torch.all(o[t] == 0) and torch.all(torch.isneginf(lse[t])), (note, t)
                    continue
                s = self.scale * (q @ c[:n].T)
                want = torch.logsumexp(s, -1)
                w = torch.exp(s - want[:, None])
                exact, A = w @ c[:n], w @ c[:n].abs()
                ds = 512 * u * self.scale * (q.abs() @ c[:n].abs().T).amax(-1)
                tol = (2.0 ** -8 + 2.0 ** -20 + 3 * ds)[:, None] * A + 2.0 ** -8 * exact.abs()
                off = (o[t] - exact).abs()
                assert torch.all(off <= tol), (note, t, float((off / tol).max()))
                assert torch.all((lse[t] - want).abs() <= ds + 2.0 ** -20 * (1 + want.abs())), (note, t)


def run(K, case, **kw):
    ws = torch.empty(max(256, K.kpool_shared_prefix_mla_workspace_size(
        len(case.q), case.H, len(case.lens), len(case.prefix))), dtype=torch.uint8, device="cuda")
    o, lse = K.kpool_shared_prefix_mla_fwd(*case.args(), workspace=ws, **kw)
    torch.cuda.synchronize()
    assert K.kpool_read_status(ws) == 0
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [64, 16])
def test_groups(K, page, H):
    """Ragged groups; prefixes that end inside a page, at its end, and of no token."""
    c = Case([(300, [(301, 1), (300 + page, 1), (417, 1)]),
              (2 * page, [(2 * page + 1, 1), (2 * page + 40, 1)]),
              (0, [(77, 1), (1, 1)]),
              (513, [(700, 1)])], H=H, page=page, seed=page + H)
    c.check(*run(K, c))


@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 24, 48, 65, 100, 127, 128])
def test_heads(K, H):
    c = Case([(130, [(140, 2), (131, 1), (260, 3)]), (5, [(9, 1), (5, 1)])], H=H, seed=H)
    c.check(*run(K, c))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1025])
def test_lengths_around_tiles(K, length):
    """One sequence of each length alone, as a prefix of two, and behind a prefix."""
    c = Case([(0, [(length, 1)]), (length, [(length, 1), (length + 1, 1)]), (33, [(40, 1), (33 + length, 1)])],
             H=8, page=16, seed=length)
    c.check(*run(K, c))


def test_several_queries_see_their_own_prefixes(K):
    """Chunks: query i of n sees length - n + i + 1 tokens, the first ones fewer than the shared ones."""
    c = Case([(200, [(210, 30), (205, 5), (201, 150)]), (300, [(300, 40)]), (64, [(100, 100), (64, 64), (65, 3)])],
             H=16, page=32, seed=5)
    c.check(*run(K, c))


def test_rows_without_tokens(K):
    """Empty sequences, more queries than tokens, sequences without queries, groups without sequences."""
    c = Case([(10, [(0, 1), (4, 1)]), (3, [(3, 5), (0, 2)]), (7, []), (20, [(25, 0), (30, 2), (20, 0)]), (0, [(0, 3)])],
             H=8, page=16, seed=1)
    c.check(*run(K, c))


def test_prefix_lengths_out_of_range(K):
    """A prefix longer than the group's first sequence is cut to it; a negative one is none."""
    c = Case([(10 ** 6, [(100, 1), (130, 1)]), (-5, [(40, 1), (50, 2)]), (90, [(100, 1), (60, 1)])], H=8, page=32)
    c.check(*run(K, c))


def test_no_queries(K):
    c = Case([(10, [(20, 0)])], H=8, page=16)
    o, lse = run(K, c)
    assert o.shape == (0, 8, W) and lse.shape == (0, 8)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3e38, 0.0])
def test_what_lies_behind_the_end_is_not_read_into_results(K, junk):
    c = Case([(100, [(103, 1), (190, 2)]), (0, [(17, 1)])], H=64, page=64, junk=junk, seed=3)
    o, lse = run(K, c)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    c.check(o, lse)


def test_nan_and_infinite_queries_stay_in_their_rows(K):
    """A query head that is not finite gives NaN in its own row, and in no other of its tile."""
    c = Case([(300, [(301, 1), (420, 2)]), (0, [(33, 1)])], H=16, page=32, seed=23)
    sick = {(0, 3): float("nan"), (2, 0): float("inf"), (3, 15): float("nan")}
    q = c.q.clone()
    for (t, h), value in sick.items():
        c.q[t, h, 7] = value
    o, lse = run(K, c)
    for t, h in sick:
        assert torch.isnan(o[t, h]).all() and not torch.isfinite(lse[t, h])
        o[t, h], lse[t, h] = 0, 0
    c.q = q
    want_o, want_l = run(K, c)
    for t, h in sick:
        want_o[t, h], want_l[t, h] = 0, 0
    assert torch.equal(o, want_o) and torch.equal(lse, want_l)


def test_units_without_tokens_in_between(K):
    """Groups with and without shared tokens, sequences with and without their own, in turn."""
    groups = []
    for k in range(150):
        p = 40 if k % 3 == 0 else 0
        groups.append((p, [(p + (k % 5 == 0) * 20, 1), (p + (k % 7 == 1) * 300, k % 2)]))
    c = Case(groups, H=8, page=16, seed=29)
    c.check(*run(K, c))


def test_sharp_and_flat_scores(K):
    """Scores hundreds apart (one weight takes all), equal scores, and scores that rise along the tokens."""
    for sharp, seed in ((60.0, 1), (0.0, 2)):
        c = Case([(400, [(500, 1), (401, 1)])], H=16, sharp=sharp, seed=seed)
        c.check(*run(K, c), note=sharp)
    c = Case([(1000, [(1100, 1), (1300, 1)])], H=16, seed=4)
    # each later token scores higher: the reference maximum moves all the way
    d = torch.zeros(W)
    d[0] = 1
    for b in range(2):
        for j in range(c.lens[b]):
            c.kv[int(c.table[b, j // c.page]), j % c.page, 0] = j / 8.0
    c.q = (torch.ones(c.q.shape) * d * 20).to(torch.bfloat16)
    c.check(*run(K, c), note="rising")


def test_large_values(K):
    """Scores of a few thousand and latents of a few hundred: nothing overflows on the way."""
    c = Case([(300, [(333, 1), (512, 1)])], H=8, seed=8, sharp=200.0)
    c.kv = (c.kv.float() * 100).to(torch.bfloat16)
    c.check(*run(K, c))


def test_same_tokens_in_one_group_or_in_many(K):
    """Sharing is a matter of speed: the same batch without groups gives the same within the tolerance."""
    c = Case([(700, [(701, 1), (810, 1), (1000, 2)])], H=32, page=32, seed=9)
    c.check(*run(K, c))
    q, kv, table, lens, cu_q, _, _, scale = c.args()
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = K.kpool_shared_prefix_mla_fwd(q, kv, table, lens, cu_q, i([0, 1, 2, 3]), i([0, 300, 1000]), scale)
    c.check(o, lse)


def test_rows_of_a_larger_table(K):
    """seq_ids picks the batch out of a pool's table, in any order; pages strided as one layer of several."""
    c = Case([(50, [(60, 1), (70, 1)]), (20, [(33, 2)])], H=24, page=16, seed=6)
    q, kv, table, lens, cu_q, cu_g, pre, scale = c.args()
    ids = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    big = torch.full((7, table.shape[1]), 1 << 30, dtype=torch.int32, device="cuda")
    blens = torch.full((7,), -1, dtype=torch.int32, device="cuda")
    big[ids.long()] = table
    blens[ids.long()] = lens
    layers = torch.full((kv.shape[0], 3, 16, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    layers[:, 1] = kv
    ws = torch.empty(K.kpool_shared_prefix_mla_workspace_size(len(q), 24, 3, 2), dtype=torch.uint8, device="cuda")
    o = torch.full_like(q, 7)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    got = K.kpool_shared_prefix_mla_fwd(q, layers[:, 1], big, blens, cu_q, cu_g, pre, scale, seq_ids=ids,
                                        workspace=ws, o=o, lse=lse)
    torch.cuda.synchronize()
    assert K.kpool_read_status(ws) == 0 and got[0] is o and got[1] is lse
    c.check(o, lse)


def test_long_prefix(K):
    """A prefix split over all of the GPU, joined with tails of one token and of thousands."""
    c = Case([(20000, [(20001, 1), (23111, 1)] + [(20000 + 37 * k, 1) for k in range(2, 8)])], H=64, page=64, seed=11)
    o, lse = run(K, c)
    c.check(o, lse, rows={0, 1, 7})
    again = run(K, c)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])       # nothing depends on the order of arrival


def test_many_sequences(K):
    """More sequences and groups than a planning block has threads."""
    rng = np.random.RandomState(2)
    groups = []
    for _ in range(1100):
        p = int(rng.randint(0, 40))
        groups.append((p, [(p + int(rng.randint(0, 30)), int(rng.randint(0, 3))) for _ in range(rng.randint(0, 3))]))
    c = Case(groups, H=2, page=16, seed=12)
    c.check(*run(K, c))


@pytest.mark.parametrize("B, groups, queries, H", [(1024, 7, 1, 1), (1025, 1025, 1, 1), (4600, 30, 1, 1),
                                                   (6143, 1, 1, 1), (6144, 5, 1, 2), (40, 4, 16, 128),
                                                   (1, 1, 600, 128), (1500, 2, 1, 128)])
def test_lists_that_the_plan_holds_on_chip_and_not(K, B, groups, queries, H):
    """Lists and units on either side of what fits the plan's shared memory."""
    rng = np.random.RandomState(B + H)
    size = -(-B // groups)
    lists = [(9, [(9 + queries + int(rng.randint(0, 20)), queries) for _ in range(min(size, B - g * size))])
             for g in range(groups) if g * size < B]
    c = Case(lists, H=H, page=16, seed=B)
    o, lse = run(K, c)
    rows = set(rng.choice(len(c.q), min(len(c.q), 300), replace=False).tolist()) | {0, len(c.q) - 1}
    c.check(o, lse, rows=rows)


def test_bad_offsets(K):
    c = Case([(10, [(20, 1), (21, 1)])], H=8, page=16)
    q, kv, table, lens, cu_q, cu_g, pre, scale = c.args()
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(K.kpool_shared_prefix_mla_workspace_size(2, 8, 2, 1), dtype=torch.uint8, device="cuda")
    for a, b in (([0, 2, 1], [0, 2]), ([0, 1, 3], [0, 2]), ([1, 1, 2], [0, 2]), ([0, 1, 2], [0, 1]),
                 ([0, 1, 2], [1, 2]), ([0, -4, 2], [0, 2]), ([0, 1, 2 ** 31 - 1], [0, 2])):
        o, lse = torch.full_like(q, 3), torch.full(q.shape[:2], 3.0, device="cuda")
        K.kpool_shared_prefix_mla_fwd(q, kv, table, lens, i(a), i(b), pre, scale, workspace=ws, o=o, lse=lse)
        torch.cuda.synchronize()
        assert K.kpool_read_status(ws) == BAD_SEQLENS, (a, b)
        assert torch.all(o == 3) and torch.all(lse == 3)
    K.kpool_shared_prefix_mla_fwd(q, kv, table, lens, cu_q, cu_g, pre, scale, workspace=ws)
    assert K.kpool_read_status(ws) == 0


def test_bad_pages_and_lengths(K):
    """Ids and lengths out of range set the status; sequences that use none of them keep their results."""
    c = Case([(40, [(50, 1), (60, 1)]), (0, [(70, 1)])], H=16, page=16, seed=7)
    q, kv, table, lens, cu_q, cu_g, pre, scale = c.args()
    ws = torch.empty(K.kpool_shared_prefix_mla_workspace_size(3, 16, 3, 2), dtype=torch.uint8, device="cuda")
    for value in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[2, 1] = value
        o, lse = K.kpool_shared_prefix_mla_fwd(q, kv, t, lens, cu_q, cu_g, pre, scale, workspace=ws)
        assert K.kpool_read_status(ws) == BAD_PAGE, value
        c.check(o, lse, rows={0, 1})
    for value in (-1, 16 * table.shape[1] + 1, 2 ** 31 - 1):
        l = lens.clone()
        l[2] = value
        t = table.clone()
        t[2] = 0
        o, lse = K.kpool_shared_prefix_mla_fwd(q, kv, t, l, cu_q, cu_g, pre, scale, workspace=ws)
        assert K.kpool_read_status(ws) == BAD_PAGE, value
        c.check(o, lse, rows={0, 1})
    ids = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    o, lse = K.kpool_shared_prefix_mla_fwd(q, kv, table, lens, cu_q, cu_g, pre, scale, seq_ids=ids, workspace=ws)
    assert K.kpool_read_status(ws) == BAD_PAGE
    c.check(o, lse, rows={0, 1})


def test_streams_and_graphs(K):
    """On a side stream with its own workspace, next to the same call on another one; captured and replayed with
    lengths that change from replay to replay."""
    c = Case([(300, [(310, 1), (333, 1)]), (100, [(150, 1), (400, 1)])], H=32, page=64, seed=13)
    args = c.args()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([K.kpool_shared_prefix_mla_fwd(*args) for _ in range(4)])
    torch.cuda.synchronize()
    for o, lse in outs[0] + outs[1]:
        assert torch.equal(o, outs[0][0][0]) and torch.equal(lse, outs[0][0][1])
    c.check(*outs[0][0])

    ws = torch.empty(K.kpool_shared_prefix_mla_workspace_size(4, 32, 4, 2), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(args[0]), torch.empty(args[0].shape[:2], device="cuda")
    graphs = []
    for _ in range(2):                             # two graphs that share the workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.kpool_shared_prefix_mla_fwd(*args, workspace=ws, o=o, lse=lse)
        graphs.append(g)
    full = list(c.lens)
    for k, cut in enumerate(([0, 0, 0, 0], [3, 20, 40, 250], [310, 1, 149, 0], [0, 0, 0, 0])):
        c.lens = [l - x for l, x in zip(full, cut)]
        args[3].copy_(torch.tensor(c.lens, dtype=torch.int32))
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        assert K.kpool_read_status(ws) == 0
        c.check(o, lse, note=k)


def test_a_cache_of_more_than_4_gb(K):
    """Pages whose byte offsets pass 32 bits, next to pages at the beginning."""
    c = Case([(150, [(200, 1), (151, 2)]), (0, [(64, 1)])], H=16, page=64, seed=19)
    n = 70000
    big = torch.full((n, 64, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    to = torch.tensor([(n - 1 - 7 * k) if k % 2 else 5 * k for k in range(c.n_pages)])
    big[to.cuda()] = c.kv.cuda()
    args = c.args()
    args[1] = big
    table = torch.from_numpy(c.table).long()
    args[2] = torch.where(table >= 0, to[table.clamp(min=0)], -1).to(torch.int32).cuda()
    o, lse = K.kpool_shared_prefix_mla_fwd(*args)
    c.check(o, lse)


@pytest.mark.parametrize("limit", [1, 3000])
def test_expired_waits(K, limit):
    """Waits that run out at once, or part way through, end the call with KPOOL_STATUS_TIMEOUT (never with a hang), and
    the next call is whole."""
    c = Case([(3000, [(3001, 1), (3300, 1), (3010, 2)])], H=64, page=64, seed=17)
    args = c.args()
    ws = torch.empty(K.kpool_shared_prefix_mla_workspace_size(4, 64, 3, 1), dtype=torch.uint8, device="cuda")
    before = K.kpool_debug_set_wait_limit_ns(limit)
    try:
        for _ in range(3):
            K.kpool_shared_prefix_mla_fwd(*args, workspace=ws)
            status = K.kpool_read_status(ws)
            assert status in (0, 1) and (limit > 1 or status == 1)
    finally:
        K.kpool_debug_set_wait_limit_ns(before)
    o, lse = K.kpool_shared_prefix_mla_fwd(*args, workspace=ws)
    assert K.kpool_read_status(ws) == 0
    c.check(o, lse)


def test_a_limit_is_for_a_wait_not_for_a_piece(K):
    """Work of half a millisecond per block, whose spans begin and end inside a chunk, under a limit of 0.15."""
    c = Case([(32700, [(32790, 80)])], H=128, page=64, seed=23)
    want = run(K, c)
    before = K.kpool_debug_set_wait_limit_ns(150000)
    try:
        got = run(K, c)
    finally:
        K.kpool_debug_set_wait_limit_ns(before)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*got, rows={0, 79})


def test_a_rollout_from_pages_to_attention(K):
    """The calls together, as a rollout makes them: a prompt's rows written, forked for three samples, each grown by its
    own tokens step by step, attended through the pool's own table, one sample retired, the pool packed."""
    page, H = 16, 16
    g = torch.Generator().manual_seed(21)
    pages = K.kpool_pages_new(5, 40, 12, page)
    store = torch.full((2, 40, page, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    host = {}
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    def grow(seqs, more):
        rows = torch.randn(2, sum(more), W, generator=g).to(torch.bfloat16)
        begin = K.kpool_pages_extend(pages, i(seqs), i(more))
        cu = np.concatenate([[0], np.cumsum(more)])
        K.kpool_pages_write(pages, i(seqs), begin, i(cu), rows.cuda(), store)
        for k, s in enumerate(seqs):
            host[s] = torch.cat([host.get(s, torch.empty(2, 0, W, dtype=torch.bfloat16)),
                                 rows[:, cu[k]:cu[k + 1]]], 1)

    def attend(seqs, prefix):
        q = (2 * torch.randn(len(seqs), H, W, generator=g)).to(torch.bfloat16)
        o, lse = K.kpool_shared_prefix_mla_fwd(
            q.cuda(), store[1], pages.page_table, pages.seq_lens, i(list(range(len(seqs) + 1))), i([0, len(seqs)]),
            i([prefix]), W ** -0.5, seq_ids=i(seqs))
        c = Case.__new__(Case)
        c.H, c.scale, c.q = H, W ** -0.5, q
        c.lens, c.nq, c.cu_q = [host[s].shape[1] for s in seqs], [1] * len(seqs), np.arange(len(seqs) + 1)
        c.tokens = lambda b: host[seqs[b]][1].double()
        c.check(o, lse)

    grow([3], [37])
    K.kpool_pages_fork(pages, i([3, 3, 3]), i([0, 4, 1]), store)
    for s in (0, 4, 1):
        host[s] = host[3]
    for step in range(4):
        grow([0, 1, 4], [1, 1, 5])
        attend([4, 0, 1], 37)
    K.kpool_pages_free(pages, i([0, 3]))
    K.kpool_pages_compact(pages, store)
    for step in range(2):
        grow([4, 1], [16, 1])
        attend([1, 4], 37)
    assert int((pages.ref_count > 0).sum()) == 40 - pages.free_count.item()


@pytest.mark.parametrize("H", [1, 16, 128])
def test_the_log_sum_of_a_nan_query_is_nan(K, H):
    """In batches whose rows are joined by a block each (up to 512 rows) and by a warp each: -inf is a row without
    tokens, and a merge by lse would drop a NaN row that had it."""
    for n in (3, 512 // H + 1):
        c = Case([(300, [(301 + k % 3, 1) for k in range(n)]), (0, [(0, 1), (40, 1)])], H=H, page=32, seed=H)
        sick = {0: float("nan"), n - 1: float("inf"), n + 1: float("nan")}
        for t, value in sick.items():
            c.q[t, H - 1, 7] = value
        o, lse = run(K, c)
        for t in sick:
            assert torch.isnan(o[t, H - 1]).all() and torch.isnan(lse[t, H - 1]), (n, t)
        assert torch.all(o[n] == 0) and torch.isneginf(lse[n]).all()
        whole = torch.ones(lse.shape, dtype=torch.bool)
        whole[n] = False
        whole[list(sick), H - 1] = False
        assert torch.isfinite(lse.cpu()[whole]).all() and torch.isfinite(o.cpu()[whole]).all()


def test_tables_that_change_in_front_of_the_attention(K):
    """One captured chain of page calls with the attention right behind those that write the table, replayed: no two
    calls in a row read the same entries, and rows share cache lines."""
    page, H, prefix = 16, 16, 37
    g = torch.Generator().manual_seed(31)
    pages = K.kpool_pages_new(5, 64, 13, page)
    store = torch.full((64, page, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    first = torch.randn(prefix, W, generator=g).to(torch.bfloat16)
    begin = K.kpool_pages_extend(pages, i([0]), i([prefix]))
    K.kpool_pages_write(pages, i([0]), begin, i([0, prefix]), first.cuda(), store)
    K.kpool_pages_fork(pages, i([0]), i([2]), store)
    parent, child, both = i([0]), (i([2]), i([3])), (i([2, 0]), i([3, 0]))
    cu, more = i([0, 3, 4]), i([3, 1])
    rows = torch.empty(2, 4, W, dtype=torch.bfloat16, device="cuda")
    q = (2 * torch.randn(3, H, W, generator=g)).to(torch.bfloat16)
    cu_q, cu_g, pre, qd = i([0, 2, 3]), i([0, 2]), i([prefix]), q.cuda()
    tables = []

    def attend(k):
        out = K.kpool_shared_prefix_mla_fwd(qd, store, pages.page_table, pages.seq_lens, cu_q, cu_g, pre, W ** -0.5,
                                            seq_ids=both[k])
        tables.append(pages.page_table[2 + k].clone())
        return out

    def half(k):
        """A new child of sequence 0 in place of the old one, each grown; attended before and after packing."""
        K.kpool_pages_fork(pages, parent, child[k], store)
        K.kpool_pages_free(pages, child[1 - k])
        begin = K.kpool_pages_extend(pages, both[k], more)
        K.kpool_pages_write(pages, both[k], begin, cu, rows[k], store)
        a = attend(k)
        K.kpool_pages_compact(pages, store)
        return [a, attend(k)]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [half(1), half(0)]
    mine, read = first, []
    for k in range(24):
        # another sequence's pages come and go in between
        if k % 2 == 0:
            K.kpool_pages_extend(pages, i([4]), i([16 * (1 + k % 5)]))
        else:
            K.kpool_pages_free(pages, i([4]))
        new = torch.randn(2, 4, W, generator=g).to(torch.bfloat16)
        rows.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for h in (1, 0):
            c = Case.__new__(Case)
            c.H, c.scale, c.q, c.cu_q, c.nq = H, W ** -0.5, q, np.array([0, 2, 3]), [2, 1]
            held = [torch.cat([mine, new[h, :3]]).double(), torch.cat([mine, new[h, 3:]]).double()]
            c.lens, c.tokens = [len(x) for x in held], lambda b: held[b]
            a, b = outs[1 - h]
            c.check(*a, note=(k, h))
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (k, h)
            mine = torch.cat([mine, new[h, 3:]])
        read += [tuple(t.tolist()) for t in tables]
    assert len(set(read[::4])) > 15 and len(set(read[2::4])) > 15      # (the table did change)
    assert K.kpool_read_status(pages.workspace) == 0

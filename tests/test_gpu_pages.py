"""The paged cache's upkeep (kpool_pages_*) against a loop-by-loop restatement
of include/kpool.h on the host.  Everything here is whole numbers or copied
bytes, so every comparison is exact: tables, lengths, reference counts, the
free list in its order, and each byte of each store, those that no call should
touch among them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAD, SHORT = 4, 8            # KPOOL_STATUS_BAD_PAGE, KPOOL_STATUS_NO_PAGES


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_kpool_compress_gb300 as K
    return K


class Host:
    """The pool and its stores in numpy; each call returns the status word."""

    def __init__(self, n_seqs, n_pages, max_pages, page_size, stores):
        self.ps, self.n_pages, self.max = page_size, n_pages, max_pages
        self.table = np.full((n_seqs, max_pages), -1, np.int64)
        self.lens = np.zeros(n_seqs, np.int64)
        self.refs = np.zeros(n_pages, np.int64)
        self.free = list(range(n_pages - 1, -1, -1))
        self.stores = stores                       # uint8 [layers, n_pages, rows, row_bytes]

    def pages_of(self, n):
        return -(-n // self.ps)

    def _bad_list(self, ids, limit):
        return any(not 0 <= i < limit for i in ids) or len(set(ids)) < len(ids)

    def copy(self, src, dst):
        if self._bad_list(dst, self.n_pages) or any(not 0 <= s < self.n_pages for s in src) or set(src) & set(dst):
            return BAD
        for st in self.stores:
            st[:, dst] = st[:, src]
        return 0

    def fork(self, parents, children):
        n = len(self.lens)
        if self._bad_list(children, n) or any(not 0 <= p < n for p in parents):
            return BAD
        if any(p == c or self.lens[c] for p, c in zip(parents, children)):
            return BAD
        length = [int(self.lens[p]) for p in parents]
        if sum(l % self.ps > 0 for l in length) > len(self.free):
            return SHORT
        for p, c, l in zip(parents, children, length):
            whole, part = divmod(l, self.ps)
            self.table[c, :whole] = self.table[p, :whole]
            self.refs[self.table[c, :whole]] += 1
            if part:
                page = self.free.pop()
                self.table[c, whole] = page
                self.refs[page] = 1
                for st in self.stores:
                    rows = -(-part * st.shape[2] // self.ps)
                    st[:, page, :rows] = st[:, self.table[p, whole], :rows]
            self.lens[c] = l
        return 0

    def extend(self, seqs, more):
        n = len(self.lens)
        if self._bad_list(seqs, n) or any(m < 0 for m in more):
            return BAD, [-1] * len(seqs)
        need = 0
        for s, m in zip(seqs, more):
            l = int(self.lens[s])
            if l + m > self.max * self.ps or (m and l % self.ps and self.refs[self.table[s, l // self.ps]] != 1):
                return BAD, [-1] * len(seqs)
            need += self.pages_of(l + m) - self.pages_of(l)
        if need > len(self.free):
            return SHORT, [-1] * len(seqs)
        begin = [int(self.lens[s]) for s in seqs]
        for s, m, l in zip(seqs, more, begin):
            for j in range(self.pages_of(l), self.pages_of(l + m)):
                self.table[s, j] = self.free.pop()
                self.refs[self.table[s, j]] = 1
            self.lens[s] = l + m
        return 0, begin

    def write(self, seqs, begin, cu, rows, k):
        st, status = self.stores[k], 0
        rpp = st.shape[2]
        taken = set()
        for i, s in enumerate(seqs):
            for r in range(cu[i], cu[i + 1]):
                at = begin[i] + r - cu[i]
                col, row = divmod(at, rpp)
                ok = 0 <= s < len(self.lens) and begin[i] >= 0 and at * self.ps < self.lens[s] * rpp and col < self.max
                page = self.table[s, col] if ok else -1
                if not ok or not 0 <= page < self.n_pages or self.refs[page] != 1:
                    status = BAD
                    continue
                st[:, page, row] = rows[:, r]
                taken.add(r)
        return status if len(taken) == rows.shape[1] else BAD

    def release(self, seqs):
        if self._bad_list(seqs, len(self.lens)):
            return BAD
        gone = []
        for s in seqs:
            for j in range(self.pages_of(int(self.lens[s]))):
                p = self.table[s, j]
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    gone.append(int(p))
                self.table[s, j] = -1
            self.lens[s] = 0
        self.free += sorted(gone)
        return 0

    def compact(self):
        k = int((self.refs > 0).sum())
        src = [p for p in range(k, self.n_pages) if self.refs[p] > 0]
        dst = [p for p in range(k) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            for st in self.stores:
                st[:, b] = st[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, l in enumerate(self.lens):
            for j in range(self.pages_of(int(l))):
                self.table[s, j] = to.get(int(self.table[s, j]), self.table[s, j])
        self.free = list(range(self.n_pages - 1, k - 1, -1))
        return 0


class Both:
    """The same pool on the host and on the GPU."""

    def __init__(self, K, n_seqs=7, n_pages=40, max_pages=6, page_size=16, layers=2, seed=0, inner_layers=False):
        self.K, g = K, np.random.RandomState(seed)
        rows = [page_size] + ([page_size // 4] if page_size % 4 == 0 else [])
        widths = [48, 16]                          # bytes: three and one 16-byte pieces
        host = [g.randint(0, 256, (layers, n_pages, r, w)).astype(np.uint8) for r, w in zip(rows, widths)]
        if inner_layers:                           # layers within pages: [n_pages, layers, rows, width]
            self.stores = [torch.from_numpy(h).cuda().transpose(0, 1).contiguous().transpose(0, 1) for h in host]
        else:
            self.stores = [torch.from_numpy(h).cuda() for h in host]
        self.host = Host(n_seqs, n_pages, max_pages, page_size, [h.copy() for h in host])
        self.gpu = K.kpool_pages_new(n_seqs, n_pages, max_pages, page_size)
        self.ws = torch.empty(max(256, K.kpool_pages_workspace_size(1000, n_seqs, n_pages)), dtype=torch.uint8,
                              device="cuda")
        self.rng = g

    def i32(self, a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    def check(self, want, note=""):
        assert self.K.kpool_read_status(self.ws) == want, note
        h, p = self.host, self.gpu
        assert p.free_count.item() == len(h.free), note
        assert p.free_list.cpu().tolist()[:len(h.free)] == h.free, note
        assert p.seq_lens.cpu().tolist() == h.lens.tolist(), note
        assert p.ref_count.cpu().tolist() == h.refs.tolist(), note
        table = p.page_table.cpu().numpy()
        for s, l in enumerate(h.lens):
            n = h.pages_of(int(l))
            assert table[s, :n].tolist() == h.table[s, :n].tolist(), (note, s)
        for a, b in zip(self.stores, h.stores):
            assert np.array_equal(a.cpu().numpy(), b), note

    def extend(self, seqs, more, want=0):
        got = self.K.kpool_pages_extend(self.gpu, self.i32(seqs), self.i32(more), workspace=self.ws)
        st, begin = self.host.extend(seqs, more)
        assert st == want
        assert got.cpu().tolist() == begin
        self.check(want, ("extend", seqs, more))
        return begin

    def write(self, seqs, begin, cu, k=0, want=0):
        st = self.host.stores[k]
        rows = self.rng.randint(0, 256, (st.shape[0], cu[-1], st.shape[3])).astype(np.uint8)
        self.K.kpool_pages_write(self.gpu, self.i32(seqs), self.i32(begin), self.i32(cu),
                                 torch.from_numpy(rows).cuda(), self.stores[k], workspace=self.ws)
        assert self.host.write(seqs, begin, cu, rows, k) == want
        self.check(want, ("write", seqs, begin, cu, k))

    def grow(self, seqs, more):
        begin = self.extend(seqs, more)
        self.write(seqs, begin, np.concatenate([[0], np.cumsum(more)]).tolist())

    def fork(self, parents, children, want=0):
        self.K.kpool_pages_fork(self.gpu, self.i32(parents), self.i32(children), self.stores, workspace=self.ws)
        assert self.host.fork(parents, children) == want
        self.check(want, ("fork", parents, children))

    def free(self, seqs, want=0):
        self.K.kpool_pages_free(self.gpu, self.i32(seqs), workspace=self.ws)
        assert self.host.release(seqs) == want
        self.check(want, ("free", seqs))

    def compact(self, want=0):
        self.K.kpool_pages_compact(self.gpu, self.stores, workspace=self.ws)
        assert self.host.compact() == want
        self.check(want, "compact")

    def copy(self, src, dst, want=0):
        self.K.kpool_pages_copy(self.i32(src), self.i32(dst), self.stores, workspace=self.ws)
        assert self.host.copy(src, dst) == want
        self.check(want, ("copy", src, dst))


@pytest.mark.parametrize("page_size", [1, 4, 5, 16, 64])
@pytest.mark.parametrize("inner_layers", [False, True])
def test_a_rollout(K, page_size, inner_layers):
    """Prompts filled, forked, grown, retired and packed, checked after every call."""
    b = Both(K, n_seqs=9, n_pages=60, max_pages=8, page_size=page_size, seed=page_size, inner_layers=inner_layers)
    ps = page_size
    b.grow([0, 5], [3 * ps + (1 if ps > 1 else 0), 2 * ps])       # one ends inside a page, one at its end
    b.fork([0, 0, 5, 0], [1, 2, 6, 4])
    b.grow([4, 1, 0, 6], [1, ps, 2 * ps - 1, 0])
    b.free([2, 0])
    b.compact()
    b.grow([1, 4], [1, 3])
    b.fork([1], [0])
    b.free([0, 1, 4, 5, 6])
    b.compact()
    assert b.gpu.free_count.item() == 60


@pytest.mark.parametrize("seed", range(6))
def test_random_calls(K, seed):
    """Calls drawn at random, refused ones among them."""
    rng = np.random.RandomState(100 + seed)
    ps = int(rng.choice([3, 8, 16]))
    b = Both(K, n_seqs=12, n_pages=50, max_pages=9, page_size=ps, layers=1 + seed % 3, seed=seed)
    statuses = set()
    for _ in range(60):
        h = b.host
        op = rng.randint(6)
        live, empty = np.flatnonzero(h.lens > 0).tolist(), np.flatnonzero(h.lens == 0).tolist()
        if op <= 1:
            seqs = rng.permutation(12)[:rng.randint(1, 6)].tolist()
            more = rng.randint(0, 3 * ps, len(seqs)).tolist()
            import copy
            st, _ = copy.deepcopy(h).extend(seqs, more)
            statuses.add(st)
            if st == 0:
                b.grow(seqs, more)
            else:
                b.extend(seqs, more, st)
        elif op == 2 and live and empty:
            n = rng.randint(1, len(empty) + 1)
            parents = rng.choice(live, n).tolist()
            children = rng.permutation(empty)[:n].tolist()
            if rng.rand() < 0.2:
                children[-1] = live[0]
            import copy
            st = copy.deepcopy(h).fork(parents, children)
            statuses.add(st)
            b.fork(parents, children, st)
        elif op == 3 and live:
            b.free(rng.permutation(12)[:rng.randint(1, 5)].tolist())
        elif op == 4:
            b.compact()
        elif op == 5:
            at = rng.permutation(50)[:2 * rng.randint(1, 12)].tolist()
            b.copy(at[::2], at[1::2])
    assert 0 in statuses


def test_lists_that_are_refused(K):
    b = Both(K, n_seqs=5, n_pages=6, max_pages=4, page_size=8)
    b.grow([0, 1], [13, 8])                       # three pages taken, three free
    for parents, children in (([0], [5]), ([0], [-1]), ([7], [2]), ([-2], [2]), ([0, 0], [2, 2]), ([0], [1]),
                              ([2], [2]), ([0, 1, 9], [2, 3, 4])):
        b.fork(parents, children, BAD)
    for seqs, more in (([0, 0], [1, 1]), ([5], [1]), ([-1], [0]), ([0], [-1]), ([0], [20]), ([2], [33])):
        b.extend(seqs, more, BAD)
    b.extend([2, 3], [17, 8], SHORT)              # four pages needed
    b.extend([2], [2 ** 31 - 1], BAD)
    for seqs in ([0, 0], [5], [-1], [1, 2, 1]):
        b.free(seqs, BAD)
    for src, dst in (([0], [6]), ([6], [0]), ([0], [-1]), ([-1], [0]), ([0, 1], [2, 2]), ([0, 1], [1, 2]), ([3], [3])):
        b.copy(src, dst, BAD)
    b.copy([0, 0, 1], [3, 4, 5])                  # a source twice
    b.grow([2], [24])
    b.fork([0], [3], SHORT)                       # its partial page has nowhere to go
    b.fork([1, 2], [3, 4])                        # whole pages need none


@pytest.mark.parametrize("n", [1, 255, 257, 1023, 1024, 1025, 3000])
def test_long_copies(K, n):
    """Around the length up to which every block checks the list itself; a doubled destination, a page on both sides
    and an id out of range at its far end."""
    rng = np.random.RandomState(n)
    b = Both(K, n_seqs=1, n_pages=2 * n + 5, max_pages=1, page_size=4, layers=2, seed=n)
    b.ws = torch.empty(K.kpool_pages_workspace_size(n, 1, 2 * n + 5), dtype=torch.uint8, device="cuda")
    at = rng.permutation(2 * n + 5)
    dst = at[:n].tolist()
    src = rng.choice(at[n:], n).tolist()
    b.copy(src, dst)
    if n > 1:
        b.copy(src, dst[:-1] + [dst[0]], BAD)
        b.copy(src[:-1] + [dst[0]], dst, BAD)
        b.copy([dst[-1]] + src[1:], dst, BAD)
    b.copy(src[:-1] + [2 * n + 5], dst, BAD)
    b.copy(src, dst[:-1] + [-1], BAD)
    b.copy(src[:-1] + [-2 ** 31], dst, BAD)


def test_copies_without_a_workspace(K):
    """On two streams at once, and captured: nothing but the status word is shared."""
    b = Both(K, n_seqs=1, n_pages=40, max_pages=1, page_size=8)
    lists = [([0, 1, 2], [10, 11, 12]), ([3, 4], [20, 21])]
    torch.cuda.synchronize()
    for src, dst in lists:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            K.kpool_pages_copy(b.i32(src), b.i32(dst), b.stores)
        b.host.copy(src, dst)
    torch.cuda.synchronize()
    for a, h in zip(b.stores, b.host.stores):
        assert np.array_equal(a.cpu().numpy(), h)
    src, dst = b.i32([5, 6]), b.i32([30, 31])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kpool_pages_copy(src, dst, b.stores)
    dst.copy_(b.i32([32, 33]))
    g.replay()
    torch.cuda.synchronize()
    b.host.copy([5, 6], [32, 33])
    for a, h in zip(b.stores, b.host.stores):
        assert np.array_equal(a.cpu().numpy(), h)


def test_writes_that_are_left_out(K):
    b = Both(K, n_seqs=4, n_pages=12, max_pages=4, page_size=8)
    b.grow([0], [12])
    b.fork([0], [1])
    b.write([0], [0], [0, 3], want=BAD)           # a shared page
    b.write([0, 1], [8, 8], [0, 4, 8])            # each sequence's own
    b.write([1], [10], [0, 5], want=BAD)          # the last three lie behind the length
    b.write([1, 4], [11, 0], [0, 1, 2], want=BAD)
    b.write([1, -1, 0], [11, 0, 9], [0, 1, 1, 2])  # no row goes to the unknown sequence
    b.write([1], [-1], [0, 2], want=BAD)          # what a refused extension returned
    b.write([2], [0], [0, 1], want=BAD)           # an empty sequence
    b.write([0, 1], [2, 2], [0, 1, 2], k=1)       # pooled rows: two per page
    b.write([1], [2 ** 31 - 1], [0, 1], want=BAD)


@pytest.mark.parametrize("rows", [1, 63, 255, 256, 257, 1030])
def test_a_status_is_of_its_own_call(K, rows):
    """Rows of one cluster and of more, with one row too many and without."""
    b = Both(K, n_seqs=2, n_pages=140, max_pages=130, page_size=8)
    b.grow([1], [rows])
    b.write([1], [0], [0, rows + 1], want=BAD)
    b.write([1], [0], [0, rows])
    b.write([0, 1], [0, 0], [0, 1, rows], want=BAD)
    b.write([0, 1], [0, 0], [0, 0, rows])


def test_nothing_listed(K):
    b = Both(K, n_seqs=3, n_pages=4, max_pages=2, page_size=8)
    b.extend([], [])
    b.fork([], [])
    b.free([])
    b.copy([], [])
    b.compact()
    b.extend([0, 1, 2], [0, 0, 0])
    b.fork([0], [1])                              # an empty parent
    b.free([0, 1, 2])                             # sequences that hold nothing


def test_a_shared_partial_page_is_not_extended(K):
    """A table made by hand, whose last partial page two sequences hold."""
    b = Both(K, n_seqs=3, n_pages=6, max_pages=3, page_size=8)
    b.grow([0], [5])
    b.gpu.page_table[1, 0] = b.host.table[1, 0] = b.host.table[0, 0]
    b.gpu.seq_lens[1] = 5
    b.host.lens[1] = 5
    b.gpu.ref_count[int(b.host.table[0, 0])] = 2
    b.host.refs[b.host.table[0, 0]] = 2
    b.extend([1], [1], BAD)
    b.extend([1], [0])
    b.free([1])
    b.grow([0], [1])


@pytest.mark.parametrize("what", ["id_high", "id_negative", "count_high", "count_negative", "list", "length"])
def test_a_broken_pool_is_not_followed(K, what):
    """Ids, counts and lengths outside their arrays set the status; no call goes where they point."""
    b = Both(K, n_seqs=4, n_pages=8, max_pages=3, page_size=8)
    b.grow([0, 1], [20, 3])
    p, i = b.gpu, b.i32
    calls = [lambda: K.kpool_pages_fork(p, i([0]), i([2]), b.stores, workspace=b.ws),
             lambda: K.kpool_pages_extend(p, i([0, 1]), i([3, 9]), workspace=b.ws),
             lambda: K.kpool_pages_free(p, i([0]), workspace=b.ws)]
    if what.startswith("id"):
        p.page_table[0, 2] = 1 << 20 if what == "id_high" else -7
    elif what.startswith("count"):
        p.free_count.fill_(9 if what == "count_high" else -1)
    elif what == "list":
        p.free_list.fill_(99)
        calls = calls[:2]
    else:
        p.seq_lens[0] = 25
    before = [s.clone() for s in b.stores]
    for call in calls:
        call()
        assert K.kpool_read_status(b.ws) & BAD
    if what != "length":
        K.kpool_pages_compact(p, b.stores, workspace=b.ws)
        torch.cuda.synchronize()
    assert all(s.shape == t.shape for s, t in zip(before, b.stores))


@pytest.mark.parametrize("n_seqs,n_pages,page_size", [(1500, 9000, 1), (1100, 40000, 4)])
def test_many_sequences_and_pages(K, n_seqs, n_pages, page_size):
    """More items than a plan block has threads, more pages than one round of its scan."""
    rng = np.random.RandomState(n_seqs)
    b = Both(K, n_seqs=n_seqs, n_pages=n_pages, max_pages=300, page_size=page_size, layers=1, seed=3)
    b.ws = torch.empty(K.kpool_pages_workspace_size(n_seqs, n_seqs, n_pages), dtype=torch.uint8, device="cuda")
    half = n_seqs // 2
    seqs = rng.permutation(half).tolist()
    b.grow(seqs, rng.randint(0, 5 * page_size, half).tolist())
    b.extend([0], [257 * page_size])               # a table row longer than a block
    b.fork(rng.randint(0, half, n_seqs - half).tolist(), (half + rng.permutation(n_seqs - half)).tolist())
    b.free(rng.permutation(n_seqs)[:n_seqs - 40].tolist())
    b.compact()


def test_pages_larger_than_a_piece(K):
    """Pages of more than one 16 KB piece, with an odd rest, in three layers."""
    ps, width = 33, 624                            # 20592 bytes a page
    b = Both(K, n_seqs=4, n_pages=9, max_pages=3, page_size=ps, layers=3)
    g = np.random.RandomState(4)
    h = g.randint(0, 256, (3, 9, ps, width)).astype(np.uint8)
    b.stores, b.host.stores = [torch.from_numpy(h).cuda()], [h.copy()]
    b.grow([0], [ps + 30])
    b.fork([0, 0], [1, 2])
    b.copy([0, 1], [7, 8])
    b.free([0])
    b.compact()


def test_a_store_of_more_than_4_gb(K):
    """Pages and layers whose byte offsets pass 32 bits."""
    n, ps, width = 3000, 32, 49152                 # 1.5 MB a page, 4.7 GB a layer
    store = torch.zeros(2, n, ps, width, dtype=torch.uint8, device="cuda")
    pages = K.kpool_pages_new(4, n, 4, ps)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pages.free_list.copy_(pages.free_list.flip(0))  # the last page is taken first
    g = torch.Generator("cuda")
    g.manual_seed(1)
    rows = torch.randint(0, 256, (2, 40, width), dtype=torch.uint8, device="cuda", generator=g)
    begin = K.kpool_pages_extend(pages, i([2]), i([40]))
    K.kpool_pages_write(pages, i([2]), begin, i([0, 40]), rows, store)
    K.kpool_pages_fork(pages, i([2]), i([0]), store)
    assert pages.page_table[2, :2].tolist() == [n - 1, n - 2]
    assert pages.page_table[0, :2].tolist() == [n - 1, n - 3]
    K.kpool_pages_copy(i([n - 1]), i([1500]), store)
    assert K.kpool_read_status(pages.workspace) == 0
    assert torch.equal(store[:, n - 1], rows[:, :32]) and torch.equal(store[:, 1500], rows[:, :32])
    assert torch.equal(store[:, n - 2, :8], rows[:, 32:]) and torch.equal(store[:, n - 3, :8], rows[:, 32:])
    K.kpool_pages_free(pages, i([2]))
    K.kpool_pages_compact(pages, store)
    assert K.kpool_read_status(pages.workspace) == 0
    # the two pages still held, n - 3 and n - 1, move to 0 and 1 in their order
    assert pages.page_table[0, :2].tolist() == [1, 0] and pages.free_count.item() == n - 2
    assert torch.equal(store[:, 1], rows[:, :32]) and torch.equal(store[:, 0, :8], rows[:, 32:])


def test_rows_wider_than_a_warp_loads_at_once(K):
    """Rows of 2 KB and a little, and of 5 KB."""
    for width in (2064, 5120):
        b = Both(K, n_seqs=3, n_pages=6, max_pages=2, page_size=4, layers=2)
        h = np.random.RandomState(width).randint(0, 256, (2, 6, 4, width)).astype(np.uint8)
        b.stores, b.host.stores = [torch.from_numpy(h).cuda()], [h.copy()]
        b.grow([1, 0], [5, 3])


def test_captured_and_replayed(K):
    """A decode step's upkeep captured once and replayed: each replay goes on from the pool as it is."""
    b = Both(K, n_seqs=4, n_pages=30, max_pages=8, page_size=8, layers=1)
    b.grow([0, 1], [10, 16])
    seqs, more, cu = b.i32([1, 0]), b.i32([1, 1]), b.i32([0, 1, 2])
    rows = torch.from_numpy(b.rng.randint(0, 256, (1, 2, 48)).astype(np.uint8)).cuda()
    child, parent = b.i32([2]), b.i32([0])

    def step():
        begin = K.kpool_pages_extend(b.gpu, seqs, more, workspace=b.ws)
        K.kpool_pages_write(b.gpu, seqs, begin, cu, rows, b.stores[0], workspace=b.ws)
        K.kpool_pages_fork(b.gpu, parent, child, b.stores, workspace=b.ws)
        K.kpool_pages_free(b.gpu, child, workspace=b.ws)
        K.kpool_pages_compact(b.gpu, b.stores, workspace=b.ws)

    def host_step():
        _, begin = b.host.extend([1, 0], [1, 1])
        b.host.write([1, 0], begin, [0, 1, 2], rows.cpu().numpy(), 0)
        b.host.fork([0], [2])
        b.host.release([2])
        b.host.compact()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                  # another stream than the default one
        step()
    torch.cuda.current_stream().wait_stream(side)
    host_step()
    b.check(0, "eager on a side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(5):
        graph.replay()
        host_step()
        b.check(0, ("replay", k))


ARRAYS = ("page_table", "seq_lens", "ref_count", "free_list", "free_count")


def _state(b):
    """Copies of the pool's five arrays and of the stores."""
    return [getattr(b.gpu, a).clone() for a in ARRAYS] + [s.clone() for s in b.stores]


def _broken(K, what):
    """Sequences of 20 and 3 tokens in pages of 8, of at most 3 each, then one number out of its range."""
    b = Both(K, n_seqs=4, n_pages=8, max_pages=3, page_size=8)
    b.grow([0, 1], [20, 3])
    p = b.gpu
    if what == "id":
        p.page_table[0, 2] = 1 << 20
    elif what == "negative id":
        p.page_table[0, 2] = -7
    elif what == "count":
        p.free_count.fill_(9)
    elif what == "negative count":
        p.free_count.fill_(-1)
    elif what == "list":
        p.free_list.fill_(99)
    elif what == "length":
        p.seq_lens[0] = 25
    else:
        p.seq_lens[0] = -1
    return b


BROKEN = ["id", "negative id", "count", "negative count", "list", "length", "negative length"]


@pytest.mark.parametrize("what", BROKEN)
def test_a_refused_call_changes_nothing(K, what):
    """Every array of the pool and every byte of the stores, whatever is wrong with the pool."""
    b = _broken(K, what)
    p, i = b.gpu, b.i32
    begin = i([7, 7])
    calls = [lambda: K.kpool_pages_fork(p, i([0]), i([2]), b.stores, workspace=b.ws),
             lambda: K.kpool_pages_extend(p, i([0, 1]), i([3, 9]), workspace=b.ws, out=begin)]
    if "id" not in what and what != "list":
        calls.append(lambda: K.kpool_pages_free(p, i([0]), workspace=b.ws))
        calls.append(lambda: K.kpool_pages_free(p, i([1, 0]), workspace=b.ws))
    before = _state(b)
    for k, call in enumerate(calls):
        call()
        assert K.kpool_read_status(b.ws) == BAD, k
        assert all(torch.equal(x, y) for x, y in zip(before, _state(b))), k
    assert begin.tolist() == [-1, -1]


@pytest.mark.parametrize("what", ["id", "negative id"])
def test_a_freed_id_out_of_range_is_skipped(K, what):
    """The other pages of the sequence are given back, and nothing else changes."""
    b = _broken(K, what)
    before = _state(b)
    one, two = before[0][0, :2].tolist()
    K.kpool_pages_free(b.gpu, b.i32([0]), workspace=b.ws)
    assert K.kpool_read_status(b.ws) == BAD
    want = [t.clone() for t in before]
    want[0][0] = -1
    want[1][0] = 0
    want[2][one] = want[2][two] = 0
    n = int(before[4])
    want[3][n:n + 2] = b.i32(sorted([one, two]))
    want[4] += 2
    assert all(torch.equal(x, y) for x, y in zip(want, _state(b)))


@pytest.mark.parametrize("what", ["count", "negative count", "length", "negative length"])
def test_a_refused_packing_changes_nothing(K, what):
    b = _broken(K, what)
    if "count" in what:
        b.gpu.ref_count[b.gpu.page_table[0, 0].long()] = 0     # (a hole, so that there is something to move)
    before = _state(b)
    K.kpool_pages_compact(b.gpu, b.stores, workspace=b.ws)
    assert K.kpool_read_status(b.ws) == BAD
    assert all(torch.equal(x, y) for x, y in zip(before, _state(b)))


@pytest.mark.parametrize("what", ["id", "negative id", "list"])
def test_packing_with_an_id_out_of_range(K, what):
    """A bad table entry is skipped, with the status; the free list is made anew, so that what it held does not matter."""
    b = _broken(K, what)
    before = _state(b)
    b.host.compact()
    K.kpool_pages_compact(b.gpu, b.stores, workspace=b.ws)
    if what == "list":
        b.check(0)
    else:
        b.host.table[0, 2] = before[0][0, 2].item()
        b.check(BAD)


def test_lengths_that_fill_the_table(K):
    """The largest length that a table row has room for, and none, are packed like others."""
    b = Both(K, n_seqs=3, n_pages=9, max_pages=3, page_size=8)
    b.grow([0, 1], [24, 24])
    b.free([0])
    b.compact()


def test_the_status_of_lists_longer_than_the_pool(K):
    """More sequences than pages, lists with repetitions: the pool's own workspace tells of the last call, whatever its
    length."""
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    n = 300
    p = K.kpool_pages_new(n, 4, 2, 8)
    store = torch.zeros(4, 8, 16, dtype=torch.uint8, device="cuda")
    every = i(list(range(n)))

    def status(want):
        assert K.kpool_read_status(p.workspace) == want

    K.kpool_pages_extend(p, i([0, 1]), i([3, 8]))
    status(0)
    assert K.kpool_pages_extend(p, every, torch.ones_like(every)).eq(-1).all()
    status(SHORT)                                  # 299 pages needed, 2 free
    K.kpool_pages_fork(p, i([1] * 298), i(list(range(2, n))), store)
    status(0)
    K.kpool_pages_fork(p, i([0] * n), every, store)
    status(BAD)
    K.kpool_pages_extend(p, i([0]), i([0]))
    status(0)
    K.kpool_pages_free(p, i([0, 0] * n))           # longer than any list that could be carried out
    status(BAD)
    K.kpool_pages_write(p, i([0] * 3 * n), i([k % 3 for k in range(3 * n)]), i([min(k, 3) for k in range(3 * n + 1)]),
                        torch.ones(3, 16, dtype=torch.uint8, device="cuda"), store)
    status(0)
    assert store[p.page_table[0, 0], :3].eq(1).all() and int(store.sum()) == 3 * 16
    K.kpool_pages_extend(p, i([0] * 3 * n), i([0] * 3 * n))
    status(BAD)
    K.kpool_pages_free(p, every)
    status(0)
    assert p.free_count.item() == 4


def test_a_pool_dropped_while_another_stream_uses_it(K):
    """The pool's own workspace goes to nobody else before the side stream's calls have ended."""
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    p = K.kpool_pages_new(6, 40, 8, 8)
    kept = [getattr(p, a) for a in ARRAYS]
    seqs, more = i([1, 4, 2]), i([20, 3, 64])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)              # some 20 ms
        begin = K.kpool_pages_extend(p, seqs, more)
        K.kpool_pages_free(p, seqs[:1])
    size, at = p.workspace.numel(), p.workspace.data_ptr()
    del p
    others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(20)]
    assert all(o.data_ptr() != at for o in others)
    torch.cuda.synchronize()
    assert begin.tolist() == [0, 0, 0] and kept[1].tolist() == [0, 0, 64, 0, 3, 0]
    assert kept[4].item() == 40 - 9


def test_a_pool_used_at_once_on_another_stream(K):
    """The first call there waits until the workspace is made; so does one in a graph, which is captured then."""
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    made = K.kpool_pages_new(6, 40, 8, 8)
    arrays = [getattr(made, a) for a in ARRAYS]
    seqs, more = i([1, 4, 2]), i([20, 3, 64])
    torch.cuda.synchronize()
    side, passed = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda._sleep(40_000_000)
    p = K.KPoolPages(*arrays, 8)
    passed.record()
    with torch.cuda.stream(side):
        K.kpool_pages_extend(p, seqs, more)
    side.synchronize()
    assert passed.query()
    assert K.kpool_read_status(p.workspace) == 0
    assert p.seq_lens.tolist() == [0, 20, 64, 0, 3, 0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        K.kpool_pages_free(p, seqs)
        K.kpool_pages_extend(p, seqs, more)
    for _ in range(3):
        graph.replay()
    assert K.kpool_read_status(p.workspace) == 0
    assert p.seq_lens.tolist() == [0, 20, 64, 0, 3, 0] and p.free_count.item() == 40 - 12


@pytest.mark.parametrize("there", [0, 1, 8, 127, 128, 129, 300])
def test_fewer_rows_than_the_offsets_count(K, there):
    """The rows that there are go to their places, and the status tells of the others."""
    b = Both(K, n_seqs=3, n_pages=60, max_pages=50, page_size=8)
    b.grow([0, 2], [there + 20, 5])
    rows = b.rng.randint(0, 256, (2, there, 48)).astype(np.uint8)
    gpu = torch.from_numpy(rows).cuda()
    for cu, want in (([0, 2, there + 3], BAD), ([0, there, there + 1], BAD), ([0, 0, there], 0)):
        K.kpool_pages_write(b.gpu, b.i32([2, 0]), b.i32([0, 0]), b.i32(cu), gpu, b.stores[0], workspace=b.ws)
        if cu[1] > 5:
            want = BAD                             # (sequence 2 has room for five)
        b.host.write([2, 0], [0, 0], [min(c, there) for c in cu], rows, 0)
        b.check(want, (there, cu))


def test_growing_by_the_lengths_themselves(K):
    """n_new is seq_lens: each sequence grows by what another one holds."""
    n = 200
    b = Both(K, n_seqs=n, n_pages=1400, max_pages=12, page_size=8, layers=1)
    b.ws = torch.empty(K.kpool_pages_workspace_size(n, n, 1400), dtype=torch.uint8, device="cuda")
    seqs = b.rng.permutation(n).tolist()
    b.extend(list(range(n)), b.rng.randint(0, 25, n).tolist())
    for _ in range(2):
        more = b.host.lens.tolist()
        begin = K.kpool_pages_extend(b.gpu, b.i32(seqs), b.gpu.seq_lens, workspace=b.ws)
        assert b.host.extend(seqs, more) == (0, begin.tolist())
        b.check(0)


def test_a_pool_made_in_inference_mode(K):
    """Used in it and behind it, with a list longer than the pool among the calls."""
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    with torch.inference_mode():
        p = K.kpool_pages_new(3, 6, 4, 8)
        K.kpool_pages_extend(p, i([0]), i([9]))
    store = torch.zeros(6, 8, 16, dtype=torch.uint8, device="cuda")
    K.kpool_pages_fork(p, i([0]), i([1]), store)
    assert K.kpool_read_status(p.workspace) == 0
    K.kpool_pages_free(p, i([0] * 7))
    assert K.kpool_read_status(p.workspace) == BAD
    with torch.inference_mode():
        K.kpool_pages_free(p, i([1, 0] * 4))
        assert K.kpool_read_status(p.workspace) == BAD
        K.kpool_pages_free(p, i([1, 0]))
    assert K.kpool_read_status(p.workspace) == 0 and p.free_count.item() == 6


@pytest.mark.parametrize("rows", [1, 32, 33, 65, 97, 129, 161, 193, 225, 256])
def test_writes_of_one_to_eight_blocks(K, rows):
    """A single layer, 32 rows to a block of the cluster."""
    b = Both(K, n_seqs=4, n_pages=80, max_pages=40, page_size=8, layers=1)
    b.extend([3, 1], [rows, 3])
    b.write([3, 1], [0, 1], [0, rows // 2, rows // 2 + 2] if rows > 3 else [0, rows, rows])
    b.write([3, 1], [0, 3], [0, rows - 1, rows], want=BAD)
    b.write([3], [0], [0, rows])

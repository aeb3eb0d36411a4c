"""Refusals of the paged-cache and shared-prefix calls, all on the host: no
argument here reaches a device."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def b():
    from sparse_attention_kpool_compress_gb300 import build as B
    B.build()
    from sparse_attention_kpool_compress_gb300 import binding
    return binding


def _fake(n=1 << 20):
    buf = ctypes.create_string_buffer(n + 512)
    return buf, (ctypes.addressof(buf) + 255) & ~255


def _pool(b, a, **kw):
    f = dict(page_table=a, seq_lens=a, ref_count=a, free_list=a, free_count=a, n_seqs=4, max_pages=8, n_pages=32,
             page_size=16)
    f.update(kw)
    return ctypes.byref(b._Pool(**f))


def _store(b, a, **kw):
    f = dict(data=a, layer_stride=32 * 16 * 1024, page_stride=16 * 1024, n_layers=2, rows_per_page=16,
             row_bytes=1024)
    f.update(kw)
    order = ("data", "layer_stride", "page_stride", "n_layers", "rows_per_page", "row_bytes")
    return b._pack_store(*(f[k] or 0 for k in order), 0)


def test_pools_and_stores_are_checked(b):
    L = b._lib
    keep, a = _fake()
    p, mis = P(a), P(a + 2)
    ws = L.kpool_pages_workspace_size(4, 4, 32)
    good = _store(b, a)

    def fork(pool=None, par=p, ch=p, n=4, st=good, n_st=1, w=p, wb=ws):
        return L.kpool_pages_fork(_pool(b, a) if pool is None else pool, par, ch, n, st, n_st, w, wb, None)

    bad = [
        (fork(pool=P(None)), -1),
        *[(fork(pool=_pool(b, a, **{k: 0})), -1) for k in ("n_seqs", "max_pages", "n_pages", "page_size")],
        *[(fork(pool=_pool(b, a, **{k: None})), -1) for k in ("page_table", "seq_lens", "ref_count", "free_list",
                                                             "free_count")],
        (fork(pool=_pool(b, a, seq_lens=a + 2)), -1),
        (fork(pool=_pool(b, a, max_pages=1 << 20, page_size=1 << 12)), -1),
        (fork(par=P(None)), -1), (fork(ch=mis), -1), (fork(n=-1), -1), (fork(n_st=9), -1), (fork(st=P(None)), -1),
        (fork(w=P(None)), -4), (fork(w=mis), -4), (fork(wb=ws - 1), -4),
        *[(fork(st=_store(b, a, **kw)), -1) for kw in (
            dict(data=None), dict(data=a + 8), dict(n_layers=0), dict(rows_per_page=0), dict(rows_per_page=5),
            dict(rows_per_page=32), dict(row_bytes=1000), dict(row_bytes=0), dict(page_stride=16 * 1024 + 8),
            dict(layer_stride=8), dict(page_stride=1024), dict(layer_stride=1024),
            dict(page_stride=-16 * 1024), dict(n_layers=5000))],
        (L.kpool_pages_extend(_pool(b, a), p, p, 4, P(None), p, ws, None), -1),
        (L.kpool_pages_extend(_pool(b, a), p, p, 4, P(a + 64), p, 16, None), -4),
        (L.kpool_pages_extend(_pool(b, a), p, P(a + 64), 4, P(a + 12), p, ws, None), -1),
        (L.kpool_pages_extend(_pool(b, a), P(a + 64), p, 4, p, p, ws, None), -1),
        (L.kpool_pages_free(_pool(b, a), P(None), 4, p, ws, None), -1),
        (L.kpool_pages_free(_pool(b, a), p, 1 << 30, p, ws, None), -1),
        (L.kpool_pages_compact(_pool(b, a), good, -1, p, ws, None), -1),
        (L.kpool_pages_copy(p, p, 4, 0, good, 1, p, ws, None), -1),
        (L.kpool_pages_copy(p, P(None), 4, 32, good, 1, p, ws, None), -1),
        (L.kpool_pages_write(_pool(b, a), p, p, p, 4, 8, P(None), 8192, good, p, ws, None), -1),
        (L.kpool_pages_write(_pool(b, a), p, p, p, 4, 8, mis, 8192, good, p, ws, None), -1),
        (L.kpool_pages_write(_pool(b, a), p, p, p, 4, 8, p, 4096, good, p, ws, None), -1),
        (L.kpool_pages_write(_pool(b, a), p, p, p, 4, -1, p, 8192, good, p, ws, None), -1),
        (L.kpool_pages_write(_pool(b, a), p, p, p, 0, 8, p, 8192, good, p, ws, None), -1),
    ]
    for k, (rc, code) in enumerate(bad):
        assert rc == code, (k, rc, L.kpool_last_error())
    assert L.kpool_last_error()
    assert L.kpool_pages_workspace_size(-1, 4, 32) == 0 and L.kpool_pages_workspace_size(4, 4, 0) == 0
    del keep


def test_shared_prefix_arguments_are_checked(b):
    L = b._lib
    keep, a = _fake()
    p, mis = P(a), P(a + 2)
    names = ("q", "kv", "stride", "n_pages", "page_size", "table", "lens", "n_rows", "max_pages", "seq_ids", "cu_q",
             "B", "cu_g", "prefix", "G", "Tq", "H", "Dc", "scale", "o", "lse", "ws", "ws_bytes", "stream")
    need = L.kpool_shared_prefix_mla_workspace_size(8, 64, 4, 2)
    assert need >= 256
    base = dict(zip(names, (p, p, 64 * 512, 32, 64, p, p, 4, 8, None, p, 4, p, p, 2, 8, 64, 512, 0.1, p, p, p, need,
                            None)))
    for change, code in (
            (dict(H=0), -2), (dict(H=129), -2), (dict(Dc=576), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
            (dict(page_size=256), -2), (dict(Tq=-1), -1), (dict(Tq=1 << 30), -1), (dict(B=0), -1), (dict(G=0), -1),
            (dict(n_rows=0), -1), (dict(n_rows=3), -1), (dict(max_pages=0), -1), (dict(max_pages=1 << 26), -1),
            (dict(n_pages=0), -1), (dict(stride=64 * 512 - 8), -1), (dict(stride=64 * 512 + 4), -1),
            (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
            (dict(q=None), -1), (dict(kv=None), -1), (dict(table=None), -1), (dict(lens=None), -1),
            (dict(cu_q=None), -1), (dict(cu_g=None), -1), (dict(prefix=None), -1), (dict(o=None), -1),
            (dict(lse=None), -1), (dict(q=mis), -1), (dict(kv=mis), -1), (dict(o=mis), -1), (dict(lse=mis), -1),
            (dict(table=mis), -1), (dict(seq_ids=mis), -1), (dict(ws=None), -4), (dict(ws=mis), -4),
            (dict(ws_bytes=need - 1), -4)):
        args = {**base, **change}
        rc = L.kpool_shared_prefix_mla_fwd(*(args[n] for n in names))
        assert rc == code, (change, rc, L.kpool_last_error())
    for bad in ((-1, 64, 4, 2), (8, 0, 4, 2), (8, 129, 4, 2), (1 << 31, 64, 4, 2), (8, 64, -1, 2)):
        assert L.kpool_shared_prefix_mla_workspace_size(*bad) == 0
    del keep


def test_tensors_are_checked(b):
    """The binding's own checks: types, shapes, strides and where a tensor lives."""
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        b.KPoolPages(i32.view(2, 2), i32, i32, i32, i32, 16)
    with pytest.raises(TypeError):
        b.KPoolPages(i32.view(2, 2).long(), i32, i32, i32, i32, 16)
    with pytest.raises(ValueError, match="contiguous"):
        b.KPoolPages(torch.zeros(4, 4, dtype=torch.int32).t()[:2], i32, i32, i32, i32, 16)
    with pytest.raises(ValueError):
        b.kpool_pages_copy(i32, i32, ())
    with pytest.raises(ValueError, match="CUDA"):
        b.kpool_pages_copy(i32, i32, [torch.zeros(2, 8, 16, 8)])


def test_the_binding_imports_without_cuda_in_torch(b, monkeypatch):
    """A CPU build of torch lacks the stream lookup: the calls that work on the host alone still do."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("binding_without_cuda", b.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    cu, total = module.kpool_num_pools([0, 5, 13], 13, 4)
    assert cu.tolist() == [0, 1, 3] and total == 3
    assert module.kpool_pages_workspace_size(4, 4, 32) == b.kpool_pages_workspace_size(4, 4, 32) > 0


@pytest.mark.parametrize("array, size", [("page_table", 32), ("seq_lens", 4), ("ref_count", 32), ("free_list", 32),
                                         ("free_count", 1)])
def test_an_output_in_the_pool_is_refused(b, array, size):
    """begin_out on the last entry of each of the pool's arrays, and across the first."""
    L = b._lib
    keep, a = _fake()
    at = {name: a + 4096 * (k + 1) for k, name in enumerate(("page_table", "seq_lens", "ref_count", "free_list",
                                                             "free_count"))}
    ws, lists = a + 65536, P(a + 32768)
    for out in (at[array] + 4 * (size - 1), at[array] - 4):
        rc = L.kpool_pages_extend(_pool(b, a, **at), lists, lists, 2, P(out), P(ws), 1 << 16, None)
        assert rc == -1 and b"overlaps the pool" in L.kpool_last_error()
    del keep


def test_a_status_is_read_on_the_device_of_its_workspace(b, monkeypatch):
    """The read waits for the current device: that has to be the workspace's, as in the calls themselves."""
    current, read = [0], []

    class Device:
        def __init__(self, device):
            self.index = device

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Lib:
        def kpool_read_status(self, workspace, out):
            read.append((current[0], workspace.value))
            return 0

    class Workspace:
        def get_device(self):
            return 3

        def data_ptr(self):
            return 4096

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(b, "_lib", Lib())
    assert b.kpool_read_status(Workspace()) == 0
    assert read == [(3, 4096)] and current == [0]

"""A workspace that is sized for the largest batch serves every smaller one: the sizes
of the sparse attention's backward calls and of its paged form never shrink as an
argument grows."""
import pytest

ROWS = [*range(0, 170), 304, 8192, (1 << 31) - 1]


@pytest.fixture(scope="module")
def b():
    from sparse_attention_kpool_compress_gb300 import build as B
    B.build()
    from sparse_attention_kpool_compress_gb300 import binding
    return binding


def _grows(sizes):
    assert all(0 < x <= y for x, y in zip(sizes, sizes[1:])), sizes


@pytest.mark.parametrize("Tk", [0, 1, 8192, 1 << 20])
def test_backward_sizes_grow_with_the_rows(b, Tk):
    _grows([b.kpool_sparse_mla_bwd_workspace_size(T, Tk) for T in ROWS])


@pytest.mark.parametrize("T", [0, 1, 5, 80, 81, 8192])
def test_backward_sizes_grow_with_the_keys(b, T):
    _grows([b.kpool_sparse_mla_bwd_workspace_size(T, Tk) for Tk in (0, 1, 63, 64, 8192, 1 << 20, (1 << 31) - 1)])


@pytest.mark.parametrize("kpool,topk", [(1, 1), (1, 2048), (4, 64), (4, 2048), (8, 512), (64, 64), (64, 4096)])
def test_paged_sizes_grow_with_the_rows(b, kpool, topk):
    _grows([b.kpool_sparse_mla_paged_workspace_size(T, kpool, topk) for T in ROWS])


@pytest.mark.parametrize("T", [0, 1, 5, 80, 81, 8192])
@pytest.mark.parametrize("kpool", [1, 4, 64])
def test_paged_sizes_grow_with_the_budget(b, T, kpool):
    _grows([b.kpool_sparse_mla_paged_workspace_size(T, kpool, kpool * n) for n in (1, 2, 3, 17, 64, 512, 4096, 1 << 20)])

"""The largest sizes of the sparse attention's backward pass and of its paged form."""
import math

import numpy as np
import pytest
import torch

from mla_grad_checks import DC, E, H, U
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

"""What the checks of the sparse attention's gradients notice, on the CPU: the kernels' roundings pass
(p and ds to BF16, FP32 sums, outputs rounded once), a row that is lost from a sum of many or counted
twice does not, although nearly all values stay within the bounds of single values."""
import pytest
import torch

from mla_grad_checks import DC, H, Grads
from mla_norm_checks import GradNorms, check_outputs

SCALE = DC ** -0.5


@pytest.fixture(scope="module")
def case():
    """400 rows over 64 latent rows, each listed by more than 300 of them."""
    T, Tk = 400, 64
    g = torch.Generator().manual_seed(7)
    normal = lambda *s, size=1.0: (torch.randn(*s, generator=g) * size).to(torch.bfloat16)  # noqa: E731
    q, kv, d_o = normal(T, H, DC), normal(Tk, DC), normal(T, H, DC, size=0.1)
    lists = [torch.randint(0, Tk, (64 if t % 2 else 40,), generator=g) for t in range(T)]
    o, lse = torch.zeros_like(q), torch.zeros(T, H)
    dq, parts = torch.zeros_like(q), torch.zeros(T, Tk, DC)
    for t, j in enumerate(lists):
        keys, qt, do = kv[j].float(), q[t].float(), d_o[t].float()
        s = SCALE * (qt @ keys.T)
        lse[t] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[t][:, None])
        pr = p.bfloat16().float()
        o[t] = (pr @ keys).bfloat16()
        ds = (SCALE * p * (do @ keys.T - (do * o[t].float()).sum(1, keepdim=True))).bfloat16().float()
        dq[t] = (ds @ keys).bfloat16()
        parts[t].index_add_(0, j, ds.T @ qt + pr.T @ do)
    args = (q, kv, lists, o, lse, d_o, SCALE)
    return args, dq, parts, Grads(*args), GradNorms(*args)


def test_the_kernels_roundings_pass(case):
    args, dq, parts, bounds, norms = case
    dkv = parts.sum(0).bfloat16()
    bounds.check(dq, dkv)
    norms.check(dq, dkv)
    check_outputs(args[3], *args[:3], SCALE)


@pytest.mark.parametrize("times", [0, 2])
@pytest.mark.parametrize("row", [0, 201])
def test_a_lost_or_repeated_row_is_noticed(case, row, times):
    _, dq, parts, bounds, norms = case
    dkv = (parts.sum(0) + (times - 1) * parts[row]).bfloat16()
    # (single values' bounds hardly tell)
    inside = (dkv.double() - bounds.dkv).abs() <= bounds.dkv_tol
    assert inside.double().mean() > 0.999
    with pytest.raises(AssertionError):
        norms.check(dq, dkv)


def test_a_lost_token_of_few_is_noticed(case):
    """One latent row that lacks the sum of a tenth of its rows; a head's dq without its last 16 tokens."""
    args, dq, parts, _, norms = case
    dkv = parts.sum(0)
    dkv[5] -= parts[:40, 5].sum(0)
    with pytest.raises(AssertionError):
        norms.check(dq, dkv.bfloat16())
    q, kv, lists, o, lse, d_o, _ = args
    few = dq.clone()
    keys, qt, do = kv[lists[3]].float(), q[3, 9].float(), d_o[3, 9].float()
    ds = SCALE * torch.exp(SCALE * (keys @ qt) - lse[3, 9]) * (keys @ do - do @ o[3, 9].float())
    few[3, 9] = (ds[:-16] @ keys[:-16]).bfloat16()
    with pytest.raises(AssertionError):
        norms.check(few, parts.sum(0).bfloat16())

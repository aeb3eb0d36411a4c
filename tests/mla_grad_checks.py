"""The sparse attention and its gradients by definition, in 64 bits, with the errors
that the kernels' arithmetic may make.

u = 2^-8 is half a BF16 step, e = 2^-24 half an FP32 step.  The scores and do . c are
sums of 512 exact products in FP32: off by at most 512 e times the sum of the products'
sizes.  A score that is off by x puts a factor e^x on its probability; 2^x in hardware
and the scaling by log2(e) add a few e of the exponent.  p and ds are rounded to BF16
before they multiply rows (u each), outputs are rounded once (u), and sums of n terms in
FP32 add n e of the terms' sizes."""
import math

import torch

U, E = 2.0 ** -8, 2.0 ** -24
H, DC = 64, 512


class Row:
    """One row's probabilities and their errors: q [64, 512], keys [n, 512] in 64 bits."""

    def __init__(self, q, keys, scale, lse=None):
        self.q, self.keys, self.scale = q, keys, scale
        self.s = scale * (q @ keys.T)
        size = 512 * E * scale * (q.abs() @ keys.abs().T)
        self.lse = torch.logsumexp(self.s, 1) if lse is None else lse
        self.p = torch.exp(self.s - self.lse[:, None])
        # relative error of p: of its exponent (the score's, the FP32 difference's), then of 2^x
        self.e_p = size + 8 * E * (self.s.abs() + self.lse.abs()[:, None] + 1) * math.log2(math.e)


def check_forward(o, lse, q, keys, scale, what=""):
    """o [64, 512], lse [64] of one row against its listed keys [n, 512] (repeats listed twice)."""
    if keys.shape[0] == 0:
        assert torch.all(o == 0) and torch.all(torch.isneginf(lse)), what
        return
    r = Row(q.double(), keys.double(), scale)
    want, size = r.p @ r.keys, (r.p * (U + 2 * r.e_p)) @ r.keys.abs()
    tol = size + U * want.abs() + 3 * keys.shape[0] * E * (r.p @ r.keys.abs()) + 1e-30
    err = (o.double() - want).abs()
    assert torch.all(err <= tol), (what, float((err / tol).max()))
    # the log of a sum of p: off by the sum's relative error
    tol = (r.p * r.e_p).sum(1) + (keys.shape[0] + 4) * E + 4 * E * (1 + r.lse.abs())
    err = (lse.double() - r.lse).abs()
    assert torch.all(err <= tol), (what, float((err / tol).max()))


class Grads:
    """Gradients over all rows by definition, with error bounds.  `lists[t]`: the latent rows that row t
    lists, a LongTensor.  `o_err`: how far the o that is given may be from the exact one (for tests
    against the true function), per element, relative."""

    def __init__(self, q, kv, lists, o, lse, d_o, scale, d_lse=None, o_err=0.0, rows=None):
        n = q.shape[0]
        self.rows = range(n) if rows is None else rows
        kvd = kv.double()
        self.dq = torch.zeros(n, H, DC, dtype=torch.float64, device=q.device)
        self.dq_tol = torch.zeros_like(self.dq)
        self.dkv = torch.zeros_like(kvd)
        size, tol = torch.zeros_like(kvd), torch.zeros_like(kvd)
        count = torch.zeros(kv.shape[0], 1, dtype=torch.float64, device=q.device)
        for t in self.rows:
            j = lists[t]
            if j.numel() == 0:
                continue
            r = Row(q[t].double(), kvd[j], scale, lse[t].double())
            do, od = d_o[t].double(), o[t].double()
            dp = do @ r.keys.T
            delta = (do * od).sum(1, keepdim=True) - (0 if d_lse is None else d_lse[t].double()[:, None])
            ds = scale * r.p * (dp - delta)
            back = (do * od).abs().sum(1, keepdim=True)
            e_dp = 512 * E * (do.abs() @ r.keys.abs().T) + 520 * E * back + o_err * back + 4 * E * (dp.abs() + delta.abs())
            e_ds = ds.abs() * (U + 2 * r.e_p) + scale * r.p * e_dp * (1 + U)
            e_p = r.p * (U + 2 * r.e_p)
            self.dq[t] = ds @ r.keys
            self.dq_tol[t] = e_ds @ r.keys.abs() + 2 * j.numel() * E * (ds.abs() @ r.keys.abs())
            self.dkv.index_add_(0, j, ds.T @ r.q + r.p.T @ do)
            size.index_add_(0, j, ds.abs().T @ r.q.abs() + r.p.T @ do.abs())
            tol.index_add_(0, j, e_ds.T @ r.q.abs() + e_p.T @ do.abs())
            count.index_add_(0, j, torch.ones(j.numel(), 1, dtype=torch.float64, device=q.device))
        # sums over a row's 128 products, then over the rows that list the token
        self.dkv_tol = tol + (128 + count) * E * size

    def check(self, dq, dkv, what=""):
        for t in self.rows:
            err, tol = (dq[t].double() - self.dq[t]).abs(), self.dq_tol[t] + U * self.dq[t].abs() + 1e-30
            assert torch.all(err <= tol), (what, "dq", t, float((err / tol).max()))
        err, tol = (dkv.double() - self.dkv).abs(), self.dkv_tol + U * self.dkv.abs() + 1e-30
        bad = err > tol
        assert not bad.any(), (what, "dkv", bad.nonzero()[:4].tolist(), float((err / tol).max()))

"""2-norms of the errors of the sparse attention's outputs and gradients, beside the bounds
of single values in mla_grad_checks: those grow with the number n of a sum's terms, and the
sum itself with sqrt(n), so that a term more or less is lost in them where many rows list a
token.

Errors of different (row, head, token) are independent: each comes from roundings of its own
data.  Call b_i the bound of the i-th term's error (mla_grad_checks: half a BF16 step of p
or ds, and the FP32 errors in them, times the row that they multiply).  FP32 sums make n
roundings more, each of a partial sum, whose square is at most the sum of the terms' squares
in the mean.  So the square of the error's 2-norm is at most V = sum_i b_i^2 + (n e)^2 sum_i
term_i^2 in the mean, and over thousands of terms it stays within some percent of that mean
(a rounding is spread over its range, so that a third of V is what it comes to).  Of one
latent row, or one (row, head), with few terms perhaps, the norm passes x times the root of V
with a probability of at most 2 exp(-x^2 / 2) (Pinelis' bound for sums of independent vectors
of norms b_i): x = 6 gives 3e-8.  The last rounding adds u of the value."""
import torch

from mla_grad_checks import DC, E, H, U, Row


def check_norms(got, want, var, what=""):
    """`got` against `want` [..., width], whole and row by row; var [..., width]: V of each value."""
    err, var, size = ((x.reshape(-1, x.shape[-1]) ** 2).sum(1) for x in (got.double() - want, var.sqrt(), want))
    whole, limit = float(err.sum().sqrt()), float(var.sum().sqrt() + U * size.sum().sqrt())
    assert whole <= limit, (what, "all rows", whole, limit)
    limits = 6 * var.sqrt() + U * size.sqrt() + 1e-30
    bad = err.sqrt() > limits
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), float((err.sqrt() / limits).max()))


def check_outputs(o, q, kv, lists, scale, what=""):
    """o [rows, 64, 512] against the definition; no row lists a token twice."""
    want = torch.zeros(o.shape, dtype=torch.float64, device=o.device)
    var, kvd = torch.zeros_like(want), kv.double()
    for t, j in enumerate(lists):
        if j.numel():
            r = Row(q[t].double(), kvd[j], scale)
            want[t] = r.p @ r.keys
            # (errors of p that all of a head's tokens share cancel against those of the sum)
            var[t] = (r.p * (U + 2 * r.e_p + j.numel() * E)) ** 2 @ r.keys ** 2 + (j.numel() * E * want[t]) ** 2
    check_norms(o, want, var, what)


class GradNorms:
    """Gradients over all rows by definition, and the V of each of their values."""

    def __init__(self, q, kv, lists, o, lse, d_o, scale, d_lse=None):
        kvd = kv.double()
        self.dq = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        self.dkv = torch.zeros_like(kvd)
        self.dq_var, self.dkv_var, size = torch.zeros_like(self.dq), torch.zeros_like(kvd), torch.zeros_like(kvd)
        count = torch.zeros(kv.shape[0], 1, dtype=torch.float64, device=q.device)
        for t, j in enumerate(lists):
            if j.numel() == 0:
                continue
            # (a token's repeats in a row have one p and one ds, and so the same errors: one term, n times as large)
            n_row = j.numel()
            j, n = j.unique(return_counts=True)
            r = Row(q[t].double(), kvd[j], scale, lse[t].double())
            r.p = r.p * n
            do, od = d_o[t].double(), o[t].double()
            dp = do @ r.keys.T
            delta = (do * od).sum(1, keepdim=True) - (0 if d_lse is None else d_lse[t].double()[:, None])
            ds = scale * r.p * (dp - delta)
            back = (do * od).abs().sum(1, keepdim=True)
            # (an error of delta is one for all of a head's tokens: in dq its parts add up)
            e_delta = scale * r.p * (520 * E * back + 4 * E * delta.abs())
            e_ds = ds.abs() * (U + 2 * r.e_p) + scale * r.p * (512 * E * (do.abs() @ r.keys.abs().T) + 4 * E * dp.abs())
            e_p = r.p * (U + 2 * r.e_p)
            self.dq[t] = ds @ r.keys
            self.dq_var[t] = (e_ds ** 2 + (n_row * E * ds) ** 2) @ r.keys ** 2 + (e_delta @ r.keys.abs()) ** 2
            self.dkv.index_add_(0, j, ds.T @ r.q + r.p.T @ do)
            self.dkv_var.index_add_(0, j, ((e_ds + e_delta) ** 2).T @ r.q ** 2 + (e_p ** 2).T @ do ** 2)
            size.index_add_(0, j, (ds ** 2).T @ r.q ** 2 + (r.p ** 2).T @ do ** 2)
            count.index_add_(0, j, n.double()[:, None])
        # sums over a row's 128 products, then over the rows that list the token
        self.dkv_var += ((2 * H + count) * E) ** 2 * size

    def check(self, dq, dkv, what=""):
        assert dq.shape[1:] == (H, DC)
        check_norms(dq, self.dq, self.dq_var, (what, "dq"))
        check_norms(dkv, self.dkv, self.dkv_var, (what, "dkv"))

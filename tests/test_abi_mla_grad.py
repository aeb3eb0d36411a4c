"""Refusals of the sparse attention's backward calls and of its paged form, all on
the host: no argument here reaches a device."""
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


def test_backward_arguments_are_checked(b):
    L = b._lib
    keep, a = _fake()
    p, mis, none = P(a), P(a + 2), P(None)
    ws, ws8 = L.kpool_sparse_mla_bwd_workspace_size(4, 8), L.kpool_sparse_mla_bwd_workspace_size(8, 8)
    assert ws >= 256 + 8 * 512 * 4
    assert L.kpool_sparse_mla_bwd_workspace_size(-1, 8) == 0
    assert L.kpool_sparse_mla_bwd_workspace_size(4, 1 << 31) == 0

    def common(call):
        return [
            (call(q=none), -1), (call(kv=none), -1), (call(o=none), -1), (call(lse=none), -1), (call(do=none), -1),
            (call(dq=none), -1), (call(dkv=none), -1), (call(lst=none), -1), (call(lst=mis), -1),
            *[(call(**{k: P(a + 8)}), -1) for k in ("q", "kv", "o", "do", "dq", "dkv")],
            (call(lse=mis), -1), (call(dl=mis), -1), (call(T=-1), -1), (call(T=1 << 31), -1), (call(H=32), -2),
            (call(Dc=576), -2), (call(scale=0.0), -1), (call(scale=float("nan")), -1), (call(scale=float("inf")), -1),
            (call(w=none), -4), (call(w=P(a + 16)), -4), (call(wb=256), -4)]

    def lists(q=p, kv=p, lst=p, o=p, lse=p, do=p, dl=none, T=4, Tk=8, W=4, H=64, Dc=512, scale=0.1, dq=p, dkv=p, w=p,
              wb=ws):
        return L.kpool_sparse_mla_bwd(q, kv, lst, o, lse, do, dl, T, Tk, W, H, Dc, scale, dq, dkv, w, wb, None)

    def pools(q=p, kv=p, lst=p, cu=p, cp=p, nd=2, o=p, lse=p, do=p, dl=none, T=8, H=64, Dc=512, kp=4, topk=8,
              scale=0.1, dq=p, dkv=p, w=p, wb=ws8):
        return L.kpool_sparse_mla_bwd_pools(q, kv, lst, cu, cp, nd, o, lse, do, dl, T, H, Dc, kp, topk, 1, scale, dq,
                                            dkv, w, wb, None)

    def at(q=p, kv=p, lst=p, cu=p, pos=p, ck=p, cp=p, nd=2, o=p, lse=p, do=p, dl=none, T=4, Tk=8, H=64, Dc=512, kp=4,
           topk=8, scale=0.1, dq=p, dkv=p, w=p, wb=ws):
        return L.kpool_sparse_mla_bwd_pools_at(q, kv, lst, cu, pos, ck, cp, nd, o, lse, do, dl, T, Tk, H, Dc, kp, topk,
                                               1, scale, dq, dkv, w, wb, None)

    bad = common(lists) + common(pools) + common(at)
    bad += [(lists(W=-1), -1), (lists(W=1 << 21), -1), (lists(Tk=-1), -1), (lists(Tk=1 << 31), -1), (lists(wb=ws - 1), -4),
            (pools(wb=ws8 - 1), -4)]
    for call in (pools, at):
        bad += [(call(kp=0), -2), (call(kp=65), -2), (call(topk=0), -1), (call(topk=7), -1), (call(nd=0), -1),
                (call(cu=none), -1), (call(cp=none), -1), (call(cu=mis), -1), (call(cp=mis), -1)]
    bad += [(at(pos=none), -1), (at(ck=none), -1), (at(pos=mis), -1), (at(ck=mis), -1)]
    for i, (got, want) in enumerate(bad):
        assert got == want, (i, got, want)
    assert L.kpool_last_error()
    del keep


def test_paged_arguments_are_checked(b):
    L = b._lib
    keep, a = _fake()
    p, mis, none = P(a), P(a + 2), P(None)
    ws = L.kpool_sparse_mla_paged_workspace_size(4, 4, 64)
    assert ws >= 256
    assert [L.kpool_sparse_mla_paged_workspace_size(*x) for x in ((-1, 4, 64), (1 << 31, 4, 64), (4, 0, 64),
                                                                 (4, 65, 65), (4, 4, 63), (4, 4, 0))] == [0] * 6

    def call(q=p, kv=p, stride=16 * 512, np_=32, ps=16, pt=p, sl=p, nr=4, mp=8, ids=p, pi=p, cq=p, pos=p, cp=p, B=3,
             Tq=4, H=64, Dc=512, kp=4, topk=64, scale=0.1, o=p, lse=p, w=p, wb=ws):
        return L.kpool_sparse_mla_fwd_pools_paged(q, kv, stride, np_, ps, pt, sl, nr, mp, ids, pi, cq, pos, cp, B, Tq,
                                                  H, Dc, kp, topk, 1, scale, o, lse, w, wb, None)

    bad = [
        *[(call(**{k: none}), -1) for k in ("q", "kv", "pt", "sl", "pi", "cq", "pos", "cp", "o", "lse")],
        *[(call(**{k: P(a + 8)}), -1) for k in ("q", "kv", "o")],
        *[(call(**{k: mis}), -1) for k in ("pt", "sl", "ids", "pi", "cq", "pos", "cp", "lse")],
        (call(stride=16 * 512 - 8), -1), (call(stride=16 * 512 + 4), -1), (call(stride=1 << 34), -1),
        (call(np_=0), -1), (call(np_=(1 << 28) + 1), -1), (call(ps=0), -1), (call(nr=0), -1), (call(mp=0), -1),
        (call(mp=(1 << 20) + 1), -1), (call(mp=1 << 20, ps=1 << 11, stride=1 << 20), -1), (call(ids=none, nr=2), -1),
        (call(B=0), -1), (call(B=(1 << 24) + 1), -1), (call(Tq=-1), -1), (call(Tq=1 << 31), -1), (call(H=128), -2),
        (call(Dc=256), -2), (call(kp=0), -2), (call(kp=65), -2), (call(topk=0), -1), (call(topk=66), -1),
        (call(scale=0.0), -1), (call(scale=float("nan")), -1), (call(w=none), -4), (call(w=P(a + 16)), -4),
        (call(wb=ws - 1), -4)]
    for i, (got, want) in enumerate(bad):
        assert got == want, (i, got, want)
    del keep


def test_the_binding_refuses_tensors_of_the_host(b):
    bf, i32 = torch.zeros(2, 64, 512, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    kv, lse = bf[0], torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        b.kpool_sparse_mla_bwd(bf, kv, i32.view(2, 2), bf, lse, bf, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        b.kpool_sparse_mla_bwd_pools_at(bf, kv, i32.view(2, 2), bf, lse, bf, 4, 8, 0.1, i32, i32, i32, i32)
    with pytest.raises(ValueError, match="CUDA"):
        b.kpool_sparse_mla_bwd_pools(bf, kv[:2], i32.view(2, 2), bf, lse, bf, 4, 8, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        b.kpool_sparse_mla_fwd_pools_paged(bf, bf, i32.view(2, 2), i32, i32.view(2, 2), 4, 8, 0.1, i32, i32, i32)

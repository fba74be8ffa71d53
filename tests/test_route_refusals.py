"""Refusals of the general router, the activation with dropout and the AWQ product, on the CPU: nothing here launches a
kernel."""
import ctypes

import pytest
import torch

import top_moe_expert_gb300 as moe
from top_moe_expert_gb300 import build

A = 1 << 20                                                    # an aligned address no call may reach
BF, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def test_route_refuses_before_launch(L):
    def fwd(logits=A, ldt=2, bias=A, M=4, E=16, k=4, score=0, groups=4, topk_groups=2, group_top=2, renorm=1, scale=1.0,
            ids=A, w=A, load=A):
        return L.moe_route(logits, ldt, bias, M, E, k, score, groups, topk_groups, group_top, renorm, scale, ids, w, load, None)

    def bwd(dw=A, logits=A, ldt=2, ids=A, M=4, E=16, k=4, score=0, renorm=1, scale=1.0, dl=A):
        return L.moe_route_bwd(dw, logits, ldt, ids, M, E, k, score, renorm, scale, dl, None)

    inf, nan = float("inf"), float("nan")
    for bad in (dict(M=-1), dict(E=0), dict(k=0), dict(k=17), dict(score=2), dict(score=-1), dict(renorm=2), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=inf), dict(scale=nan), dict(logits=None), dict(ids=None), dict(logits=A + 2),
                dict(ids=A + 2)):
        assert fwd(**bad) == 1 and bwd(**bad) == 1, bad
    for bad in (dict(groups=0), dict(groups=3), dict(groups=32), dict(topk_groups=0), dict(topk_groups=5), dict(k=9),
                dict(group_top=0), dict(group_top=3), dict(w=None), dict(bias=A + 2), dict(w=A + 1), dict(load=A + 2)):
        assert fwd(**bad) == 1, bad
    for bad in (dict(dw=None), dict(dl=None), dict(dw=A + 2), dict(dl=A + 2), dict(dl=A + 1, ldt=0)):
        assert bwd(**bad) == 1, bad
    for bad in (dict(ldt=3), dict(ldt=-1), dict(E=1025, groups=1, topk_groups=1), dict(E=64, groups=1, topk_groups=1, k=33),
                dict(E=128, groups=64), dict(M=2 ** 31 - 1)):
        assert fwd(**bad) == 2, bad
    for bad in (dict(ldt=3), dict(E=1025), dict(E=64, k=33), dict(M=2 ** 31 - 1)):
        assert bwd(**bad) == 2, bad
    assert fwd(M=0, logits=None, ids=None, w=None, bias=None, load=None) == 0
    assert bwd(M=0, dw=None, logits=None, ids=None, dl=None) == 0


def test_swiglu_refuses_before_launch(L):
    def both(dh=A, gu=A, dt=0, R=4, I=16, p=0.1, rng=A, out=A):
        return (L.moe_swiglu_dropout(gu, dt, R, I, p, rng, out, None), L.moe_swiglu_dropout_bwd(dh, gu, dt, R, I, p, rng, out, None))

    for bad in (dict(R=-1), dict(I=0), dict(I=-8), dict(p=-0.1), dict(p=1.0), dict(p=1 - 2.0 ** -17), dict(p=float("nan")),
                dict(gu=None), dict(out=None), dict(rng=None), dict(rng=A + 4), dict(gu=A + 1), dict(out=A + 1),
                dict(gu=A + 2, dt=2)):
        assert both(**bad) == (1, 1), bad
    assert both(dh=None, gu=None)[1] == 1 and both(dh=A + 1, gu=None)[1] == 1
    for bad in (dict(dt=3), dict(I=2 ** 31 - 1), dict(R=2 ** 31 - 1, I=17), dict(R=2 ** 20, I=2 ** 15)):
        assert both(**bad) == (2, 2), bad
    assert both(R=0, dh=None, gu=None, rng=None, out=None) == (0, 0)


def test_awq_product_refuses_before_launch(L):
    def call(x=A, dt=0, fmt=1, E=2, N=64, K=256, q=A, scale=A, zero=A, off=A, R=4, y=A, ydt=0, st=None):
        w = moe.moe_weights_t(fmt, E, N, K, q, scale, zero)
        return L.moe_grouped_mm_awq(x, dt, ctypes.byref(w), off, R, y, ydt, st, None)

    assert L.moe_grouped_mm_awq(A, 0, None, A, 4, A, 0, None, None) == 1
    for bad in (dict(R=-1), dict(E=0), dict(N=0), dict(K=0), dict(N=12), dict(K=192), dict(x=None), dict(q=None),
                dict(scale=None), dict(zero=None), dict(off=None), dict(y=None), dict(x=A + 8), dict(q=A + 4),
                dict(scale=A + 8), dict(zero=A + 8), dict(off=A + 2), dict(y=A + 2), dict(st=A + 2)):
        assert call(**bad) == 1, bad
    for bad in (dict(fmt=0), dict(fmt=3), dict(dt=2), dict(ydt=1), dict(dt=1, ydt=0), dict(E=1025), dict(R=2 ** 31 - 8),
                dict(N=2 ** 31 - 8), dict(K=2 ** 31 - 128), dict(E=1024, R=2 ** 24)):
        assert call(**bad) == 2, bad
    assert call(R=0, x=None, y=None, off=None) == 0


class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.startswith(("moe_route", "moe_swiglu", "moe_grouped_mm_awq")):
            return lambda *a: self.calls.append(name) or 0
        return getattr(self.real, name)


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_is_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_stream", lambda stream=None, device=None: ctypes.c_void_p(0))
    return r


def test_route_binding_checks(rec):
    l, b = torch.zeros((5, 16)), torch.zeros(16)
    ids, w = moe.moe_route(l, 4, bias=b, groups=4, topk_groups=2, group_top=2)
    assert ids.shape == w.shape == (5, 4) and ids.dtype == I32 and w.dtype == F32
    dl = moe.moe_route_bwd(w, l.bfloat16(), ids)
    assert dl.shape == (5, 16) and dl.dtype == BF and len(rec.calls) == 2
    for bad in (dict(k=0), dict(k=17), dict(k=9, groups=4, topk_groups=2), dict(score=2), dict(groups=3), dict(groups=0),
                dict(groups=4, topk_groups=5), dict(topk_groups=0), dict(group_top=3), dict(scale=0.0), dict(scale=float("nan")),
                dict(bias=b.bfloat16()), dict(bias=b[:8]), dict(bias=[0.0] * 16), dict(load=b), dict(load=torch.zeros(8, dtype=I32)),
                dict(topk_ids=ids[:, :3]), dict(topk_ids=w), dict(topk_w=w.double()), dict(topk_w=torch.zeros((4, 5)).t())):
        with pytest.raises(ValueError):
            moe.moe_route(l, **{"k": 4, **bad})
    for bad in (l[0], l.double(), l.t(), None, l.int()):
        with pytest.raises(ValueError):
            moe.moe_route(bad, 4)
    for a in ((w[:4], l, ids), (w, l, ids[:4]), (w.bfloat16(), l, ids), (w, l, ids.long()), (w, l[0], ids), (None, l, ids),
              (w, None, ids), (w, l, None), (w, l[:, :3].contiguous(), ids)):
        with pytest.raises(ValueError):
            moe.moe_route_bwd(*a)
    with pytest.raises(ValueError):
        moe.moe_route_bwd(w, l, ids, dlogits=torch.zeros((5, 16), dtype=BF))
    assert len(rec.calls) == 2


def test_swiglu_binding_checks(rec):
    gu, rng = torch.zeros((5, 32), dtype=F16), torch.zeros(2, dtype=torch.int64)
    h = moe.moe_swiglu_dropout(gu, 0.1, rng)
    assert h.shape == (5, 16) and h.dtype == F16
    assert moe.moe_swiglu_dropout_bwd(h, gu, 0.1, rng).shape == (5, 32)
    moe.moe_swiglu_dropout(gu)
    moe.moe_swiglu_dropout(gu, 2.0 ** -18)
    moe.moe_swiglu_dropout_bwd(h, gu, 0.1, rng, dgu=gu)
    assert len(rec.calls) == 5
    for a in ((gu, 0.1), (gu, -0.1, rng), (gu, 1.0, rng), (gu, float("nan"), rng), (gu, 0.1, rng.int()), (gu, 0.1, rng[:1]),
              (gu, 0.1, [0, 0]), (gu[:, :31].contiguous(), 0.1, rng), (gu.t(), 0.1, rng), (gu[0], 0.1, rng), (None, 0.1, rng),
              (gu.double(), 0.1, rng), (torch.zeros((3, 0)), 0.1, rng)):
        with pytest.raises(ValueError):
            moe.moe_swiglu_dropout(*a)
        with pytest.raises(ValueError):
            moe.moe_swiglu_dropout_bwd(h, *a)
    for dh in (h.float(), h[:4], h[:, :8].contiguous(), None):
        with pytest.raises(ValueError):
            moe.moe_swiglu_dropout_bwd(dh, gu, 0.1, rng)
    with pytest.raises(ValueError):
        moe.moe_swiglu_dropout(gu, 0.1, rng, h=h.float())
    assert len(rec.calls) == 5


def test_awq_product_binding_checks(rec):
    q, s, z = torch.zeros((2, 16, 32), dtype=I32), torch.zeros((2, 16, 2), dtype=F16), torch.zeros((2, 2, 2), dtype=I32)
    w, x, off = moe.Weights(moe.MOE_W_AWQ4, q, s, z), torch.zeros((5, 256), dtype=BF), torch.zeros(3, dtype=I32)
    assert moe.moe_grouped_mm_awq(x, w, off).dtype == BF
    assert moe.moe_grouped_mm_awq(x.half(), w, off, out_dtype=F32).shape == (5, 16)
    assert len(rec.calls) == 2
    other = moe.Weights(moe.MOE_W_MXFP8, torch.zeros((2, 16, 256), dtype=torch.uint8), torch.zeros((2, 16, 8), dtype=torch.uint8))
    for a in ((x, other, off), (x, q, off), (x, None, off), (x.float(), w, off), (x[:, :128].contiguous(), w, off), (x.t(), w, off),
              (x, w, off[:2]), (x, w, off.long()), (x, w, [0, 1, 2]), (None, w, off), (x[0], w, off)):
        with pytest.raises(ValueError):
            moe.moe_grouped_mm_awq(*a)
    for kw in (dict(out_dtype=F16), dict(y=torch.zeros((5, 8), dtype=BF)), dict(y=torch.zeros((5, 16), dtype=F16)),
               dict(dev_status=torch.zeros(1, dtype=I32)), dict(dev_status=torch.zeros(2))):
        with pytest.raises(ValueError):
            moe.moe_grouped_mm_awq(x, w, off, **kw)
    assert len(rec.calls) == 2

"""Fp4 objects: what a launch takes from them is what was checked (CPU; launches are recorded)."""
import copy
import ctypes
import pickle

import pytest
import torch

import top_moe_expert_gb300 as moe


class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        return (lambda *a: self.calls.append(a) or 0) if name == "moe_grouped_mm_fp4" else getattr(self.real, name)


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_is_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_stream", lambda stream=None, device=None: ctypes.c_void_p(0))
    return r


def _pair():
    q, s, q3, s3 = (torch.zeros(n, dtype=torch.uint8) for n in ((5, 32), (5, 16), (2, 64, 32), (2, 64, 16)))
    return moe.Fp4(0, q, s, torch.ones(1)), moe.Fp4(0, q3, s3, torch.ones(2)), torch.zeros(3, dtype=torch.int32)


def test_fields_are_fixed(rec):
    x, w, off = _pair()
    for field, value in (("s", torch.zeros(3)), ("alpha", None), ("q", x.q[:2]), ("fmt", 1), ("other", 0)):
        with pytest.raises(AttributeError):
            setattr(x, field, value)
    for field in ("fmt", "q", "s", "alpha"):
        with pytest.raises(AttributeError):
            delattr(x, field)
    moe.moe_grouped_mm_fp4(x, w, off)
    assert len(rec.calls) == 1 and rec.calls[0][2] == x.alpha.data_ptr()


def test_copies_are_checked_again(rec):
    x, w, off = _pair()
    for f in (copy.copy, copy.deepcopy, lambda t: pickle.loads(pickle.dumps(t))):
        y = f(w)
        assert y is not w and y.fmt == w.fmt and torch.equal(y.q, w.q) and torch.equal(y.alpha, w.alpha)
        moe.moe_grouped_mm_fp4(x, y, off)
    assert len(rec.calls) == 3


def test_arguments_of_other_kinds_are_refused(rec):
    x, w, off = _pair()
    for a in ((x.q, w, off), (x, w.q, off), (None, w, off), (x, None, off), (x, w, [0, 1, 2]), (x, w, None), (x, w, off.float())):
        with pytest.raises(ValueError):
            moe.moe_grouped_mm_fp4(*a)
    t = torch.zeros((5, 32), dtype=torch.bfloat16)
    for f in (moe.moe_grouped_mm, moe.moe_grouped_mm_dgrad, moe.moe_grouped_mm_wgrad):
        for a in ((t, None, off), (None, t, off), (t, t, [0, 1, 2]), (t, t, None)):
            with pytest.raises(ValueError):
                f(*a)
    for f in (lambda: moe.moe_fp4_quantize(None, 1), lambda: moe.moe_fp4_quantize(t, 0, [1.0]),
              lambda: moe.moe_fp4_dequantize(x.q, None, 1), lambda: moe.Fp4(0, x.q, None, x.alpha), lambda: moe.Fp4(0, None, x.s)):
        with pytest.raises(ValueError):
            f()
    assert not rec.calls

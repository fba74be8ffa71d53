"""Refusals of the ragged grouped products and the 4-bit formats, on the CPU: nothing here launches a kernel."""
import ctypes

import pytest
import torch

import top_moe_expert_gb300 as moe
from top_moe_expert_gb300 import build

BF = torch.bfloat16
A = 1 << 20                                                    # an aligned address no call may reach


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def _mm(L, fn, x=A, w=A, dt=0, off=A, R=4, E=2, N=64, K=32, y=A, ydt=0, *more):
    return getattr(L, fn)(x, w, dt, off, R, E, N, K, y, ydt, *more, None, None)


@pytest.mark.parametrize("fn,more", [("moe_grouped_mm", ()), ("moe_grouped_mm_dgrad", ()), ("moe_grouped_mm_wgrad", (0,))])
def test_products_refuse_before_launch(L, fn, more):
    call = lambda **k: _mm(L, fn, *[k.get(n, d) for n, d in zip(  # noqa: E731
        ("x", "w", "dt", "off", "R", "E", "N", "K", "y", "ydt"), (A, A, 0, A, 4, 2, 64, 32, A, 0))], *more)
    for bad in (dict(R=-1), dict(E=0), dict(N=0), dict(K=0), dict(x=None), dict(w=None), dict(off=None), dict(y=None),
                dict(x=A + 8), dict(w=A + 2), dict(y=A + 4), dict(off=A + 2)):
        assert call(**bad) == 1, bad
    for bad in (dict(dt=2), dict(ydt=1), dict(N=60), dict(K=20), dict(E=1025), dict(dt=7), dict(ydt=9)):
        assert call(**bad) == 2, bad


def test_sizes_past_32_bits(L):
    """Sides whose tiles, or tile count with any offsets, would not count in 32 bits; the binding's that a C int cuts."""
    top = 2 ** 31 - 8
    for fn, more in (("moe_grouped_mm", ()), ("moe_grouped_mm_dgrad", ()), ("moe_grouped_mm_wgrad", (0,))):
        for sides in ((top, 8, 8), (8, top, 8), (8, 8, top)):
            assert _mm(L, fn, A, A, 0, A, sides[0], 2, *sides[1:], A, 0, *more) == 2, (fn, sides)
        assert _mm(L, fn, A, A, 0, A, 2 ** 30, 1024, 2 ** 20, 2 ** 20, A, 0, *more) == 2
    for sides in ((top, 8, 32), (8, top, 32), (8, 8, 2 ** 31 - 32), (2 ** 30, 2 ** 20, 32)):
        assert L.moe_grouped_mm_fp4(A, A, None, A, A, None, 1, A, sides[0], 1024, *sides[1:], A, 0, None, None) == 2, sides
    for rows, K in ((2 ** 62, 64), (2 ** 32, 32), (1, 2 ** 31 - 32)):
        assert L.moe_fp4_quantize(A, 0, rows, K, 1, None, 1, A, A, None) == 2, (rows, K)
        assert L.moe_fp4_dequantize(A, A, rows, K, 1, None, 1, A, 0, None) == 2, (rows, K)


def test_wgrad_flag(L):
    assert _mm(L, "moe_grouped_mm_wgrad", A, A, 0, A, 4, 2, 64, 32, A, 0, 2) == 1


def test_no_rows_touch_nothing(L):
    assert _mm(L, "moe_grouped_mm", None, None, 0, None, 0) == 0
    assert _mm(L, "moe_grouped_mm_dgrad", None, None, 0, None, 0) == 0


def test_fp4_refusals(L):
    n = ctypes.c_int32()
    for K, fmt, cols in ((32, 0, 16), (256, 0, 16), (288, 0, 32), (2048, 0, 128), (32, 1, 16), (768, 1, 32), (2048, 1, 64)):
        assert L.moe_fp4_scale_cols(K, fmt, ctypes.byref(n)) == 0 and n.value == cols
        assert moe._fp4_shape(K, fmt, "K") == cols
    assert L.moe_fp4_scale_cols(0, 0, ctypes.byref(n)) == 1 and L.moe_fp4_scale_cols(48, 0, ctypes.byref(n)) == 1
    assert L.moe_fp4_scale_cols(64, 2, ctypes.byref(n)) == 2

    def quant(v=A, vdt=0, rows=4, K=64, fmt=0, alpha=A, groups=1, q=A, s=A):
        return (L.moe_fp4_quantize(v, vdt, rows, K, fmt, alpha, groups, q, s, None),
                L.moe_fp4_dequantize(q, s, rows, K, fmt, alpha, groups, v, vdt, None))

    for bad in (dict(rows=-1), dict(K=0), dict(K=48), dict(groups=0), dict(groups=3), dict(alpha=None), dict(v=None),
                dict(q=None), dict(s=None), dict(v=A + 4), dict(q=A + 8), dict(s=A + 1), dict(fmt=1)):
        assert quant(**bad) == (1, 1), bad
    for bad in (dict(fmt=2), dict(vdt=3)):
        assert quant(**bad) == (2, 2), bad
    assert quant(rows=0, v=None, q=None, s=None) == (0, 0)

    def mm(xq=A, xs=A, xa=A, wq=A, ws=A, wa=A, fmt=0, off=A, R=4, E=2, N=64, K=64, y=A, ydt=0):
        return L.moe_grouped_mm_fp4(xq, xs, xa, wq, ws, wa, fmt, off, R, E, N, K, y, ydt, None, None)

    for bad in (dict(R=-1), dict(E=0), dict(N=0), dict(K=-32), dict(xq=None), dict(xs=None), dict(xa=None), dict(wq=None),
                dict(ws=None), dict(wa=None), dict(off=None), dict(y=None), dict(fmt=1), dict(xq=A + 8), dict(ws=A + 4),
                dict(y=A + 2)):
        assert mm(**bad) == 1, bad
    for bad in (dict(fmt=5), dict(ydt=4), dict(E=2000), dict(N=12), dict(K=48)):
        assert mm(**bad) == 2, bad
    assert mm(R=0, xq=None, y=None) == 0


class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.startswith("moe_grouped_mm") or name in ("moe_fp4_quantize", "moe_fp4_dequantize"):
            return lambda *a: self.calls.append(name) or 0
        return getattr(self.real, name)


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_is_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_stream", lambda stream=None, device=None: ctypes.c_void_p(0))
    return r


def test_binding_checks(rec):
    x, w, dy = torch.zeros((5, 32), dtype=BF), torch.zeros((2, 64, 32), dtype=BF), torch.zeros((5, 64), dtype=BF)
    off = torch.zeros(3, dtype=torch.int32)
    assert moe.moe_grouped_mm(x, w, off).shape == (5, 64)
    assert moe.moe_grouped_mm_dgrad(dy, w, off).shape == (5, 32)
    assert moe.moe_grouped_mm_wgrad(dy, x, off).dtype == torch.float32
    assert rec.calls == ["moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad"]
    bad = [
        lambda: moe.moe_grouped_mm(x.half(), w, off),
        lambda: moe.moe_grouped_mm(x.float(), w.float(), off),
        lambda: moe.moe_grouped_mm(x[0], w, off),
        lambda: moe.moe_grouped_mm(x, w[0], off),
        lambda: moe.moe_grouped_mm(x, w.transpose(1, 2), off),
        lambda: moe.moe_grouped_mm(x, torch.zeros((3, 64, 32), dtype=BF), off),
        lambda: moe.moe_grouped_mm(x, torch.zeros((2, 64, 40), dtype=BF), off),
        lambda: moe.moe_grouped_mm(x, w, off.long()),
        lambda: moe.moe_grouped_mm(x, w, off[:1]),
        lambda: moe.moe_grouped_mm(x, w, off, y=torch.zeros((4, 64), dtype=BF)),
        lambda: moe.moe_grouped_mm(x, w, off, out_dtype=torch.float16),
        lambda: moe.moe_grouped_mm(x, w, off, dev_status=torch.zeros(1, dtype=torch.int32)),
        lambda: moe.moe_grouped_mm_dgrad(x, w, off),
        lambda: moe.moe_grouped_mm_dgrad(dy, w, off, dx=torch.zeros((5, 64), dtype=BF)),
        lambda: moe.moe_grouped_mm_wgrad(dy, x[:4], off),
        lambda: moe.moe_grouped_mm_wgrad(dy, x, off, accumulate=True),
        lambda: moe.moe_grouped_mm_wgrad(dy, x, off, dw=torch.zeros((2, 32, 64))),
    ]
    q, s, q3, s3 = (torch.zeros(n, dtype=torch.uint8) for n in ((5, 32), (5, 16), (2, 64, 32), (2, 64, 16)))
    one, two = torch.ones(1), torch.ones(2)
    X, W = moe.Fp4(0, q, s, one), moe.Fp4(0, q3, s3, two)
    assert moe.moe_grouped_mm_fp4(X, W, off).shape == (5, 64)
    bad += [
        lambda: moe.Fp4(2, q, s, one),
        lambda: moe.Fp4(0, q, s),
        lambda: moe.Fp4(1, q, s, one),
        lambda: moe.Fp4(0, q, s[:, :8], one),
        lambda: moe.Fp4(0, q3, s3, one),
        lambda: moe.Fp4(0, q.int(), s, one),
        lambda: moe.moe_grouped_mm_fp4(W, W, off),
        lambda: moe.moe_grouped_mm_fp4(moe.Fp4(1, q, s), W, off),
        lambda: moe.moe_grouped_mm_fp4(X, W, torch.zeros(2, dtype=torch.int32)),
        lambda: moe.moe_grouped_mm_fp4(X, W, off, out_dtype=torch.float64),
        lambda: moe.moe_fp4_quantize(torch.zeros((4, 48)), 1),
        lambda: moe.moe_fp4_quantize(torch.zeros((4, 64)), 0),
        lambda: moe.moe_fp4_quantize(torch.zeros((4, 64)), 1, one),
        lambda: moe.moe_fp4_quantize(torch.zeros((4, 64)), 0, torch.ones(3)),
        lambda: moe.moe_fp4_quantize(torch.zeros((4, 64)), 1, q=torch.zeros((4, 31), dtype=torch.uint8)),
        lambda: moe.moe_fp4_dequantize(q, s[:4], 1),
        lambda: moe.moe_fp4_dequantize(q, s, 1, out_dtype=torch.int32),
    ]
    n = len(rec.calls)
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    assert len(rec.calls) == n


def test_binding_refuses_sizes_that_would_be_cut(rec):
    """Meta tensors of 2^32 + 8 rows or columns, which a C int takes for 8."""
    big = 2 ** 32 + 8
    m = lambda *s, t=BF: torch.empty(s, dtype=t, device="meta")  # noqa: E731
    off = m(2, t=torch.int32)
    n = len(rec.calls)
    for f in (lambda: moe.moe_grouped_mm(m(big, 8), m(1, 8, 8), off),
              lambda: moe.moe_grouped_mm(m(8, big), m(1, 8, big), off),
              lambda: moe.moe_grouped_mm_dgrad(m(8, 8), m(1, 8, big), off),
              lambda: moe.moe_grouped_mm_wgrad(m(big, 8), m(big, 8), off),
              lambda: moe.moe_fp4_quantize(m(1, 2 ** 32 + 32), 1),
              lambda: moe.moe_fp4_dequantize(m(1, 2 ** 31 + 16, t=torch.uint8), m(1, 16, t=torch.uint8), 1)):
        with pytest.raises(ValueError, match="32 bits"):
            f()
    assert len(rec.calls) == n


def test_captured_backward_beside_an_eager_graph_is_refused(rec, monkeypatch):
    """The leaves' accumulation belongs to the stream of a graph that lives: refused in a capture on another stream."""
    from types import SimpleNamespace

    from top_moe_expert_gb300 import ragged

    state = SimpleNamespace(stream=1, capturing=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=state.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    x = torch.zeros((5, 32), dtype=BF).requires_grad_()
    w = torch.zeros((2, 64, 32), dtype=BF).requires_grad_()
    off = torch.zeros(3, dtype=torch.int32)
    eager = ragged.grouped_linear(x.detach(), w, off)
    state.stream, state.capturing = 2, True
    y = ragged.grouped_linear(x, w, off)
    with pytest.raises(RuntimeError, match="another stream lives"):
        y.sum().backward()
    ragged.grouped_linear(x, w.detach(), off).sum().backward()          # x is not part of the eager graph
    with torch.no_grad():
        ragged.grouped_linear(x, w, off)
    del eager, y
    ragged.grouped_linear(x, w, off).sum().backward()                   # and w no longer is
    state.stream, state.capturing = 1, False
    kept = ragged.grouped_linear(x, w, off)
    kept.sum().backward()
    state.stream = 3
    ragged.grouped_linear(x, w, off).sum().backward()                   # without a capture any stream will do


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.moe_grouped_mm(torch.zeros((5, 32), dtype=BF), torch.zeros((2, 64, 32), dtype=BF), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.moe_fp4_quantize(torch.zeros((4, 64)), 1)

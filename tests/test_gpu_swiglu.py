"""The experts' activation with dropout and its gradient against the plain form in 64 bits; the same elements dropped."""
import gc

import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import route_ref as ref
from top_moe_expert_gb300 import ragged

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def _round(want, tol, dt):
    if dt == F32:
        return tol + 1e-37
    return tol + torch.finfo(dt).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if dt == F16 else 1e-37)


def _check(R, I, p, dt, seed=1, offset=0, std=1.0, g=None):
    g = g or torch.Generator().manual_seed(R + I)
    gu, dh = (std * torch.randn((R, 2 * I), generator=g)).to(dt), torch.randn((R, I), generator=g).to(dt)
    rng = _rng(seed, offset) if ref.threshold(p) else None
    h = moe.moe_swiglu_dropout(gu.cuda(), p, rng).cpu()
    dgu = moe.moe_swiglu_dropout_bwd(dh.cuda(), gu.cuda(), p, rng).cpu()
    assert h.dtype == dgu.dtype == dt and h.shape == (R, I) and dgu.shape == (R, 2 * I)
    keep = ref.kept(R, I, p, seed, offset)
    want, bwd = ref.swiglu(gu, p, keep)
    # exp(-|g|): 2 + 1.7 |g| ulp and a rounded argument, the quotient 3, three products; twice as much for 1 + g (1 - s)
    e = (12 + 2.5 * gu.double()[:, :I].abs().clamp(max=100)) * 2.0 ** -23
    off = (h.double() - want).abs() - _round(want, e * want.abs(), dt)
    assert not (off > 0).any(), float(off.max())
    dwant, mag = bwd(dh)
    off = (dgu.double() - dwant).abs() - _round(dwant, 2 * torch.cat([e, e], dim=1) * mag, dt)
    assert not (off > 0).any(), float(off.max())
    assert not h[~keep].any() and not dgu[torch.cat([~keep, ~keep], dim=1)].any()
    return gu, dh, h, dgu


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("R,I", [(1, 1), (1, 8), (3, 7), (2, 16), (5, 129), (37, 1001), (64, 768), (300, 24), (1025, 40), (9, 4096), (2, 1 << 20),
                                 (3, (1 << 18) + 3), (70000, 8), (70001, 3)])
def test_values_and_gradients(dt, R, I):
    for p in (0.0, 0.1, 0.5, 1e-6, 0.9999):
        _check(R, I, p, dt, seed=R * 1000 + I, offset=3)


@pytest.mark.parametrize("seed,offset", [(0, 0), (2 ** 63 - 1, 2 ** 62 + 5), (-1, -1), (-2 ** 63, 2 ** 32), (1 << 32, (1 << 32) - 1)])
def test_seeds_and_offsets(seed, offset):
    _check(40, 72, 0.3, BF, seed=seed, offset=offset)


@pytest.mark.parametrize("dt", [BF, F16, F32])
def test_large_gates(dt):
    """Gates where exp(-g) or exp(g) leaves FP32."""
    _check(33, 64, 0.2, dt, std=40.0 if dt == F16 else 300.0)


def test_masked_places_may_hold_anything():
    g = torch.Generator().manual_seed(3)
    gu, dh = torch.randn((20, 64), generator=g), torch.randn((20, 32), generator=g)
    keep = ref.kept(20, 32, 0.5, 7, 1)
    both = torch.cat([keep, keep], dim=1)
    args = (0.5, _rng(7, 1))
    h, d = moe.moe_swiglu_dropout(gu.cuda(), *args), moe.moe_swiglu_dropout_bwd(dh.cuda(), gu.cuda(), *args)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(F32).min):
        gb, db = torch.where(both, gu, bad).cuda(), torch.where(keep, dh, bad).cuda()
        assert torch.equal(moe.moe_swiglu_dropout(gb, *args), h)
        assert torch.equal(moe.moe_swiglu_dropout_bwd(db, gb, *args), d)
    gu[0, 0] = float("nan")
    assert moe.moe_swiglu_dropout(gu.cuda()).isnan().sum() == 1          # kept: seen


def test_far_rows():
    """Over 2^31 elements: the last rows have the factors of their own row numbers."""
    R, I = 1_050_000, 1024
    gu = torch.ones((R, 2 * I), dtype=BF, device="cuda")
    h = moe.moe_swiglu_dropout(gu, 0.25, _rng(5, 6))
    one = float(moe.moe_swiglu_dropout(gu[:1])[0, 0]) * 65536 / (65536 - ref.threshold(0.25))
    for lo in (0, 524287, R - 3):
        n = min(3, R - lo)
        keep = ref.kept(n, I, 0.25, 5, 6, row0=lo)
        got = h[lo:lo + n].cpu()
        assert torch.equal(got != 0, keep) and (got[keep].float() - one).abs().max() <= 2.0 ** -8
    dgu = moe.moe_swiglu_dropout_bwd(h, gu, 0.25, _rng(5, 6), dgu=gu)
    assert torch.equal(dgu[-3:, :I].cpu() != 0, ref.kept(3, I, 0.25, 5, 6, row0=R - 3)) and dgu is gu


def test_streams_graphs_and_alignment():
    g = torch.Generator().manual_seed(4)
    gu, dh, rng = torch.randn((77, 208), generator=g).to(BF).cuda(), torch.randn((77, 104), generator=g).to(BF).cuda(), _rng(9, 0)
    h, d = moe.moe_swiglu_dropout(gu, 0.3, rng), moe.moe_swiglu_dropout_bwd(dh, gu, 0.3, rng)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h2, d2 = moe.moe_swiglu_dropout(gu, 0.3, rng, stream=side), moe.moe_swiglu_dropout_bwd(dh, gu, 0.3, rng, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, h2) and torch.equal(d, d2)
    # rows that do not start on 16 bytes, in place
    odd = lambda t: torch.empty(t.numel() + 1, dtype=BF, device="cuda")[1:].view(t.shape).copy_(t)  # noqa: E731
    og = odd(gu)
    assert torch.equal(moe.moe_swiglu_dropout(og, 0.3, rng), h) and torch.equal(moe.moe_swiglu_dropout_bwd(odd(dh), og, 0.3, rng, dgu=og), d)
    # a graph follows rng
    graph = torch.cuda.CUDAGraph()
    h3, d3 = torch.empty_like(h), torch.empty_like(d)
    with torch.cuda.graph(graph):
        moe.moe_swiglu_dropout(gu, 0.3, rng, h=h3)
        moe.moe_swiglu_dropout_bwd(dh, gu, 0.3, rng, dgu=d3)
        rng[1:].add_(1)
    seen = []
    for turn in range(3):
        graph.replay()
        assert torch.equal(h3.cpu() != 0, ref.kept(77, 104, 0.3, 9, turn) & (h3.cpu() != 0))
        assert torch.equal(h3, moe.moe_swiglu_dropout(gu, 0.3, _rng(9, turn))) and torch.equal(
            d3, moe.moe_swiglu_dropout_bwd(dh, gu, 0.3, _rng(9, turn)))
        seen.append(h3.clone())
    assert torch.equal(seen[0], h) and not torch.equal(seen[0] != 0, seen[1] != 0)
    assert moe.moe_swiglu_dropout(gu[:0], 0.3, rng).shape == (0, 104)


def test_autograd():
    """The backward pass drops what the forward pass dropped, though rng has moved on; against differences of the plain
    form: h^2 times the third derivative (below 4 along a unit direction, times |dh| sqrt(n)), and FP32."""
    g = torch.Generator().manual_seed(5)
    gu, dh, rng = torch.randn((12, 40), generator=g), torch.randn((12, 20), generator=g), _rng(3, 4)
    leaf = gu.cuda().requires_grad_()
    h = ragged.swiglu_dropout(leaf, 0.4, rng)
    rng.add_(1)
    (h * dh.cuda()).sum().backward()
    keep = ref.kept(12, 20, 0.4, 3, 4)
    f = lambda x: float((ref.swiglu(x, 0.4, keep)[0] * dh.double()).sum())  # noqa: E731
    for _ in range(8):
        d = torch.randn((12, 40), generator=g).double()
        d /= d.norm()
        diff = (f(gu.double() + 1e-4 * d) - f(gu.double() - 1e-4 * d)) / 2e-4
        assert abs(diff - float((leaf.grad.cpu().double() * d).sum())) < 1e-5
    assert ragged.swiglu_dropout(leaf).requires_grad


def test_capture_beside_an_eager_graph():
    leaf, rng = torch.randn((64, 32), device="cuda").requires_grad_(), _rng(1, 2)
    make = lambda: ragged.swiglu_dropout(leaf, 0.1, rng).sum()  # noqa: E731
    want, = torch.autograd.grad(make(), leaf)
    eager = make()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="another stream lives"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(make(), leaf)
    del eager
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad, = torch.autograd.grad(make(), leaf)
    graph.replay()
    assert torch.equal(grad, want)

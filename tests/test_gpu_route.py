"""The general router and its gradient against the plain forms in 64 bits: the same ids, weights and gradients within the
bounds of their FP32 steps."""
import gc

import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import route_ref as ref
from top_moe_expert_gb300 import ragged

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SOFT, SIG = moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID
INF = float("inf")


def _dev(t):
    return None if t is None else t.cuda()


def _weight_bound(l, w, E):
    """Relative error of a weight, in units of 2^-23: exp to 2 ulp and a rounded argument (|x| / 2), the sum over all
    experts (its terms by the fast exp, 2 + 1.7 |x| weighed to at most 2 + 1.7 ln E; E / 32 + 5 additions, twice the lanes
    for odd groups), a quotient and the scale."""
    l = torch.where(l > -INF, l, 0.0)
    span = (l.amax(dim=1, keepdim=True) - l.amin(dim=1, keepdim=True)).clamp(max=110)
    return (40 + E / 16 + span / 2) * 2.0 ** -23 * w.abs() + 1e-36


def _check(l, k, **kw):
    M, E = l.shape
    ids, w = moe.moe_route(l.cuda(), k, **{n: _dev(v) if n == "bias" else v for n, v in kw.items()})
    rids, rw, gap = ref.route(l, k, **kw)
    # 64-bit values that differ by a few of their own roundings have no order to test
    clear = gap > 1e-13 * (1 + (0 if kw.get("bias") is None else kw["bias"][kw["bias"].abs() < INF].abs().max().item()))
    # (a property of the inputs: sums of two scores d up and d down differ from two equal ones by d^2 = 4e-15 at d = 2^-24)
    assert clear.double().mean() > 0.5
    assert torch.equal(ids.cpu().long()[clear], rids[clear]), (ids.cpu()[clear] != rids[clear]).nonzero()[:4]
    w, rw = w.cpu().double()[clear], rw[clear]
    assert torch.equal(w.isnan(), rw.isnan())
    tol = _weight_bound(l.double()[clear], rw, E)
    off = (w - rw).abs() - tol
    assert not (off > 0).any(), (float(off.max()), w[off > 0][:4], rw[off > 0][:4])
    return ids, w


def _logits(M, E, dt, g, std=1.0):
    return (std * torch.randn((M, E), generator=g)).to(dt)


@pytest.mark.parametrize("dt", [F32, BF, F16])
@pytest.mark.parametrize("E,k,groups,topk_groups", [
    (1, 1, 1, 1), (2, 2, 1, 1), (7, 3, 1, 1), (8, 8, 8, 8), (32, 32, 1, 1), (64, 6, 1, 1), (100, 12, 1, 1), (128, 8, 1, 1),
    (160, 6, 8, 3), (256, 8, 8, 4), (256, 1, 1, 1), (320, 9, 5, 2), (384, 8, 2, 1), (512, 10, 16, 16), (512, 32, 1, 1),
    (1000, 8, 5, 2), (1003, 8, 17, 9), (1024, 12, 8, 1), (512, 12, 16, 4), (512, 20, 4, 1), (1024, 32, 32, 20), (1024, 4, 1, 1), (31, 31, 31, 31)])
def test_choice_and_weights(dt, E, k, groups, topk_groups):
    g = torch.Generator().manual_seed(E * 100 + k)
    for i, (score, with_bias, top, renorm) in enumerate([(SOFT, 0, 1, True), (SOFT, 0, 2, False), (SIG, 1, 2, True),
                                                         (SIG, 0, 2, False), (SOFT, 1, 1, False), (SIG, 1, 1, False)]):
        M = (1, 5, 33, 64, 7, 130)[(i + E) % 6]
        bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
        _check(_logits(M, E, dt, g), k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=top,
               renorm=renorm, scale=(1.0, 2.5)[i % 2])


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("groups,topk_groups,top", [(1, 1, 1), (8, 3, 1), (8, 4, 2)])
def test_nearly_equal_values(score, groups, topk_groups, top):
    """Logits a few units in the last place apart, and biases that almost make up for the difference: what decides is
    below the errors of 32 bits for most tokens."""
    g = torch.Generator().manual_seed(7 + groups + top)
    M, E = 300, 64
    l = torch.full((M, E), 0.625) + torch.randint(-3, 4, (M, E), generator=g) * 2.0 ** -24
    l[:, ::3] += 0.25
    bias = torch.zeros(E)
    bias[::3] = -float(torch.sigmoid(torch.tensor(0.875).double()) - torch.sigmoid(torch.tensor(0.625).double()))
    bias += torch.randint(-3, 4, (E,), generator=g) * 2.0 ** -27
    _check(l, 8, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=top)
    _check(l, 8, score=score, groups=groups, topk_groups=topk_groups, group_top=top)


@pytest.mark.parametrize("dt", [F32, BF])
def test_equal_values_go_by_index(dt):
    for E, groups, topk_groups in ((128, 1, 1), (256, 8, 3), (48, 3, 2), (1024, 1, 1)):
        l = torch.zeros((3, E), dtype=dt)
        l[1] = 2.0
        l[2, E // 2:] = 1.0
        for kw in (dict(), dict(score=SIG, bias=torch.zeros(E)), dict(score=SOFT, bias=torch.full((E,), -0.5))):
            for top in (1, 2):
                ids, _ = moe.moe_route(l.cuda(), 5, groups=groups, topk_groups=topk_groups, group_top=top,
                                       **{n: _dev(v) if n == "bias" else v for n, v in kw.items()})
                assert torch.equal(ids.cpu().long(), ref.route(l, 5, groups=groups, topk_groups=topk_groups, group_top=top, **kw)[0])


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [False, True])
def test_unavailable_experts(score, renorm, with_bias):
    """Masks by -inf that leave a part, one or none of a token's experts, groups without any, and the types' lowest value."""
    g = torch.Generator().manual_seed(11)
    E, k = 64, 6
    for dt in (F32, BF, F16):
        low = torch.finfo(dt).min
        l = _logits(12, E, dt, g)
        l[0] = -INF
        l[1, 1:] = -INF
        l[2, :60] = -INF
        l[3, 8:] = -INF
        l[4] = low
        l[5, 5:] = low
        l[6, 3:] = -INF
        l[6, :3] = low
        l[7, ::2] = -INF
        bias = None
        if with_bias:
            bias = 0.1 * torch.randn(E, generator=g)
            bias[10:20] = -INF
        for groups, topk_groups, top in ((1, 1, 1), (8, 3, 2), (8, 2, 1)):
            ids, w = _check(l, k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=top, renorm=renorm)
            assert (ids[0] == -1).all() and not w[0].any()
            assert ids[1].tolist() == [0] + [-1] * (k - 1) and not w[1, 1:].any()


def test_very_negative_sigmoids():
    """Scores that all vanish in FP32 still have a ratio."""
    g = torch.Generator().manual_seed(12)
    for at in (-50.0, -59.0, -61.0, -90.0, -1000.0, -3e38):
        l = torch.randn((9, 32), generator=g) + at
        ids, w = _check(l, 4, score=SIG)
        assert (w.sum(dim=1) - 1).abs().max() < 1e-6


def test_not_a_number():
    """NaN or +inf: the token's weights are NaN, its ids those of the others; other tokens have what they had."""
    g = torch.Generator().manual_seed(13)
    l = _logits(6, 40, F32, g)
    good = moe.moe_route(l.cuda(), 4, score=SIG, groups=4, topk_groups=2)
    l[1, 7], l[4, 3], l[5] = float("nan"), INF, float("nan")
    for kw in (dict(score=SIG, groups=4, topk_groups=2), dict(), dict(renorm=False), dict(score=SIG, bias=torch.zeros(40))):
        ids, w = _check(l, 4, **kw)
        assert w[[1, 4, 5]].isnan().all() and not w[[0, 2, 3]].isnan().any() and (ids[5] == -1).all()
        if kw.get("groups"):
            assert torch.equal(ids[[0, 2, 3]], good[0][[0, 2, 3]]) and torch.equal(w[[0, 2, 3]].float(), good[1].cpu()[[0, 2, 3]])
    bias = torch.zeros(40)
    bias[9] = float("nan")
    _check(l, 4, score=SIG, bias=bias)
    dl = moe.moe_route_bwd(torch.ones((6, 4), device="cuda"), l.cuda(), good[0], score=SIG).cpu()
    assert dl[[1, 4, 5]].isnan().all() and not dl[[0, 2, 3]].isnan().any()


def test_many_tokens():
    """A grid of many CTAs, an odd number of tokens; on the GPU's own sort as reference where the choice is by logit."""
    g = torch.Generator(device="cuda").manual_seed(14)
    l = torch.randn((70001, 128), generator=g, device="cuda")
    ids, w = moe.moe_route(l, 8)
    order = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :8]
    assert torch.equal(ids.long(), order)
    want, wr = moe.moe_topk_softmax(l, 8)
    assert torch.equal(ids, want) and (w - wr).abs().max() < 4e-6          # 13 units of 2^-23 each
    s = torch.sigmoid(l.double()) + 0.125
    ids, _ = moe.moe_route(l, 8, score=SIG, bias=torch.full((128,), 0.125, device="cuda"))
    assert torch.equal(ids.long(), torch.sort(s, dim=1, descending=True, stable=True)[1][:, :8])


@pytest.mark.parametrize("E,k,groups,topk_groups,top", [(64, 6, 1, 1, 1), (64, 16, 4, 3, 2), (128, 8, 1, 1, 1), (128, 4, 8, 2, 1),
                                                        (256, 8, 8, 4, 2), (256, 16, 16, 5, 2), (256, 1, 1, 1, 1), (256, 8, 2, 1, 1)])
def test_many_rows_agree_with_few(E, k, groups, topk_groups, top):
    """Calls of many tokens, which two of them share a warp's steps in, give each row what a call of few gives it: random
    logits, equal ones, nearly equal ones, masks that leave a part or nothing, NaN; an odd number of rows."""
    g = torch.Generator().manual_seed(E + k + groups)
    for dt in (F32, BF):
        few = _logits(150, E, dt, g)
        few[20:30] = (few[20:30] * 2).round() / 2
        few[30:40] = 0.625 + (torch.randint(-3, 4, (10, E), generator=g) * 2.0 ** -24)
        few[40] = -INF
        few[41:50, E // 3:] = -INF
        few[50:60, ::2] = -INF
        few[60, 1:] = -INF
        few[61, 3], few[62, 5] = float("nan"), INF
        few[63] = torch.finfo(dt).min
        few[64:70] = 1e-40 * torch.randint(-3, 4, (6, E), generator=g).float()
        few[70:80] = few[70:80] * 30
        few = few.to(dt)
        order = torch.cat([torch.arange(150), torch.randint(0, 150, (9001,), generator=g)])
        many = few[order].cuda()
        b = 0.05 * torch.randn(E, generator=g)
        off = b.clone()
        off[5:9] = -INF
        for kw in (dict(score=SIG, bias=b, scale=2.5), dict(score=SIG, bias=torch.zeros(E)), dict(score=SOFT, bias=off, renorm=False),
                   dict(score=SOFT, renorm=False), dict(score=SIG), dict()):
            kw = {n: _dev(v) if n == "bias" else v for n, v in kw.items()}
            kw.update(groups=groups, topk_groups=topk_groups, group_top=top)
            i1, w1 = moe.moe_route(few.cuda(), k, **kw)
            i2, w2 = moe.moe_route(many, k, **kw)
            assert torch.equal(i2, i1[order.cuda()])
            w1 = w1[order.cuda()]
            assert torch.equal(w1.isnan(), w2.isnan())
            span = 110.0
            assert ((w1 - w2).abs().nan_to_num() <= 2 * (40 + E / 16 + span / 2) * 2.0 ** -23 * w1.abs().nan_to_num() + 1e-36).all()


def test_subnormal_logits():
    """Maxima of subnormal logits, of either sign, are found."""
    l = torch.tensor([[1e-40, 3e-40, 2e-40, -1e-40], [-1e-40, -3e-40, -2e-40, -4e-40]]).repeat(1, 8)
    for dt in (F32, BF):
        x = l.to(dt)
        for kw in (dict(), dict(groups=4, topk_groups=2), dict(groups=4, topk_groups=2, group_top=2, score=SIG)):
            assert torch.equal(moe.moe_route(x.cuda(), 3, **kw)[0].cpu().long(), ref.route(x, 3, **kw)[0])


def test_load_is_added():
    g = torch.Generator().manual_seed(15)
    l = _logits(1000, 48, BF, g)
    l[3] = -INF
    load = torch.arange(48, dtype=torch.int32, device="cuda")
    ids, _ = moe.moe_route(l.cuda(), 5, score=SIG, bias=torch.zeros(48, device="cuda"), load=load)
    v = ids.cpu().long().flatten()
    assert torch.equal(load.cpu().long(), torch.arange(48) + torch.bincount(v[v >= 0], minlength=48))


# ---------------------------------------------------------------- gradient

def _grad_bound(dl, mag, l, E, dt):
    """In units of 2^-23 of the terms' magnitudes: the weights' bound, sums over the slots (32 additions and 5), the same
    for the scores of all experts, products; then one rounding to the type."""
    l = torch.where(l > -INF, l, 0.0)
    span = (l.amax(dim=1, keepdim=True) - l.amin(dim=1, keepdim=True)).clamp(max=110)
    tol = (100 + E / 8 + 2 * span) * 2.0 ** -23 * mag + 1e-36
    if dt != F32:
        tol = tol + torch.finfo(dt).eps / 2 * (dl.abs() + tol) + (2.0 ** -25 if dt == F16 else 0.0)
    return tol


@pytest.mark.parametrize("dt", [F32, BF, F16])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (5, 9, 4), (33, 128, 8), (130, 256, 8), (7, 1000, 12), (3, 1024, 32), (64, 31, 31)])
def test_gradient(dt, score, renorm, M, E, k):
    g = torch.Generator().manual_seed(M + E + k)
    l, dw = _logits(M, E, dt, g), torch.randn((M, k), generator=g)
    if E > 8:
        l[0, 2:8] = -INF
    ids, _ = moe.moe_route(l.cuda(), k, score=score, renorm=renorm, scale=2.5)
    dl = moe.moe_route_bwd(dw.cuda(), l.cuda(), ids, score=score, renorm=renorm, scale=2.5)
    assert dl.dtype == dt
    want, mag = ref.route_bwd(dw, l, ids.cpu().long(), score, renorm, 2.5)
    off = (dl.cpu().double() - want).abs() - _grad_bound(want, mag, l.double(), E, dt)
    assert not (off > 0).any(), float(off.max())
    assert not dl.cpu()[l == -INF].any()


@pytest.mark.parametrize("E", [64, 100, 128, 256, 512])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_masked_rows(E, score, renorm):
    """A token without any expert gets zeros, beside others, one expert alone its own gradient."""
    g = torch.Generator().manual_seed(E)
    for dt in (F32, BF):
        l, dw = _logits(7, E, dt, g), torch.randn((7, 4), generator=g)
        l[1] = l[6] = -INF
        l[3, 1:] = -INF
        l[4] = torch.finfo(dt).min
        ids, _ = moe.moe_route(l.cuda(), 4, score=score, renorm=renorm)
        dl = moe.moe_route_bwd(dw.cuda(), l.cuda(), ids, score=score, renorm=renorm).cpu()
        assert not dl[[1, 6]].any() and torch.isfinite(dl).all()
        want, mag = ref.route_bwd(dw, l, ids.cpu().long(), score, renorm, 1.0)
        off = (dl.double() - want).abs() - _grad_bound(want, mag, l.double(), E, dt)
        assert not (off[[0, 2, 3, 4, 5]] > 0).any(), float(off.max())


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_given_ids(score, renorm):
    """Ids that no choice gave: the same expert several times, none at all, ids out of range (whose dw is not read)."""
    g = torch.Generator().manual_seed(21)
    l, dw = torch.randn((6, 20), generator=g), torch.randn((6, 5), generator=g)
    ids = torch.tensor([[3, 3, 3, 3, 3], [1, 2, 1, 2, 19], [-1] * 5, [0, -7, 20, 2 ** 31 - 1, 4], [5, 5, -1, 6, 6], [0, 1, 2, 3, 4]])
    nan = torch.where((ids < 0) | (ids > 19), float("nan"), dw)
    dl = moe.moe_route_bwd(nan.cuda(), l.cuda(), ids.int().cuda(), score=score, renorm=renorm).cpu().double()
    clean = torch.where((ids < 0) | (ids > 19), -1, ids)
    want, mag = ref.route_bwd(dw, l, clean, score, renorm, 1.0)
    off = (dl - want).abs() - _grad_bound(want, mag, l.double(), 20, F32)
    assert not (off > 0).any(), float(off.max())
    assert not dl[2].any()


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Directional differences of the plain weights at the chosen ids: h^2 of the third derivative (below 20 sum |dw|
    along a unit direction) and the kernel's own 1e-5."""
    g = torch.Generator().manual_seed(22)
    l, dw = torch.randn((20, 32), generator=g), torch.randn((20, 4), generator=g)
    leaf = l.cuda().requires_grad_()
    ids, w = ragged.route(leaf, 4, score=score, renorm=renorm, groups=4, topk_groups=2, scale=2.0)
    (w * dw.cuda()).sum().backward()
    f = lambda x: float((ref.weights(x, ids.cpu().long(), score, renorm, 2.0) * dw.double()).sum())  # noqa: E731
    for _ in range(8):
        d = torch.randn((20, 32), generator=g).double()
        d /= d.norm()
        h = 1e-4
        diff = (f(l.double() + h * d) - f(l.double() - h * d)) / (2 * h)
        assert abs(diff - float((leaf.grad.cpu().double() * d).sum())) < 1e-5 + 40 * float(dw.abs().sum()) * h * h


def test_two_calls_at_once_share_a_load():
    """Whole numbers added from two streams at a time."""
    g = torch.Generator().manual_seed(31)
    l = _logits(20000, 64, BF, g).cuda()
    load, side = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [moe.moe_route(l, 6, load=load, stream=s) for s in (None, side) * 3]
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs)
    assert torch.equal(load.long(), 6 * torch.bincount(outs[0][0].flatten().long(), minlength=64))


# ---------------------------------------------------------------- streams, graphs, repeatability

def test_streams_graphs_and_outputs():
    g = torch.Generator().manual_seed(23)
    l, bias = _logits(513, 256, BF, g).cuda(), 0.1 * torch.randn(256, generator=g).cuda()
    kw = dict(score=SIG, bias=bias, groups=8, topk_groups=4, group_top=2, scale=2.5)
    ids, w = moe.moe_route(l, 8, **kw)
    dw = torch.randn((513, 8), generator=g).cuda()
    dl = moe.moe_route_bwd(dw, l, ids, score=SIG, scale=2.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i2, w2 = moe.moe_route(l, 8, stream=side, **kw)
    d2 = moe.moe_route_bwd(dw, l, i2, score=SIG, scale=2.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(i2, ids) and torch.equal(w2, w) and torch.equal(d2, dl)
    i3, w3, d3, load = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(dl), torch.zeros(256, dtype=torch.int32, device="cuda")
    x = l.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        load.zero_()
        moe.moe_route(x, 8, topk_ids=i3, topk_w=w3, load=load, **kw)
        moe.moe_route_bwd(dw, x, i3, score=SIG, scale=2.5, dlogits=d3)
    for turn in range(3):
        x.copy_(l.roll(turn, 0))
        graph.replay()
        want = moe.moe_route(x, 8, **kw)
        assert torch.equal(i3, want[0]) and torch.equal(w3, want[1])
        assert torch.equal(d3, moe.moe_route_bwd(dw, x, i3, score=SIG, scale=2.5))
        assert torch.equal(load.long(), torch.bincount(i3.flatten().long(), minlength=256))
    # two at once, and a row's result beside other rows
    with torch.cuda.stream(side):
        a = moe.moe_route(l, 8, **kw)
    b = moe.moe_route(l[100:101].contiguous(), 8, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a[0], ids) and torch.equal(b[0], ids[100:101]) and torch.equal(b[1], w[100:101])
    # rows that do not start on 16 bytes
    odd = torch.empty(513 * 256 + 1, dtype=BF, device="cuda")[1:].view(513, 256).copy_(l)
    c = moe.moe_route(odd, 8, **kw)
    assert torch.equal(c[0], ids) and torch.equal(c[1], w) and torch.equal(moe.moe_route_bwd(dw, odd, ids, score=SIG, scale=2.5), dl)
    empty = moe.moe_route(l[:0], 8, **kw)
    assert empty[0].shape == (0, 8) and moe.moe_route_bwd(dw[:0], l[:0], empty[0]).shape == (0, 256)


def test_capture_beside_an_eager_graph():
    leaf = torch.randn((64, 32), device="cuda").requires_grad_()
    make = lambda: (ragged.route(leaf, 4)[1] * torch.arange(4, device="cuda")).sum()  # noqa: E731
    want, = torch.autograd.grad(make(), leaf)
    eager = make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="another stream lives"):
        with torch.cuda.graph(graph):
            torch.autograd.grad(make(), leaf)
    del eager
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad, = torch.autograd.grad(make(), leaf)
    graph.replay()
    assert torch.equal(grad, want)

"""The general router at the ends of its arguments' ranges, against the plain forms in 64 bits."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import route_ref as ref
from tests.test_gpu_route import _weight_bound

pytestmark = pytest.mark.gpu

F32 = torch.float32
SOFT, SIG = moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID
TOP = torch.finfo(F32).max


def _biases(E, groups, g):
    """Biases with one large finite value at: all groups but one, all but two experts, a share of the experts."""
    n = E // groups
    for at in (-TOP, TOP, -2e38, 2e38, -1e9, 1e9):
        for which in range(5):
            b = 0.1 * torch.randn(E, generator=g)
            if which == 0:
                b[n:] = at                                            # the first group is left
            elif which == 1:
                b[:(groups - 1) * n] = at                             # the last one
            elif which == 2:
                b[torch.randperm(E, generator=g)[2:]] = at
            elif which == 3:
                b[torch.rand(E, generator=g) < 0.5] = at
            else:
                b[:] = at
            yield b


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,k,groups,topk_groups", [(64, 12, 8, 2), (8, 4, 4, 2), (256, 32, 8, 4), (160, 30, 8, 3), (48, 20, 3, 2),
                                                    (64, 6, 1, 1)])
def test_biases_of_any_finite_size(score, top, E, k, groups, topk_groups):
    """Only -inf takes an expert out: a finite bias, the type's lowest value among them, puts it behind the others, in the
    order of the sums in binary64.  (Values that differ there at all differ by 1e-7 beside 1e9, and by what the gap says
    among the others; the score's own rounding in binary64 is 1e-16.)"""
    g = torch.Generator().manual_seed(E + k + top)
    l = torch.randn((7, E), generator=g)
    for i, b in enumerate(_biases(E, groups, g)):
        kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=top, renorm=i % 2 == 0)
        ids, w = moe.moe_route(l.cuda(), k, bias=b.cuda(), **kw)
        rids, rw, gap = ref.route(l, k, bias=b, **kw)
        clear = gap > 1e-12
        assert clear.double().mean() > 0.5
        assert (rids >= 0).all()
        assert torch.equal(ids.cpu().long()[clear], rids[clear]), (i, ids.cpu()[clear][:2], rids[clear][:2])
        off = (w.cpu().double() - rw).abs() - _weight_bound(l.double(), rw, E)
        assert not (off[clear] > 0).any(), (i, float(off[clear].max()))


def test_most_rows_there_can_be():
    """M * k just below 2^31: a row for every count of 32 bits, in both directions.  Sigmoid of 0: w = 1/2, dl = dw / 4."""
    M = 2 ** 31 - 1
    l = torch.zeros((M, 1), dtype=torch.bfloat16, device="cuda")
    load = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w = moe.moe_route(l, 1, score=SIG, renorm=False, load=load)
    assert load.item() == M and not ids.any() and (w == 0.5).all()
    del w
    dw = torch.ones((M, 1), device="cuda")
    dl = torch.full((M, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_route_bwd(dw, l, ids, score=SIG, renorm=False, dlogits=dl)
    assert (dl == 0.25).all()


def _hard_rows(E, g):
    """Rows whose choice binary32 does not settle, beside ordinary ones: equal logits (more candidates than a warp's lanes
    hold), nearly equal ones, masks, NaN."""
    l = torch.randn((90, E), generator=g)
    l[0:20] = 0.0
    l[20:40] = 0.625 + torch.randint(-3, 4, (20, E), generator=g) * 2.0 ** -24
    l[40:45] = -float("inf")
    l[45:50, E // 3:] = -float("inf")
    l[50:55] = -TOP
    l[55, 3] = float("nan")
    l[56:60, 1:] = -float("inf")
    return l


HARD = [dict(), dict(score=SOFT, bias=0.0), dict(score=SIG, bias=0.0), dict(score=SOFT, renorm=False),
        dict(score=SOFT, bias=0.0, groups=8, topk_groups=3, group_top=2), dict(score=SIG, bias=0.0, groups=8, topk_groups=3, group_top=2),
        dict(score=SOFT, groups=4, topk_groups=2, group_top=2), dict(score=SIG, groups=4, topk_groups=2, group_top=1)]


@pytest.mark.parametrize("E,k", [(128, 8), (160, 6), (384, 8), (1024, 32)])
@pytest.mark.parametrize("how", HARD, ids=str)
def test_load_counts_every_slot_once(E, k, how):
    """Tokens whose choice is settled in a second pass are counted there alone."""
    g = torch.Generator().manual_seed(E + k)
    l = _hard_rows(E, g)[torch.randint(0, 90, (6001,), generator=g)].cuda()
    how = dict(how)
    if "bias" in how:
        how["bias"] = (torch.randint(-3, 4, (E,), generator=g) * 2.0 ** -27).cuda()
    load = torch.full((E,), 5, dtype=torch.int32, device="cuda")
    ids, _ = moe.moe_route(l, k, load=load, **how)
    v = ids.long().flatten()
    assert ((v >= -1) & (v < E)).all()
    assert torch.equal(load.long(), 5 + torch.bincount(v[v >= 0], minlength=E))


@pytest.mark.parametrize("E,k", [(128, 8), (160, 6), (384, 8), (1024, 32)])
@pytest.mark.parametrize("how", HARD, ids=str)
def test_a_row_has_the_same_bits_beside_others(E, k, how):
    g = torch.Generator().manual_seed(E + k + 1)
    few = _hard_rows(E, g)
    order = torch.cat([torch.arange(90), torch.randint(0, 90, (9001,), generator=g)]).cuda()
    how = dict(how)
    if "bias" in how:
        how["bias"] = (torch.randint(-3, 4, (E,), generator=g) * 2.0 ** -27).cuda()
    few = few.cuda()
    i1, w1 = moe.moe_route(few, k, **how)
    i2, w2 = moe.moe_route(few[order], k, **how)
    assert torch.equal(i2, i1[order]) and torch.equal(w2.view(torch.int32), w1[order].view(torch.int32))
    for r in (0, 25, 42, 47, 55, 57, 70):
        i, w = moe.moe_route(few[r:r + 1].contiguous(), k, **how)
        assert torch.equal(i[0], i1[r]) and torch.equal(w[0].view(torch.int32), w1[r].view(torch.int32))


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("E,groups,topk_groups", [(2, 1, 1), (6, 1, 1), (32, 1, 1), (40, 1, 1), (60, 4, 3), (64, 8, 5), (256, 16, 3)])
def test_few_distinct_values(score, E, groups, topk_groups):
    """Runs of experts with the same logit and bias that reach past the last slot, and others, lower or higher by less than
    binary32 tells apart, behind them: logits a few units in the last place apart, sigmoids near 1 and scores near 0,
    biases that take the scores' bits away.  (Differences in binary64: 1e-8 of scores near 1/2; 1e-9 of sigmoids at 17;
    beside a bias of 10^4 they are those of scores 0.1 apart.)"""
    g = torch.Generator().manual_seed(E)
    for base, step, shift in ((0.625, 2.0 ** -24, 0.0), (17.0, 0.25, 0.0), (-22.0, 0.25, 0.0), (0.0, 0.5, 1e4), (0.0, 0.5, -1e4)):
        if score == SOFT and base == 17.0:
            continue
        for kinds in (2, 3):
            l = base + step * torch.randint(0, kinds, (60, E), generator=g).float()
            l[::4] = base
            l[::4, -1] += step                                         # the best one is the last
            if base == -22.0 and score == SOFT:
                l[:, 0] = 0.0                                          # the others' scores are near 0
            b = torch.full((E,), shift)
            if kinds == 3:
                b[torch.rand(E, generator=g) < 0.3] += 0.25
            for k in (1, 2, 3, 8, 16):
                if k > topk_groups * (E // groups):
                    continue
                kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=1 + k % 2)
                ids, w = moe.moe_route(l.cuda(), k, bias=b.cuda(), **kw)
                rids, rw, gap = ref.route(l, k, bias=b, **kw)
                clear = gap > 1e-13 * (1 + abs(shift))
                assert clear.double().mean() > 0.5
                assert torch.equal(ids.cpu().long()[clear], rids[clear]), (base, shift, k, (ids.cpu() != rids).any(dim=1).nonzero()[:4])
                off = (w.cpu().double() - rw).abs() - _weight_bound(l.double(), rw, E)
                assert not (off[clear] > 0).any(), (base, shift, k, float(off[clear].max()))


def test_weights_of_tiny_sigmoids():
    """Renormalised weights keep their relative accuracy where some of the chosen sigmoids are below FP32's normal range
    and their sum is tiny too; the gradient's terms likewise.  All experts are chosen.  (4e-37: scores below 2^-126 are off
    by 2 units of 2^-149, times the scale 2 over a sum of at least e^-18; in the gradient times |dw| and its mean, below 10
    together.)"""
    g = torch.Generator().manual_seed(5)
    top = torch.cat([torch.arange(-64.0, -10.0, 0.5), torch.tensor([0.0, 5.0])])
    l = top[:, None] - 85.0 * torch.rand((top.numel(), 32), generator=g)
    l[:, 0] = top
    ids, w = moe.moe_route(l.cuda(), 32, score=SIG, scale=2.0)
    rids, rw, _ = ref.route(l, 32, score=SIG, scale=2.0)
    assert torch.equal(ids.cpu().long(), rids)
    # the chosen logits span up to 85: exp of such an argument is off by 85 / 2 units, by itself 40 more with the sum
    off = (w.cpu().double() - rw).abs() - (40 + 32 / 16 + 85 / 2) * 2.0 ** -23 * rw - 4e-37
    assert not (off > 0).any(), (float(off.max()), (off > 0).nonzero()[:4])
    dw = torch.randn((top.numel(), 32), generator=g)
    dl = moe.moe_route_bwd(dw.cuda(), l.cuda(), ids, score=SIG, scale=2.0).cpu().double()
    want, mag = ref.route_bwd(dw, l, rids, SIG, True, 2.0)
    off = (dl - want).abs() - (100 + 32 / 8 + 2 * 85) * 2.0 ** -23 * mag - 4e-36
    assert not (off > 0).any(), float(off.max())

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

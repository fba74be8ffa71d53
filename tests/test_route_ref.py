"""The plain forms that the router, the dropout and their gradients are tested against (CPU)."""
import numpy as np
import pytest
import torch

from tests import route_ref as ref


def test_philox_known_answers():
    """The published answers of the generator's authors."""
    for c, k, want in (([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
                       ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
                       ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
                        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert ref.philox(np.array(c, dtype=np.uint64), k).tolist() == want


def test_kept_share_and_independence():
    """Over 2^20 elements the share is within five standard deviations of p, and neighbours agree no more than chance."""
    for p in (0.1, 0.5):
        k = ref.kept(1024, 1024, p, 12345, 6).double()
        n = k.numel()
        assert abs(float(k.mean()) - (1 - p)) < 5 * (p * (1 - p) / n) ** 0.5
        for a, b in ((k[:, 1:], k[:, :-1]), (k[1:], k[:-1]), (k[:, 8:], k[:, :-8])):
            both = ((a - a.mean()) * (b - b.mean())).mean() / (p * (1 - p))
            assert abs(float(both)) < 5 / n ** 0.5 * 1.01


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(1)
    l, dw = torch.randn((5, 9), generator=g).double(), torch.randn((5, 3), generator=g).double()
    ids = ref.route(l, 3, score)[0]
    ids[2, 1] = -1
    dl, mag = ref.route_bwd(dw, l, ids, score, renorm, 2.5)
    f = lambda x: float((ref.weights(x, ids, score, renorm, 2.5) * dw).sum())  # noqa: E731
    for t in range(5):
        for e in range(9):
            d = torch.zeros_like(l)
            d[t, e] = 1e-6
            assert abs((f(l + d) - f(l - d)) / 2e-6 - float(dl[t, e])) < 1e-8       # h^2 and 2^-53 / h
            assert abs(float(dl[t, e])) <= float(mag[t, e]) * (1 + 1e-12)


def test_swiglu_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    gu, dh = torch.randn((4, 12), generator=g).double(), torch.randn((4, 6), generator=g).double()
    keep = ref.kept(4, 6, 0.3, 5, 9)
    dgu, mag = ref.swiglu(gu, 0.3, keep)[1](dh)
    f = lambda x: float((ref.swiglu(x, 0.3, keep)[0] * dh).sum())  # noqa: E731
    for r in range(4):
        for i in range(12):
            d = torch.zeros_like(gu)
            d[r, i] = 1e-6
            assert abs((f(gu + d) - f(gu - d)) / 2e-6 - float(dgu[r, i])) < 1e-8
    assert (dgu.abs() <= mag * (1 + 1e-12)).all()


def test_route_plain_form_cases():
    """Groups by their best, by their two best, ties by index, unavailable experts."""
    l = torch.tensor([[1.0, 5.0, 3.0, 3.0, 4.0, 0.0]])
    assert ref.route(l, 2)[0].tolist() == [[1, 4]]
    assert ref.route(l, 3)[0].tolist() == [[1, 4, 2]]
    assert ref.route(l, 2, groups=3, topk_groups=1)[0].tolist() == [[1, 0]]
    assert ref.route(l, 2, groups=3, topk_groups=2)[0].tolist() == [[1, 4]]
    assert ref.route(l, 2, score=1, groups=3, topk_groups=1, group_top=2)[0].tolist() == [[2, 3]]
    b = torch.tensor([0.0, -ref.INF, 0.0, 0.0, 0.0, 1.0])
    ids, w, _ = ref.route(l, 4, score=1, bias=b, renorm=False)
    assert ids.tolist() == [[5, 4, 2, 3]] and w[0, 0] == 0.5
    l[0, :4] = -ref.INF
    ids, w, _ = ref.route(l, 3)
    assert ids.tolist() == [[4, 5, -1]] and w[0, 2] == 0 and abs(float(w.sum()) - 1) < 1e-15

"""A backward pass captured beside a living eager graph of the same leaves: an exception, and a working context after it,
for leaves that the layer gathers, weighs with or gets cast."""
import gc

import pytest
import torch

from top_moe_expert_gb300 import ragged

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _check(make, leaf):
    want, = torch.autograd.grad(make(leaf).sum(), leaf)
    eager = make(leaf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="another stream lives"):
        with torch.cuda.graph(graph):
            y = make(leaf).sum()
            torch.autograd.grad(y, leaf)
    del eager, y
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad, = torch.autograd.grad(make(leaf).sum(), leaf)
    graph.replay()
    assert torch.equal(grad, want)


@pytest.mark.parametrize("what", ["x", "topk_w", "master"])
def test_capture_beside_an_eager_graph(what):
    g = torch.Generator().manual_seed(4)
    M, E, k, d, I = 20, 4, 2, 64, 32
    x = torch.randn((M, d), generator=g).to(BF).cuda()
    w13 = torch.randn((E, 2 * I, d), generator=g).mul_(d ** -0.5).cuda()
    w2 = torch.randn((E, d, I), generator=g).mul_(I ** -0.5).to(BF).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(M)]).to(torch.int32).cuda()
    w = torch.rand((M, k), generator=g).cuda()
    if what == "x":
        _check(lambda t: ragged.expert_layer(t, ids, w, w13.bfloat16(), w2), x.requires_grad_())
    elif what == "topk_w":
        _check(lambda t: ragged.expert_layer(x, ids, t, w13.bfloat16(), w2), w.requires_grad_())
    else:
        _check(lambda t: ragged.expert_layer(x, ids, w, t.bfloat16(), w2), w13.requires_grad_())

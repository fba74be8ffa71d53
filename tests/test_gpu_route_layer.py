"""The new operators together, as they are used: a trained router with expert dropout, and a router before 4-bit experts."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as rr
from tests import route_ref as ref
from top_moe_expert_gb300 import ragged

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SIG = moe.MOE_SCORE_SIGMOID


def _layer(x, ids, w, w13, w2, groups, p, rng):
    """The layer in 64 bits on the CPU, differentiable; h and gate/up rounded to bf16 as the layer does."""
    E, k = w13.shape[0], ids.shape[1]
    row, R = groups.row.cpu(), ids.numel()
    xr = x[groups.token.cpu()]
    off = groups.offsets.tolist()
    gu = torch.cat([xr[off[e]:off[e + 1]] @ w13[e].T for e in range(E)] + [torch.zeros((R - off[-1], w13.shape[1]), dtype=x.dtype)])
    gu = gu + (gu.bfloat16().double() - gu).detach()
    g, u = gu.chunk(2, dim=1)
    h = torch.nn.functional.silu(g) * u
    if p:
        h = h * ref.kept(R, h.shape[1], p, *rng) * (65536.0 / (65536 - ref.threshold(p)))
    h = h + (h.bfloat16().double() - h).detach()
    y = torch.cat([h[off[e]:off[e + 1]] @ w2[e].T for e in range(E)] + [torch.zeros((R - off[-1], w2.shape[1]), dtype=x.dtype)])
    y = y + (y.bfloat16().double() - y).detach()
    return (y[row.clamp(max=R - 1)] * torch.where(row < R, w, 0.0).unsqueeze(2)).sum(dim=1)


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_trained_router_and_experts(p):
    """One training step: every gradient within a few bf16 roundings (2^-8 of its norm; three products in a row, each of
    them and their operands rounded: 8 of them) of the 64-bit layer's."""
    g = torch.Generator().manual_seed(1)
    M, E, k, d, I = 60, 16, 4, 64, 48
    x = torch.randn((M, d), generator=g).to(BF)
    w13, w2 = (0.125 * torch.randn((E, 2 * I, d), generator=g)).to(BF), (0.14 * torch.randn((E, d, I), generator=g)).to(BF)
    wr, bias = 0.125 * torch.randn((d, E), generator=g), 0.05 * torch.randn(E, generator=g)
    dy = torch.randn((M, d), generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, w13, w2, wr)]
    lx, l13, l2, lr = leaves
    load, rng = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.tensor([5, 6], device="cuda")
    logits = lx.float() @ lr
    ids, w = ragged.route(logits, k, score=SIG, bias=bias.cuda(), groups=4, topk_groups=2, group_top=2, scale=2.5, load=load)
    y = ragged.expert_layer(lx, ids, w, l13, l2, dropout=p, rng=rng)
    rng.add_(1)
    (y * dy.cuda()).sum().backward()
    groups = ragged.group_routes(ids, E)
    cl = [t.double().requires_grad_() for t in (x, w13, w2, wr)]
    cw = ref.weights(cl[0] @ cl[3], ids.cpu().long(), SIG, True, 2.5)
    want = _layer(cl[0], ids.cpu(), cw, cl[1], cl[2], groups, p, (5, 6))
    (want * dy.double()).sum().backward()
    assert (y.detach().cpu().double() - want.detach()).norm() <= 8 * 2.0 ** -8 * want.detach().norm()
    for a, b in zip(leaves, cl):
        assert (a.grad.cpu().double() - b.grad).norm() <= 8 * 2.0 ** -8 * b.grad.norm()
    assert torch.equal(load.long(), torch.bincount(ids.flatten().long(), minlength=E))


def test_dropout_needs_rng_and_none_changes_nothing():
    g = torch.Generator().manual_seed(2)
    M, E, k, d, I = 20, 4, 2, 64, 32
    x, w13, w2 = (torch.randn(s, generator=g).mul_(0.1).to(BF).cuda() for s in ((M, d), (E, 2 * I, d), (E, d, I)))
    ids, w = moe.moe_route(torch.randn((M, E), generator=g).cuda(), k)
    with pytest.raises(ValueError, match="rng"):
        ragged.expert_layer(x, ids, w, w13, w2, dropout=0.1)
    a = ragged.expert_layer(x, ids, w, w13, w2)
    assert torch.equal(a, ragged.expert_layer(x, ids, w, w13, w2, dropout=0.0, rng=torch.zeros(2, dtype=torch.int64, device="cuda")))


def test_captured_step_draws_anew():
    """A captured forward and backward pass with the offset moved on in the graph: each replay drops other elements."""
    g = torch.Generator().manual_seed(3)
    M, E, k, d, I = 32, 8, 2, 64, 32
    x, w13, w2 = (torch.randn(s, generator=g).mul_(0.2).to(BF).cuda() for s in ((M, d), (E, 2 * I, d), (E, d, I)))
    logits, rng = torch.randn((M, E), generator=g).cuda().requires_grad_(), torch.tensor([1, 0], device="cuda")

    def step(r):
        ids, w = ragged.route(logits, k, renorm=False)
        y = ragged.expert_layer(x, ids, w, w13, w2, dropout=0.5, rng=r)
        return y, torch.autograd.grad(y.square().sum(), logits)[0]

    want = [step(torch.tensor([1, i], device="cuda")) for i in range(3)]
    torch.cuda.synchronize()
    want = [(y.detach().clone(), dl.clone()) for y, dl in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dl = step(rng)
        rng[1:].add_(1)
    for i in range(3):
        graph.replay()
        assert torch.equal(y, want[i][0]) and torch.equal(dl, want[i][1])
    assert not torch.equal(want[0][0], want[1][0])


@pytest.mark.parametrize("M", [1, 40])
def test_router_before_awq_experts(M):
    """The layer's products in 4 bits by hand (moe_grouped_mm_awq, the activation without dropout) against 64 bits on the
    same weights, and the fused decode path fed by the same router."""
    g = torch.Generator().manual_seed(4)
    E, k, d, I = 16, 4, 1024, 256
    q13, q2 = ref.awq_random(E, 2 * I, d, g), ref.awq_random(E, d, I, g)
    w13, w2 = (moe.Weights(moe.MOE_W_AWQ4, *(t.cuda() for t in q)) for q in (q13, q2))
    x = torch.randn((M, d), generator=g).to(F16).cuda()
    logits = torch.randn((M, E), generator=g).to(BF).cuda()
    ids, w = moe.moe_route(logits, k, score=SIG, bias=torch.zeros(E, device="cuda"), groups=4, topk_groups=2, group_top=2, scale=2.5)
    groups = ragged.group_routes(ids, E)
    gu = moe.moe_grouped_mm_awq(x[groups.token], w13, groups.offsets)
    h = moe.moe_swiglu_dropout(gu)
    rows = moe.moe_grouped_mm_awq(h, w2, groups.offsets, out_dtype=F32)
    y = (rows[groups.row] * w.unsqueeze(2)).sum(dim=1)
    sizes = torch.diff(groups.offsets).tolist()
    vgu, _ = rr.mm(x[groups.token].cpu(), ref.awq_values(*q13), sizes)
    vh, _ = ref.swiglu(vgu, 0.0, torch.ones((M * k, I), dtype=torch.bool))
    vr, _ = rr.mm(vh, ref.awq_values(*q2), sizes)
    want = (vr[groups.row.cpu()] * w.cpu().double().unsqueeze(2)).sum(dim=1)
    assert (y.cpu().double() - want).norm() <= 4 * 2.0 ** -11 * want.norm()      # gate/up, h and their products in fp16
    z = moe.moe_ffn_decode(x, ids, w, w13, w2, out_dtype=F32)
    assert (z.cpu().double() - want).norm() <= 4 * 2.0 ** -11 * want.norm()

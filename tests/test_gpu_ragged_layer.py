"""The ragged expert layer (top_moe_expert_gb300.ragged): routing to groups, its outputs and gradients against a 64-bit
layer, the 4-bit layer against a 64-bit layer on the same codes, and a captured training step."""
import gc

import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as ref
from top_moe_expert_gb300 import ragged

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _layer64(x, ids, w, w13, w2, h_round=lambda h: h):
    """The layer in float64, by token and slot; leaves of autograd where they require gradients."""
    E = w13.shape[0]
    ys = []
    for t in range(x.shape[0]):
        y = torch.zeros(w2.shape[1], dtype=torch.float64)
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < E:
                g, u = (w13[e] @ x[t]).chunk(2)
                y = y + w[t, j] * (w2[e] @ h_round(torch.nn.functional.silu(g) * u))
        ys.append(y)
    return torch.stack(ys)


def test_group_routes():
    g = torch.Generator().manual_seed(1)
    M, k, E = 37, 3, 11
    ids = torch.randint(-1, E + 1, (M, k), generator=g, dtype=torch.int32)     # -1 and E are invalid
    gr = ragged.group_routes(ids.cuda(), E)
    valid = (ids >= 0) & (ids < E)
    counts = [int((ids[valid] == e).sum()) for e in range(E)]
    assert gr.offsets.tolist() == ref.offsets_of(counts).tolist() and gr.offsets.dtype == torch.int32
    flat = ids.flatten().tolist()
    order = sorted((i for i in range(M * k) if 0 <= flat[i] < E), key=lambda i: (flat[i], i))
    assert gr.token[:len(order)].tolist() == [i // k for i in order]
    row = gr.row.flatten().tolist()
    assert all(row[i] == r for r, i in enumerate(order)) and all(row[i] == M * k for i in range(M * k) if not 0 <= flat[i] < E)


def _problem(M, E, k, d, I, seed, invalid):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, d), generator=g).to(BF)
    w13 = (torch.randn((E, 2 * I, d), generator=g) * d ** -0.5).to(BF)
    w2 = (torch.randn((E, d, I), generator=g) * I ** -0.5).to(BF)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(M)]).to(torch.int32)
    if invalid:
        ids[::5, 0], ids[3] = -1, E
    w = torch.rand((M, k), generator=g)
    return x, ids, w, w13, w2


@pytest.mark.parametrize("M,E,k,d,I,invalid", [(1, 4, 2, 64, 32, False), (23, 6, 3, 136, 72, True), (70, 5, 2, 128, 64, False)])
def test_layer_and_gradients(M, E, k, d, I, invalid):
    x, ids, w, w13, w2 = _problem(M, E, k, d, I, M, invalid)
    leaves = [t.cuda().requires_grad_() for t in (x, w, w13, w2)]
    y = ragged.expert_layer(leaves[0], ids.cuda(), *leaves[1:])
    dy = torch.randn((M, d), generator=torch.Generator().manual_seed(9))
    (y * dy.cuda()).sum().backward()
    want = [t.double().requires_grad_() for t in (x, w, w13, w2)]
    y64 = _layer64(want[0], ids, *want[1:])
    (y64 * dy.double()).sum().backward()
    # roundings to bf16 on the way: the two products' outputs, h and, backward, their gradients -- each at most 2^-9 of its
    # value (half a step), a handful of them in any path; 12 of them bound the relative 2-norm of every result
    for got, exp in ((y, y64), *((a.grad, b.grad) for a, b in zip(leaves, want))):
        rel = float((got.detach().cpu().double() - exp.detach()).norm() / exp.detach().norm())
        assert rel <= 12 * 2.0 ** -9, rel
    if invalid:
        assert not y[3].any() and not leaves[0].grad[3].any()


def test_gradient_from_an_odd_address():
    """The product's gradient as a contiguous view that does not start on 16 bytes: the same gradients bit for bit."""
    g = torch.Generator().manual_seed(8)
    x, w = torch.randn((19, 64), generator=g).to(BF).cuda(), torch.randn((3, 40, 64), generator=g).to(BF).cuda()
    off = torch.tensor([0, 5, 5, 19], dtype=torch.int32, device="cuda")
    dy = torch.randn((19, 40), generator=g).to(BF).cuda()
    grads = []
    for odd in (0, 3):
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = ragged.grouped_linear(a, b, off)
        whole = torch.cat([y.new_ones(odd), y.flatten()])
        whole.backward(torch.cat([dy.new_ones(odd), dy.flatten()]))
        grads.append((a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*grads))


@pytest.mark.parametrize("M", [0, 1, 3])
def test_no_valid_route(M):
    """No tokens, or tokens all of whose routes are invalid: zeros forward and backward, whatever x and the weights hold."""
    E, k, d, I = 4, 2, 64, 32
    x, w = torch.full((M, d), float("nan")), torch.full((M, k), float("inf"))
    ids = torch.tensor([[-1, E]], dtype=torch.int32).repeat(M, 1)
    _, _, _, w13, w2 = _problem(1, E, k, d, I, 5, False)
    leaves = [t.cuda().requires_grad_() for t in (x.to(BF), w, w13, w2)]
    y = ragged.expert_layer(leaves[0], ids.cuda(), *leaves[1:])
    y.sum().backward()
    assert y.shape == (M, d) and not y.any()
    assert all(t.grad.shape == t.shape and not t.grad.any() for t in leaves)
    q13, q2 = (ragged.quantize_experts(t.cuda(), moe.MOE_FP4_MXFP4) for t in (w13, w2))
    y4 = ragged.expert_layer_fp4(x.to(BF).cuda(), ids.cuda(), w.cuda(), q13, q2)
    assert y4.shape == (M, d) and not y4.any()


@pytest.mark.parametrize("fmt", [moe.MOE_FP4_NVFP4, moe.MOE_FP4_MXFP4])
def test_fp4_layer_on_the_same_codes(fmt):
    """x and the weights as their codes stand; h is quantized by the layer, compared through the same quantizer."""
    M, E, k, d, I = 21, 5, 2, 128, 64
    x, ids, w, w13, w2 = _problem(M, E, k, d, I, 3, True)
    nv = fmt == moe.MOE_FP4_NVFP4
    q13, q2 = ragged.quantize_experts(w13.cuda(), fmt), ragged.quantize_experts(w2.cuda(), fmt)
    ax = ragged.tensor_alpha(x.cuda()) if nv else None
    ah = torch.full((1,), 0.002, device="cuda") if nv else None
    y = ragged.expert_layer_fp4(x.cuda(), ids.cuda(), w.cuda(), q13, q2, ax, ah).cpu().double()

    def back(q):
        v = torch.from_numpy(ref.values(q.q.cpu(), q.s.cpu(), fmt))
        return v * q.alpha.cpu().double().view(-1, 1, 1) if nv else v

    xq, xs = ref.quantize(x.double().numpy(), fmt, ax.cpu().numpy() if nv else None)
    xv = torch.from_numpy(ref.values(xq, xs, fmt)) * (float(ax) if nv else 1.0)

    def h_round(h):
        q, s = ref.quantize(h.float().double().numpy()[None], fmt, ah.cpu().numpy() if nv else None)
        return torch.from_numpy(ref.values(q, s, fmt))[0] * (float(ah) if nv else 1.0)

    want = _layer64(xv, ids, w.double(), back(q13), back(q2), h_round)
    # h differs by FP32 rounding, so a few of its values may fall on the other side of a 4-bit border (a step there is up to
    # a third of the value): allow one value in 50, whose squares add up to (1/3)^2 / 50 of h's
    rel = float((y - want).norm() / want.norm())
    assert rel <= (1 / 3) * 50 ** -0.5, rel
    assert not y[3].any()


def test_capture_beside_an_eager_graph():
    """Refused with an exception while the eager graph lives; captured, with the eager gradients, once it is dropped."""
    g = torch.Generator().manual_seed(12)
    x, w = torch.randn((19, 64), generator=g).to(BF).cuda(), torch.randn((3, 40, 64), generator=g).to(BF).cuda().requires_grad_()
    off = torch.tensor([0, 5, 5, 19], dtype=torch.int32, device="cuda")
    eager = ragged.grouped_linear(x, w, off).sum()
    want, = torch.autograd.grad(eager, w, retain_graph=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="another stream lives"):
        with torch.cuda.graph(graph):
            y = ragged.grouped_linear(x, w, off).sum()
            torch.autograd.grad(y, w)
    del eager, y
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad, = torch.autograd.grad(ragged.grouped_linear(x, w, off).sum(), w)
    graph.replay()
    assert torch.equal(grad, want)


def test_captured_training_step_matches_eager():
    """Forward, loss and backward of fresh leaves in a graph: the same bits as eager, and the replay follows new inputs."""
    M, E, k, d, I = 40, 4, 2, 128, 64
    x, ids, w, w13, w2 = _problem(M, E, k, d, I, 5, False)
    ids, w = ids.cuda(), w.cuda()

    def eager(x):
        leaves = [t.cuda().requires_grad_() for t in (x, w13, w2)]
        ragged.expert_layer(leaves[0], ids, w, *leaves[1:]).square().sum().backward()
        return [t.grad.clone() for t in leaves]

    want = eager(x), eager(-x + 1)
    xs = x.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                                  # warm-up on the capture's stream, its graph freed
        eager(x)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    leaves = [xs.requires_grad_(), w13.cuda().requires_grad_(), w2.cuda().requires_grad_()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ragged.expert_layer(leaves[0], ids, w, *leaves[1:]).square().sum()
        grads = torch.autograd.grad(out, leaves)
        del out
    for new, exp in ((x, want[0]), (-x + 1, want[1])):
        with torch.no_grad():
            leaves[0].copy_(new)
        graph.replay()
        for a, b in zip(grads, exp):
            assert torch.equal(a, b)

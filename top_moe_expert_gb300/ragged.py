"""The routed expert layer on ragged groups: trained in bf16 or fp16, served in
NVFP4 or MXFP4.

    ids, w = moe.moe_topk_softmax(logits, k)
    y = ragged.expert_layer(x, ids, w, w13, w2)              # differentiable
    q13, q2 = (ragged.quantize_experts(t, moe.MOE_FP4_NVFP4) for t in (w13, w2))
    y = ragged.expert_layer_fp4(x, ids, w, q13, q2, alpha_x, alpha_h)

Routes are ordered by expert (moe_align_block_size with blocks of one row, no
padding between groups), the experts' products run on the groups as they are
(moe_grouped_mm, its gradients, moe_grouped_mm_fp4), and each token sums its
slots in slot order.  Routes to experts outside [0, E) contribute nothing.
moe_topk_softmax has no gradient; a router is trained through weights formed
from its choice, w = logits.gather(1, ids.long()).softmax(-1) (the same values).
Gathers, SwiGLU and the sum over slots are torch operations.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

import top_moe_expert_gb300 as moe


class Groups(NamedTuple):
    """Routes in expert order: `token` [R] of each row (0 for padding rows),
    `row` [M, k] of each route (R for an invalid route), `offsets` [E + 1]."""
    token: torch.Tensor
    row: torch.Tensor
    offsets: torch.Tensor


def group_routes(topk_ids: torch.Tensor, E: int, dev_status=None) -> Groups:
    """Rows for the routes topk_ids [M, k]: R = M * k of them, the valid routes
    first, by expert and then by route; the rest are padding."""
    M, k = topk_ids.shape
    R = M * k
    routes, experts, _ = moe.moe_align_block_size(topk_ids, E, 1, dev_status=dev_status)
    routes, experts = routes[:R], experts[:R]
    e = torch.where(experts < 0, E, experts)
    offsets = torch.searchsorted(e, torch.arange(E + 1, device=e.device, dtype=e.dtype), out_int32=True)
    row = torch.full((R + 1,), R, dtype=torch.int64, device=e.device)
    row[routes.long()] = torch.arange(R, device=e.device)            # padding rows all write entry R
    return Groups(torch.where(routes < R, routes // k, 0).long(), row[:R].view(M, k), offsets)


# A leaf's gradient is accumulated on the stream of its first use, for as long as
# any graph through it lives.  Where that is not the stream of a capture, the
# accumulation would end the capture, and the process with it; the stream is kept
# with the accumulating node, and an input that leads to one of another stream
# goes through a node that refuses before its gradient gets there.
_STREAM = "top_moe_expert_gb300.stream"
_NEAR = 8                               # nodes looked at per input: a cast, a gather, a softmax lie between


def _accumulators(t: torch.Tensor) -> list:
    """The accumulating nodes among the first _NEAR behind t."""
    nodes = [torch.autograd.graph.get_gradient_edge(t).node if t.is_leaf else t.grad_fn]
    for node in nodes:                                                # grows on the way
        if len(nodes) >= _NEAR:
            break
        for n, _ in node.next_functions:
            if n is not None:
                nodes.append(n)
    return [n for n in nodes if hasattr(n, "variable")]


class _Refuse(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t):
        return t.view_as(t)

    @staticmethod
    def backward(ctx, dt):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a backward pass cannot be captured while a graph of the same leaves from another "
                               "stream lives: drop its outputs, or warm up on the stream of the capture")
        return dt


def _guarded(*inputs):
    """The inputs, behind a refusing node where they need one, and the
    accumulating nodes, which the caller keeps until the new graph holds them."""
    if not torch.is_grad_enabled():
        return inputs, None
    nodes = [_accumulators(t) if t.requires_grad and moe._is_gpu(t) else () for t in inputs]
    if any(nodes):
        here = torch.cuda.current_stream(inputs[0].device).cuda_stream
        inputs = [_Refuse.apply(t) if any([n.metadata.setdefault(_STREAM, here) != here for n in ns]) else t
                  for t, ns in zip(inputs, nodes)]
    return inputs, nodes


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, dev_status):
        ctx.save_for_backward(x, w, offsets)
        ctx.dev_status = dev_status
        return moe.moe_grouped_mm(x, w, offsets, dev_status=dev_status)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16:                                       # a view into a larger gradient
            dy = dy.clone()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = moe.moe_grouped_mm_dgrad(dy, w, offsets, dev_status=ctx.dev_status)
        if ctx.needs_input_grad[1]:
            dw = moe.moe_grouped_mm_wgrad(dy, x, offsets, out_dtype=w.dtype, dev_status=ctx.dev_status)
        return dx, dw, None, None


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, dev_status=None) -> torch.Tensor:
    """moe_grouped_mm with gradients: rows x [R, K] of each expert times its
    w [E, N, K], transposed; first derivatives of x and w.  dev_status takes the
    device errors of the forward pass and, later, of the backward pass.  To capture the
    backward pass, drop earlier graphs of the same leaves first: one that came
    through here on another stream is refused, for x, w and what they are made
    of within a few operations (a leaf that only other operations have used,
    or one further off, is not known here)."""
    (x, w), kept = _guarded(x, w)
    return _GroupedLinear.apply(x, w, offsets, dev_status)


def _swiglu(h: torch.Tensor) -> torch.Tensor:
    g, u = h.float().chunk(2, dim=-1)
    return torch.nn.functional.silu(g) * u


def _weights(topk_w: torch.Tensor, groups: Groups) -> torch.Tensor:
    return topk_w.masked_fill(groups.row == groups.token.shape[0], 0.0)    # an invalid route: weight 0 of the zero row


def _combine(rows: torch.Tensor, groups: Groups, weights: torch.Tensor) -> torch.Tensor:
    rows = torch.cat([rows, rows.new_zeros((1, rows.shape[1]))])
    return (rows[groups.row].float() * weights.unsqueeze(-1)).sum(dim=1)


def expert_layer(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, w13: torch.Tensor,
                 w2: torch.Tensor, dev_status=None) -> torch.Tensor:
    """y [M, d] (fp32): sum_j w_j W2_e (SiLU(Wg_e x) * Wu_e x), differentiable in
    x [M, d], topk_w [M, k], w13 [E, 2I, d] and w2 [E, d, I] (one of bf16 and
    fp16; h is rounded to it).  dev_status int32 [2]: invalid routes are counted
    in the first, a device error of either pass is left in the second."""
    groups = group_routes(topk_ids, w13.shape[0], dev_status)
    (rows, weights, w13, w2), kept = _guarded(x[groups.token], _weights(topk_w, groups), w13, w2)
    h = _swiglu(_GroupedLinear.apply(rows, w13, groups.offsets, dev_status)).to(x.dtype)
    return _combine(_GroupedLinear.apply(h, w2, groups.offsets, dev_status), groups, weights)


def tensor_alpha(v: torch.Tensor) -> torch.Tensor:
    """NVFP4's constant of a tensor of activations: largest magnitude / (6 * 448), [1]."""
    return (v.abs().amax().float() / 2688.0).reshape(1)


def quantize_experts(w: torch.Tensor, fmt: int) -> "moe.Fp4":
    """w [E, N, K] in NVFP4 (a constant per expert) or MXFP4."""
    alpha = w.abs().amax(dim=(1, 2)).float() / 2688.0 if fmt == moe.MOE_FP4_NVFP4 else None
    return moe.Fp4(fmt, *moe.moe_fp4_quantize(w, fmt, alpha), alpha)


def expert_layer_fp4(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, w13: "moe.Fp4", w2: "moe.Fp4",
                     alpha_x: torch.Tensor | None = None, alpha_h: torch.Tensor | None = None,
                     dev_status=None) -> torch.Tensor:
    """expert_layer on 4-bit experts and activations: x and h are quantized to
    the experts' format; alpha_x, alpha_h [1]: NVFP4's constants of x and h,
    e.g. tensor_alpha of calibration data.  dev_status as expert_layer's."""
    fmt = w13.fmt
    groups = group_routes(topk_ids, w13.q.shape[0], dev_status)
    q, s = moe.moe_fp4_quantize(x, fmt, alpha_x)                      # a token's codes serve all its routes
    rows = moe.Fp4(fmt, q[groups.token], s[groups.token], alpha_x)
    h = _swiglu(moe.moe_grouped_mm_fp4(rows, w13, groups.offsets, out_dtype=torch.float32, dev_status=dev_status))
    hq = moe.Fp4(fmt, *moe.moe_fp4_quantize(h, fmt, alpha_h), alpha_h)
    y = moe.moe_grouped_mm_fp4(hq, w2, groups.offsets, out_dtype=torch.float32, dev_status=dev_status)
    return _combine(y, groups, _weights(topk_w, groups))


def main() -> None:
    """Fits a layer of experts to another one's outputs, then serves it in 4 bits."""
    E, k, d, I, M = 16, 4, 512, 256, 512
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t13, t2 = draw(E, 2 * I, d).mul_(d ** -0.5).bfloat16(), draw(E, d, I).mul_(I ** -0.5).bfloat16()
    m13, m2 = t13.float() + 0.02 * draw(E, 2 * I, d), t2.float() + 0.02 * draw(E, d, I)      # 32-bit masters
    w13, w2 = (t.bfloat16().requires_grad_() for t in (m13, m2))
    router = draw(d, E) * d ** -0.5
    for step in range(61):
        x = draw(M, d)
        ids, w = moe.moe_topk_softmax((x @ router).contiguous(), k)
        x = x.bfloat16()
        loss = (expert_layer(x, ids, w, w13, w2) - expert_layer(x, ids, w, t13, t2)).square().mean()
        loss.backward()
        with torch.no_grad():
            for p, m in ((w13, m13), (w2, m2)):
                m.sub_(p.grad.float(), alpha=200.0)
                p.copy_(m)
                p.grad = None
        if step % 20 == 0:
            print(f"step {step:3d}  loss {loss.item():.3e}")
    with torch.no_grad():
        y = expert_layer(x, ids, w, w13, w2)
        groups = group_routes(ids, E)
        h = _swiglu(moe.moe_grouped_mm(x[groups.token], w13.detach(), groups.offsets))
        for name, fmt in (("NVFP4", moe.MOE_FP4_NVFP4), ("MXFP4", moe.MOE_FP4_MXFP4)):
            ax, ah = (tensor_alpha(x), tensor_alpha(h)) if fmt == moe.MOE_FP4_NVFP4 else (None, None)
            y4 = expert_layer_fp4(x, ids, w, quantize_experts(w13.detach(), fmt), quantize_experts(w2.detach(), fmt), ax, ah)
            print(f"{name}: |y4 - y| / |y| = {((y4 - y).norm() / y.norm()).item():.3f}")


if __name__ == "__main__":
    main()

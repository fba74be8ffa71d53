"""Which captured backward passes the ragged layer refuses, on the CPU: accumulations on the stream of a graph that lives,
of leaves that are passed as they are, gathered or cast, and only where the pass asks for them."""
import ctypes
import gc
from types import SimpleNamespace

import pytest
import torch

import top_moe_expert_gb300 as moe
from top_moe_expert_gb300 import ragged

BF = torch.bfloat16


class _Zeros:
    """The library with products that leave their (zeroed) results alone."""
    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        return (lambda *a: 0) if name.startswith("moe_grouped_mm") else getattr(self.real, name)


@pytest.fixture
def state(monkeypatch):
    z = _Zeros(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: z)
    monkeypatch.setattr(moe, "_is_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_stream", lambda stream=None, device=None: ctypes.c_void_p(0))
    st = SimpleNamespace(stream=1, capturing=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=st.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: st.capturing)
    M, k, E = 3, 2, 2
    groups = ragged.Groups(torch.tensor([0, 1, 2, 0, 1, 2]), torch.tensor([[0, 3], [1, 4], [2, 5]]),
                           torch.tensor([0, 3, 6], dtype=torch.int32))
    monkeypatch.setattr(ragged, "group_routes", lambda ids, E, dev_status=None: groups)
    return st


def _layer():
    return SimpleNamespace(ids=torch.zeros((3, 2), dtype=torch.int32), x=torch.zeros((3, 32), dtype=BF).requires_grad_(),
                           w=torch.zeros((3, 2)).requires_grad_(), w13=torch.zeros((2, 64, 32), dtype=BF).requires_grad_(),
                           w2=torch.zeros((2, 32, 32), dtype=BF).requires_grad_())


def _run(t):
    return ragged.expert_layer(t.x, t.ids, t.w, t.w13, t.w2)


def _capture(state, make, *inputs):
    state.stream, state.capturing = 2, True
    try:
        return torch.autograd.grad(make().sum(), inputs)
    finally:
        state.stream, state.capturing = 1, False
        gc.collect()


@pytest.mark.parametrize("leaf", ["x", "w", "w13", "w2"])
def test_every_leaf_of_the_layer_is_guarded(state, leaf):
    t = _layer()
    eager = _run(t)
    with pytest.raises(RuntimeError, match="another stream lives"):
        _capture(state, lambda: _run(t), getattr(t, leaf))
    del eager
    gc.collect()
    _capture(state, lambda: _run(t), getattr(t, leaf))


def test_a_leaf_behind_a_cast_or_a_gather(state):
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    for make, leaf in (
            (lambda m: ragged.grouped_linear(torch.zeros((6, 32), dtype=BF), m.bfloat16(), off), torch.zeros((2, 64, 32))),
            (lambda m: ragged.grouped_linear(m[torch.tensor([0, 1, 2, 2, 1, 0])], torch.zeros((2, 64, 32), dtype=BF), off),
             torch.zeros((3, 32), dtype=BF)),
            (lambda m: ragged.grouped_linear((m * 2).bfloat16()[torch.tensor([0, 1, 2, 2, 1, 0])],
                                             torch.zeros((2, 64, 32), dtype=BF), off), torch.zeros((3, 32)))):
        leaf.requires_grad_()
        eager = make(leaf)
        with pytest.raises(RuntimeError, match="another stream lives"):
            _capture(state, lambda: make(leaf), leaf)
        del eager
        gc.collect()
        _capture(state, lambda: make(leaf), leaf)


def test_only_what_the_pass_asks_for(state):
    """An eager graph through w does not stand in the way of x's gradient alone."""
    x, w = torch.zeros((6, 32), dtype=BF).requires_grad_(), torch.zeros((2, 64, 32), dtype=BF).requires_grad_()
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    eager = ragged.grouped_linear(x.detach(), w, off)
    assert _capture(state, lambda: ragged.grouped_linear(x, w, off), x)[0].shape == x.shape
    with pytest.raises(RuntimeError, match="another stream lives"):
        _capture(state, lambda: ragged.grouped_linear(x, w, off), x, w)
    del eager


def test_eager_passes_and_the_capture_s_own_stream(state):
    t = _layer()
    kept = _run(t)
    state.stream = 3
    torch.autograd.grad(_run(t).sum(), (t.x, t.w, t.w13, t.w2))         # another stream, no capture
    state.stream, state.capturing = 1, True
    torch.autograd.grad(_run(t).sum(), (t.x, t.w, t.w13, t.w2))         # a capture on the graph's own stream
    state.capturing = False
    del kept

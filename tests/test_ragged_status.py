"""The ragged layer hands dev_status to every launch of its forward and backward passes (CPU: launches are recorded)."""
import ctypes

import pytest
import torch

import top_moe_expert_gb300 as moe
from top_moe_expert_gb300 import ragged

BF = torch.bfloat16
# where the entry points take dev_status
AT = {"moe_grouped_mm": 10, "moe_grouped_mm_dgrad": 10, "moe_grouped_mm_wgrad": 11, "moe_grouped_mm_fp4": 14}


class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in AT or name == "moe_fp4_quantize":
            return lambda *a: self.calls.append((name, a)) or 0
        return getattr(self.real, name)


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_is_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_stream", lambda stream=None, device=None: ctypes.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type("S", (), dict(cuda_stream=0)))
    groups = ragged.Groups(torch.zeros(6, dtype=torch.int64), torch.zeros((3, 2), dtype=torch.int64),
                           torch.tensor([0, 3, 6], dtype=torch.int32))
    r.routed = []
    monkeypatch.setattr(ragged, "group_routes", lambda ids, E, st=None: r.routed.append(st) or groups)
    return r


def _statuses(rec):
    return [a[AT[n]] for n, a in rec.calls if n in AT]


@pytest.mark.parametrize("given", [True, False])
def test_every_launch_gets_it(rec, given):
    st = torch.zeros(2, dtype=torch.int32) if given else None
    at = st.data_ptr() if given else None
    x, w = torch.zeros((6, 32), dtype=BF).requires_grad_(), torch.zeros((2, 64, 32), dtype=BF).requires_grad_()
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    ragged.grouped_linear(x, w, off, dev_status=st).sum().backward()
    assert _statuses(rec) == [at] * 3
    rec.calls.clear()
    ids, tw = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    w2 = torch.zeros((2, 32, 32), dtype=BF).requires_grad_()
    ragged.expert_layer(x[:3], ids, tw, w, w2, dev_status=st).sum().backward()
    assert _statuses(rec) == [at] * 6
    rec.calls.clear()
    with torch.no_grad():
        q13, q2 = (ragged.quantize_experts(t.detach(), moe.MOE_FP4_MXFP4) for t in (w, w2))
        ragged.expert_layer_fp4(x[:3].detach(), ids, tw, q13, q2, dev_status=st)
    assert _statuses(rec) == [at] * 2
    assert len(rec.routed) == 2 and all(r is st for r in rec.routed)


def test_a_wrong_one_is_refused(rec):
    x, w, off = torch.zeros((6, 32), dtype=BF), torch.zeros((2, 64, 32), dtype=BF), torch.zeros(3, dtype=torch.int32)
    for st in (torch.zeros(1, dtype=torch.int32), torch.zeros(2), [0, 0]):
        with pytest.raises(ValueError):
            ragged.grouped_linear(x, w, off, dev_status=st)
    assert not rec.calls

"""Device errors and invalid routes reach the caller of the ragged layer, from both passes."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from top_moe_expert_gb300 import ragged

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_bad_offsets_are_reported_by_both_passes():
    x = torch.ones((12, 32), dtype=BF, device="cuda").requires_grad_()
    w = torch.ones((2, 64, 32), dtype=BF, device="cuda").requires_grad_()
    for bad in ([0, 8, 20], [1, 4, 12]):
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        y = ragged.grouped_linear(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), dev_status=st)
        assert st.tolist() == [0, 7]
        st.zero_()
        y.sum().backward()
        assert st.tolist() == [0, 7]


def test_layers_count_invalid_routes_and_report_nothing_else():
    g = torch.Generator().manual_seed(3)
    M, E, k, d, I = 9, 4, 2, 64, 32
    x = torch.randn((M, d), generator=g).to(BF).cuda().requires_grad_()
    w13 = torch.randn((E, 2 * I, d), generator=g).to(BF).cuda().requires_grad_()
    w2 = torch.randn((E, d, I), generator=g).to(BF).cuda().requires_grad_()
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    ids[2, 0], ids[5] = -1, E
    w = torch.rand((M, k), generator=g).cuda()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    ragged.expert_layer(x, ids.cuda(), w, w13, w2, dev_status=st).sum().backward()
    assert st.tolist() == [3, 0]
    with torch.no_grad():
        q13, q2 = (ragged.quantize_experts(t, moe.MOE_FP4_MXFP4) for t in (w13, w2))
        ragged.expert_layer_fp4(x, ids.cuda(), w, q13, q2, dev_status=st)
    assert st.tolist() == [6, 0]

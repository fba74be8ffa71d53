"""The product with 4-bit AWQ weights where CTAs take 32 rows of them: exact sums in every form of the kernel."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as rr
from tests import route_ref as ref

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _wide(sizes, N):
    """The rule of the kernel's host code: 32 rows of w per CTA leave eight CTAs for every SM."""
    live = min(len(sizes), sum(sizes))
    return live * -(-N // 32) >= 8 * torch.cuda.get_device_properties(0).multi_processor_count


def _check(x, w, off, want, out, R):
    y = torch.full((R, want.shape[1]), float("nan"), dtype=out, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    moe.moe_grouped_mm_awq(x, w, off, out_dtype=out, y=y, dev_status=st)
    assert torch.equal(y.cpu(), want.to(out)) and st.tolist() == [0, 0]


@pytest.mark.parametrize("K", [384, 4224])
def test_one_expert(K):
    """N ends 8 rows into a CTA's 32; an odd number of groups, over two and over four warps; runs of 1, 8, 9 and 17 rows.
    Whole x up to 4 and scales 1/2, 1, 2: every partial sum is a multiple of 1/2 below 2^23."""
    g = torch.Generator().manual_seed(K)
    N = 40960 + 8
    q, s, z = ref.awq_random(1, N, K, g, [0.5, 1.0, 2.0])
    x = torch.randint(-4, 5, (17, K), generator=g)
    want = torch.cat([x.double() @ ref.awq_values(q[:, n:n + 4096], s[:, n:n + 4096], z[:, n // 8:n // 8 + 512])[0].T
                      for n in range(0, N, 4096)], dim=1)
    assert 4 * 15 * 2 * K < 2 ** 23
    w = moe.Weights(moe.MOE_W_AWQ4, q.cuda(), s.cuda(), z.cuda())
    for R in (1, 8, 9, 17):
        assert _wide([R], N)
        for dt in (BF, F16):
            for out in (dt, F32):
                _check(x[:R].to(dt).cuda(), w, rr.offsets_of([R]).cuda(), want[:R], out, R)


@pytest.mark.parametrize("N,K,sizes", [(1000, 384, [9 + e % 9 for e in range(40)]), (1000, 4224, [9 + e % 9 for e in range(40)]),
                                       (5000, 4224, [1, 0, 1, 3, 1, 1, 0, 1]), (5000, 384, [1, 0, 1, 3, 1, 1, 0, 1])])
def test_many_experts(N, K, sizes):
    """The same over experts of unequal rows; rows behind the last one are zeros."""
    g = torch.Generator().manual_seed(N + K)
    E, R = len(sizes), sum(sizes)
    pad = 2 if R > 8 else 0
    assert _wide(sizes, N)
    q, s, z = ref.awq_random(E, N, K, g, [0.5, 1.0, 2.0])
    x = torch.randint(-4, 5, (R + pad, K), generator=g)
    off, want = rr.offsets_of(sizes), torch.zeros((R + pad, N), dtype=torch.float64)
    for e in range(E):
        if sizes[e]:
            want[off[e]:off[e + 1]] = x[off[e]:off[e + 1]].double() @ ref.awq_values(q[e:e + 1], s[e:e + 1], z[e:e + 1])[0].T
    w = moe.Weights(moe.MOE_W_AWQ4, q.cuda(), s.cuda(), z.cuda())
    for dt in (BF, F16):
        for out in (dt, F32):
            _check(x.to(dt).cuda(), w, off.cuda(), want, out, R + pad)

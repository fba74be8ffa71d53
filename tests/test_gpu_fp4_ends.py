"""The 4-bit product at the ends of its ranges."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NV, MX = moe.MOE_FP4_NVFP4, moe.MOE_FP4_MXFP4


def _rows(shape, K, fmt, g, scales):
    """Random codes, scales drawn from the given bytes."""
    q = torch.randint(0, 256, (*shape, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    nb = K // ref.BLOCK[fmt]
    s = torch.zeros((*shape, (nb + 15) // 16 * 16), dtype=torch.uint8)
    pick = torch.tensor(scales, dtype=torch.uint8)
    s[..., :nb] = pick[torch.randint(0, len(scales), (*shape, nb), generator=g)]
    return q, s


@pytest.mark.parametrize("xe,we", [(-75, -75), (-80, -80), (-62, -61), (-100, -30), (70, 70), (100, 20), (100, -100), (-100, 100),
                                   (50, 60), (0, 0)])
@pytest.mark.parametrize("sizes", [[20, 0, 70], [400]])
def test_constants_at_the_ends_of_their_range(xe, we, sizes):
    """Powers of two from 2^-100 to 2^100: exact sums times an exact power, rounded to FP32 once whatever the product of
    the two constants is; a row of zeros stays zero."""
    g = torch.Generator().manual_seed(xe * 7 + we)
    N, K, R, E = 136, 96, sum(sizes) + 2, len(sizes)
    for scales in ([0x30, 0x38, 0x40], [0x70, 0x78], [0x08, 0x10]):        # about 1, up to 256, down to 2^-6
        xq, xs = _rows((R,), K, NV, g, scales)
        wq, ws = _rows((E, N), K, NV, g, scales)
        xq[3] = 0
        xa, wa = torch.tensor([2.0 ** xe]), torch.tensor([2.0 ** we] * E)
        want, _ = ref.mm(torch.from_numpy(ref.values(xq, xs, NV)), torch.from_numpy(ref.values(wq, ws, NV)), sizes)
        want = (want * 2.0 ** xe * 2.0 ** we).float()
        for out in (F32, BF):
            y = moe.moe_grouped_mm_fp4(moe.Fp4(NV, xq.cuda(), xs.cuda(), xa.cuda()),
                                       moe.Fp4(NV, wq.cuda(), ws.cuda(), wa.cuda()), ref.offsets_of(sizes).cuda(),
                                       out_dtype=out).cpu()
            assert torch.equal(y, want.to(out)), (scales, out, int((y != want.to(out)).sum()))
        assert not y[3].any()

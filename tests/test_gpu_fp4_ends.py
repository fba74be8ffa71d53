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


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("K,out", [(8192, F32), (8224, F32), (10336, F32), (16384, F32), (32768, BF), (32800, BF),
                                   (34816, torch.float16)])
@pytest.mark.parametrize("sizes,N", [([1, 0, 40], 136), ([130, 33], 264)])
def test_long_sums_exact(fmt, K, out, sizes, N):
    """Around the lengths from which the sums are added in parts: sums that are exact in FP32."""
    g = torch.Generator().manual_seed(K + N)
    R, E = sum(sizes) + 1, len(sizes)
    scales = [0x30, 0x38, 0x40] if fmt == NV else [126, 127, 128]
    xq, xs = _rows((R,), K, fmt, g, scales)
    wq, ws = _rows((E, N), K, fmt, g, scales)
    xa, wa = (torch.tensor([0.5], device="cuda"), torch.ones(E, device="cuda")) if fmt == NV else (None, None)
    want, _ = ref.mm(torch.from_numpy(ref.values(xq, xs, fmt)), torch.from_numpy(ref.values(wq, ws, fmt)), sizes)
    want = want * (0.5 if fmt == NV else 1.0)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_mm_fp4(moe.Fp4(fmt, xq.cuda(), xs.cuda(), xa), moe.Fp4(fmt, wq.cuda(), ws.cuda(), wa),
                               ref.offsets_of(sizes).cuda(), out_dtype=out, dev_status=st).cpu()
    assert st.tolist() == [0, 0]
    assert torch.equal(y, want.to(out)), int((y != want.to(out)).sum())


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("K", [2048, 7168, 8192, 8224, 32768, 131072])
def test_long_sums_of_one_sign_do_not_drift(fmt, K):
    """Codes of one sign, scales over a wide range.  An MMA adds 64 products and may lose 2^-23 of the sum; past 8192
    elements a part has 32 of them, and adding the parts loses at most 2^-24 of the sum each."""
    g = torch.Generator().manual_seed(K)
    N, R = 64, 40
    scales = list(range(0x01, 0x7F)) if fmt == NV else list(range(117, 138))
    xq, xs = _rows((R,), K, fmt, g, scales)
    wq, ws = _rows((1, N), K, fmt, g, scales)
    xq, wq = xq & 0x77, wq & 0x77
    one = torch.ones(1, device="cuda") if fmt == NV else None
    y = moe.moe_grouped_mm_fp4(moe.Fp4(fmt, xq.cuda(), xs.cuda(), one), moe.Fp4(fmt, wq.cuda(), ws.cuda(), one),
                               ref.offsets_of([R]).cuda(), out_dtype=F32).cpu().double()
    want = torch.from_numpy(ref.values(xq, xs, fmt)) @ torch.from_numpy(ref.values(wq, ws, fmt))[0].T
    bound = K / 64 * 2.0 ** -23 if K <= 8192 else 32 * 2.0 ** -23 + -(-K // 2048) * 2.0 ** -24
    rel = ((y - want).abs() / want).max()
    assert rel <= bound + 2.0 ** -24, (float(rel), bound)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("sizes", [[700, 0, 33, 900], [8] * 40])
def test_same_bits_beside_other_work(fmt, sizes):
    """Repeated calls, alone and beside a stream that keeps the memory busy, give the bits of the first, which are exact."""
    g = torch.Generator().manual_seed(len(sizes))
    R, E, N, K = sum(sizes), len(sizes), 1032, 4192
    scales = [0x30, 0x38, 0x40] if fmt == NV else [126, 127, 128]
    xq, xs = _rows((R,), K, fmt, g, scales)
    wq, ws = _rows((E, N), K, fmt, g, scales)
    a = (torch.ones(1, device="cuda"), torch.ones(E, device="cuda")) if fmt == NV else (None, None)
    X, W = moe.Fp4(fmt, xq.cuda(), xs.cuda(), a[0]), moe.Fp4(fmt, wq.cuda(), ws.cuda(), a[1])
    off = ref.offsets_of(sizes).cuda()
    want, _ = ref.mm(torch.from_numpy(ref.values(xq, xs, fmt)), torch.from_numpy(ref.values(wq, ws, fmt)), sizes)
    first = moe.moe_grouped_mm_fp4(X, W, off, out_dtype=F32)
    assert torch.equal(first.cpu().double(), want)
    side, buf = torch.cuda.Stream(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(120):
        if i >= 60:
            with torch.cuda.stream(side):
                buf.fill_(i)
        differ += (moe.moe_grouped_mm_fp4(X, W, off, out_dtype=F32) != first).sum()
    torch.cuda.synchronize()
    assert int(differ) == 0

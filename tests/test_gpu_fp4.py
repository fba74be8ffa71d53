"""NVFP4 / MXFP4 quantization (bit for bit), the values back, and the ragged product on them."""
import numpy as np
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NV, MX = moe.MOE_FP4_NVFP4, moe.MOE_FP4_MXFP4


def _alpha(v, groups):
    return (v.double().reshape(groups, -1).abs().amax(dim=1) / 2688).float()


def _check_codes(v, fmt, alpha):
    rows = v.reshape(-1, v.shape[-1])
    want = ref.quantize(rows.double().numpy(), fmt, None if alpha is None else alpha.numpy())
    q, s = moe.moe_fp4_quantize(v.cuda(), fmt, None if alpha is None else alpha.cuda())
    q, s = q.cpu().numpy().reshape(want[0].shape), s.cpu().numpy().reshape(want[1].shape)
    assert np.array_equal(s, want[1]), f"{(s != want[1]).sum()} scales differ, first at {np.argwhere(s != want[1])[0]}"
    assert np.array_equal(q, want[0]), f"{(q != want[0]).sum()} codes differ, first at {np.argwhere(q != want[0])[0]}"
    return q, s


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("rows,K,groups", [(1, 32, 1), (3, 64, 3), (7, 96, 1), (8, 544, 2), (5, 2048, 1), (130, 768, 10),
                                           (257, 1056, 1)])
def test_codes_and_values(fmt, dt, rows, K, groups):
    g = torch.Generator().manual_seed(rows * K)
    v = (torch.randn((rows, K), generator=g) * torch.exp(torch.randn((K,), generator=g))).to(dt)
    alpha = _alpha(v, groups) if fmt == NV else None
    q, s = _check_codes(v, fmt, alpha)
    want = ref.values(q, s, fmt)
    if alpha is not None:
        want = want * np.repeat(alpha.numpy().astype(np.float64), rows // groups)[:, None]
    qc, sc = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    for out in (BF, HF, F32):
        got = moe.moe_fp4_dequantize(qc, sc, fmt, None if alpha is None else alpha.cuda(), out_dtype=out).cpu()
        w = torch.from_numpy(want)
        # S * code is exact; alpha times it is one FP32 rounding, the output type one more
        tol = w.abs() * (2.0 ** -24 + (0 if out == F32 else torch.finfo(out).eps / 2) * (1 + 2.0 ** -24))
        if out == HF:
            tol = tol + 2.0 ** -25
        assert ((got.double() - w).abs() <= tol).all()


@pytest.mark.parametrize("fmt", [NV, MX])
def test_ties_zeros_signs_and_extremes(fmt):
    """Values on the rounding borders, signed zeros, subnormals, the largest values, blocks of zeros."""
    K = 64
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = []
    for scale in (1.0, 2.0 ** -20, 2.0 ** 30, 2.0 ** -126, 2.0 ** -140, 2.0 ** 124):
        r = torch.cat([mids, -mids]).repeat(K // 16) * scale
        rows += [r, torch.nextafter(r, torch.zeros_like(r)), torch.nextafter(r, r * 4)]
    rows += [torch.zeros(K), -torch.zeros(K), torch.full((K,), 3.4e38), torch.full((K,), 1e-45)]
    v = torch.stack(rows).float()
    v = torch.where(v.isinf(), torch.full_like(v, 3e38), v)
    alpha = None
    if fmt == NV:                                              # alpha where the rows' own scale puts them at 6 * S
        alpha = torch.full((v.shape[0],), 1.0)
        for i in range(v.shape[0]):
            top = float(v[i].abs().max())
            alpha[i] = min(max(top / 6, 2.0 ** -100), 2.0 ** 100)
    _check_codes(v, fmt, alpha)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_blocks_with_nan_or_infinity_read_back_as_nan(fmt, dt):
    g = torch.Generator().manual_seed(4)
    v = torch.randn((4, 96), generator=g).to(dt)
    v[0, 5], v[1, 40], v[2, 95], v[3, 31] = float("nan"), float("inf"), float("-inf"), float("nan")
    alpha = torch.tensor([0.002]) if fmt == NV else None
    q, s = _check_codes(v, fmt, alpha)
    back = moe.moe_fp4_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), fmt,
                                  None if alpha is None else alpha.cuda()).cpu()
    b = ref.BLOCK[fmt]
    for r, k in ((0, 5), (1, 40), (2, 95), (3, 31)):
        assert back[r, k // b * b:k // b * b + b].isnan().all()
        assert int(back[r].isnan().sum()) == b


def test_zero_alpha_over_zero_rows():
    q, s = moe.moe_fp4_quantize(torch.zeros((2, 64), device="cuda"), NV, torch.zeros(1, device="cuda"))
    assert not q.any() and not s.any()
    assert not moe.moe_fp4_dequantize(q, s, NV, torch.zeros(1, device="cuda")).any()


def test_quantize_past_32_bits_of_elements():
    rows, K = 1_050_000, 2048                                   # > 2^31 elements
    v = torch.zeros((rows, K), dtype=BF, device="cuda")
    tail = torch.randn((3, K), generator=torch.Generator().manual_seed(6)).to(BF)
    v[-3:] = tail.cuda()
    q, s = moe.moe_fp4_quantize(v, MX)
    want = ref.quantize(tail.double().numpy(), MX)
    assert np.array_equal(q[-3:].cpu().numpy(), want[0]) and np.array_equal(s[-3:].cpu().numpy(), want[1])
    assert not q[:-3].any() and not s[:-3].any()
    back = moe.moe_fp4_dequantize(q, s, MX, out_dtype=BF)
    assert np.array_equal(back[-3:].cpu().double().numpy(), ref.values(*want, MX))


def test_no_rows():
    for fmt, a in ((NV, torch.ones(1, device="cuda")), (MX, None)):
        q, s = moe.moe_fp4_quantize(torch.empty((0, 64), device="cuda"), fmt, a)
        assert q.shape == (0, 32) and s.shape == (0, 16)
        assert moe.moe_fp4_dequantize(q, s, fmt, a).shape == (0, 64)


# ---------------------------------------------------------------- the product

def _codes(shape, K, fmt, g, exact):
    """Random codes and scales.  exact: scales 1/2, 1 or 2, so that sums of a few thousand products are exact in FP32."""
    q = torch.randint(0, 256, (*shape, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    nb, Ks = K // ref.BLOCK[fmt], (K // ref.BLOCK[fmt] + 15) // 16 * 16
    s = torch.zeros((*shape, Ks), dtype=torch.uint8)
    if exact:
        pick = torch.tensor([0x30, 0x38, 0x40] if fmt == NV else [126, 127, 128], dtype=torch.uint8)
        s[..., :nb] = pick[torch.randint(0, 3, (*shape, nb), generator=g)]
    else:
        lo, hi = (0x01, 0x7F) if fmt == NV else (117, 138)
        s[..., :nb] = torch.randint(lo, hi, (*shape, nb), generator=g, dtype=torch.int32).to(torch.uint8)
    return q, s


def _product(fmt, sizes, N, K, g, exact, out, pad=3):
    R, E = sum(sizes) + pad, len(sizes)
    xq, xs = _codes((R,), K, fmt, g, exact)
    wq, ws = _codes((E, N), K, fmt, g, exact)
    xa, wa = (torch.tensor([0.5]), 2.0 ** torch.randint(-2, 3, (E,), generator=g).float()) if fmt == NV else (None, None)
    if fmt == NV and not exact:
        xa, wa = torch.rand(1, generator=g) + 0.5, torch.rand(E, generator=g) + 0.5
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = torch.full((R, N), float("nan"), dtype=out, device="cuda")
    moe.moe_grouped_mm_fp4(moe.Fp4(fmt, c(xq), c(xs), c(xa)), moe.Fp4(fmt, c(wq), c(ws), c(wa)),
                           ref.offsets_of(sizes).cuda(), y=y, dev_status=st)
    assert st.tolist() == [0, 0]
    x, w = torch.from_numpy(ref.values(xq, xs, fmt)), torch.from_numpy(ref.values(wq, ws, fmt))
    if fmt == NV:
        w = w * (xa.double() * wa.double())[:, None, None]
    want, mag = ref.mm(x, w, sizes)
    return y.cpu(), want, mag


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("sizes", [[1], [0, 0, 1, 0], [1, 0, 1, 1, 0, 1, 1], [15, 16, 17, 31, 0, 33, 65], [95, 96, 97, 193, 191],
                                   [0, 0], [1, 400, 0, 260]])
@pytest.mark.parametrize("N,K", [(8, 32), (128, 256), (136, 96), (264, 544), (512, 512), (1000, 800)])
def test_product_exact(fmt, sizes, N, K):
    g = torch.Generator().manual_seed(N + K + len(sizes))
    y, want, _ = _product(fmt, sizes, N, K, g, True, F32)
    bad = y.double() != want
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("out", [BF, HF, F32])
@pytest.mark.parametrize("sizes,N,K", [([300, 0, 7], 256, 2048), ([1, 1, 1], 768, 768), ([513], 136, 1056)])
def test_product_within_the_sums_bound(fmt, out, sizes, N, K):
    g = torch.Generator().manual_seed(N * K)
    y, want, mag = _product(fmt, sizes, N, K, g, False, out)
    fits = want.abs() < (torch.finfo(out).max if out == HF else float("inf"))
    # the constant alpha is one more FP32 rounding, and so is its product with the sum
    tol = ref.tolerance(want, mag, K + 4, out)
    err = (y.double() - want).abs()
    assert (err <= tol)[fits].all(), float((err / (mag + 1e-30))[fits].max())


@pytest.mark.parametrize("fmt", [NV, MX])
def test_product_nan_scales(fmt):
    """A NaN scale reaches the results of its row (x) or column (w) and no other."""
    g = torch.Generator().manual_seed(8)
    sizes, N, K = [20, 140], 136, 256
    xq, xs = _codes((160,), K, fmt, g, True)
    wq, ws = _codes((2, N), K, fmt, g, True)
    nan = 0x7F if fmt == NV else 0xFF
    xs[30, 3], ws[0, 7, 5] = nan, nan
    one = torch.ones(1, device="cuda") if fmt == NV else None
    two = torch.ones(2, device="cuda") if fmt == NV else None
    y = moe.moe_grouped_mm_fp4(moe.Fp4(fmt, xq.cuda(), xs.cuda(), one), moe.Fp4(fmt, wq.cuda(), ws.cuda(), two),
                               ref.offsets_of(sizes).cuda(), out_dtype=F32).cpu()
    want = torch.zeros((160, N), dtype=torch.bool)
    want[30], want[:20, 7] = True, True
    assert torch.equal(y.isnan(), want)


def test_product_past_32_bits_and_same_bits():
    g = torch.Generator().manual_seed(9)
    E, N, K = 70, 8192, 8192                                    # E*N*K > 2^32 elements
    wq = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    tq, ts = _codes((N,), K, MX, g, True)
    wq[-1], ws[-1] = tq.cuda(), ts.cuda()
    xq, xs = _codes((40,), K, MX, g, True)
    off = ref.offsets_of([0] * (E - 1) + [40]).cuda()
    call = lambda: moe.moe_grouped_mm_fp4(moe.Fp4(MX, xq.cuda(), xs.cuda()), moe.Fp4(MX, wq, ws), off, out_dtype=F32)  # noqa: E731
    y = call()
    want = torch.from_numpy(ref.values(xq, xs, MX)) @ torch.from_numpy(ref.values(tq, ts, MX)).T
    assert torch.equal(y.cpu().double(), want)
    assert torch.equal(y, call())


def test_quantize_and_product_on_another_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(10)
    N, K, R = 256, 512, 50
    v = torch.randn((R, K), generator=g).to(BF).cuda()
    wq, ws = (t.cuda() for t in _codes((1, N), K, NV, g, True))
    xa, wa = torch.full((1,), 0.002, device="cuda"), torch.ones(1, device="cuda")
    off = ref.offsets_of([R]).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, sc = torch.empty((R, K // 2), dtype=torch.uint8, device="cuda"), torch.empty((R, K // 16), dtype=torch.uint8, device="cuda")
    y = torch.empty((R, N), device="cuda")

    def step(stream=None):
        moe.moe_fp4_quantize(v, NV, xa, q=q, s=sc, stream=stream)
        moe.moe_grouped_mm_fp4(moe.Fp4(NV, q, sc, xa), moe.Fp4(NV, wq, ws, wa), off, y=y, stream=stream)

    step(s)
    torch.cuda.current_stream().wait_stream(s)
    first = y.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    y.fill_(0)
    gr.replay()
    assert torch.equal(y, first)
    rq, rs = ref.quantize(v.cpu().double().numpy(), NV, xa.cpu().numpy())
    x, w = torch.from_numpy(ref.values(rq, rs, NV)), torch.from_numpy(ref.values(wq.cpu(), ws.cpu(), NV))
    want, mag = ref.mm(x * float(xa), w, [R])
    assert ((first.cpu().double() - want).abs() <= ref.tolerance(want, mag, K + 4, F32)).all()

"""The grouped product with 4-bit AWQ weights: exact where the sums are, within the derived bound elsewhere."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as rr
from tests import route_ref as ref

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def _weights(E, N, K, g, scales=None):
    q, s, z = ref.awq_random(E, N, K, g, scales)
    return moe.Weights(moe.MOE_W_AWQ4, q.cuda(), s.cuda(), z.cuda()), ref.awq_values(q, s, z)


def _bound(want, mag, K, dt):
    """Groups of 128: at most 2^-23 of the terms' magnitudes per 16; their sums by FMA and over the warps, 2^-24 each."""
    tol = (8 + (K // 128 + 9) / 2) * 2.0 ** -23 * mag
    if dt != F32:
        tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if dt == F16 else 0)
    return tol + 1e-37


SIZES = [[1], [8], [9], [33], [100], [0, 1, 0], [1] * 8, [3, 0, 8, 9, 1], [0, 40, 0, 65, 7, 0], [2] * 40, [0, 0]]


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("N,K", [(8, 128), (24, 256), (136, 640), (1000, 1152), (64, 4224)])
def test_exact_sums(dt, sizes, N, K):
    """Whole x up to 4 and scales 1/2, 1, 2: every partial sum is a multiple of 1/2 below 2^23."""
    g = torch.Generator().manual_seed(sum(sizes) + N + K)
    E, R = len(sizes), sum(sizes) + 3
    w, values = _weights(E, N, K, g, [0.5, 1.0, 2.0])
    x = torch.randint(-4, 5, (R, K), generator=g).to(dt)
    want, mag = rr.mm(x, values, sizes)
    assert mag.max() < 2 ** 23
    for out in (dt, F32):
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        y = torch.full((R, N), NAN, dtype=out, device="cuda")
        moe.moe_grouped_mm_awq(x.cuda(), w, rr.offsets_of(sizes).cuda(), out_dtype=out, y=y, dev_status=st)
        assert torch.equal(y.cpu(), want.to(out)) and st.tolist() == [0, 0]


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("sizes,N,K", [([3], 8, 131072), ([700, 0, 813], 136, 256), ([1] * 1024, 8, 128), ([0] * 1023 + [17], 40, 128)],
                         ids=["long", "many rows", "an expert each", "the last expert"])
def test_extreme_sizes(dt, sizes, N, K):
    """Exact sums as above: x up to 1 over the long ones."""
    g = torch.Generator().manual_seed(N + K)
    E, R, top = len(sizes), sum(sizes) + 1, 1 if K > 10000 else 4
    w, values = _weights(E, N, K, g, [0.5, 1.0, 2.0])
    x = torch.randint(-top, top + 1, (R, K), generator=g).to(dt)
    want, mag = rr.mm(x, values, sizes)
    assert mag.max() < 2 ** 23
    y = moe.moe_grouped_mm_awq(x.cuda(), w, rr.offsets_of(sizes).cuda(), out_dtype=F32)
    assert torch.equal(y.cpu(), want.float())


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("sizes,N,K", [([1], 4096, 7168), ([8, 0, 1, 33], 72, 2048), ([5], 256, 16384), ([20, 70], 512, 768),
                                       ([1] * 64, 40, 384)])
def test_normal_inputs(dt, sizes, N, K):
    g = torch.Generator().manual_seed(N + K)
    w, values = _weights(len(sizes), N, K, g)
    x = torch.randn((sum(sizes), K), generator=g).to(dt)
    want, mag = rr.mm(x, values, sizes)
    for out in (dt, F32):
        y = moe.moe_grouped_mm_awq(x.cuda(), w, rr.offsets_of(sizes).cuda(), out_dtype=out).cpu().double()
        off = (y - want).abs() - _bound(want, mag, K, out)
        assert not (off > 0).any(), float(off.max())


@pytest.mark.parametrize("dt", [BF, F16])
def test_large_values(dt):
    """x up to the type's end, the largest scales, FP32 sums that stay finite."""
    g = torch.Generator().manual_seed(3)
    w, values = _weights(1, 16, 256, g, [60000.0, 2.0 ** -14, 2.0 ** -24])
    x = (torch.randn((3, 256), generator=g) * (1e30 if dt == BF else 2e4)).to(dt)
    want, mag = rr.mm(x, values, [3])
    y = moe.moe_grouped_mm_awq(x.cuda(), w, rr.offsets_of([3]).cuda(), out_dtype=F32).cpu().double()
    assert not ((y - want).abs() > _bound(want, mag, 256, F32)).any()


def test_rows_do_not_reach_each_other():
    """NaN and infinity in another expert's, the same expert's and the padding rows; the same bits beside other rows."""
    g = torch.Generator().manual_seed(4)
    sizes = [3, 9, 0, 34]
    w, _ = _weights(4, 48, 512, g)
    x, off = torch.randn((50, 512), generator=g).to(BF), rr.offsets_of(sizes).cuda()
    y = moe.moe_grouped_mm_awq(x.cuda(), w, off)
    bad = x.clone()
    for r, v in ((1, NAN), (5, float("inf")), (45, NAN), (47, NAN), (49, float("inf"))):
        bad[r] = v
    z = moe.moe_grouped_mm_awq(bad.cuda(), w, off)
    rest = [r for r in range(50) if r not in (1, 5, 45)]
    assert torch.equal(y[rest], z[rest]) and not z[46:].any() and not torch.isfinite(z[[1, 5, 45]].float()).any()
    one = moe.Weights(moe.MOE_W_AWQ4, w.q[3:].contiguous(), w.scale[3:].contiguous(), w.zero[3:].contiguous())
    for lo, n in ((12, 1), (20, 8), (12, 34)):
        alone = moe.moe_grouped_mm_awq(x[lo:lo + n].cuda(), one, rr.offsets_of([n]).cuda())
        assert torch.equal(alone, y[lo:lo + n])


@pytest.mark.parametrize("R", [6, 60])
@pytest.mark.parametrize("off", [[0, 4, 2, 6], [0, 3, 5, 2000], [-5, 2, 4, 6], [2, 3, 4, 6], [0, 6, 6, 5], [0, 2 ** 31 - 1, 0, 1]])
def test_offsets_out_of_contract(off, R):
    """Clamped to the rows and reported; the context lives and the next call is right."""
    g = torch.Generator().manual_seed(5)
    w, values = _weights(3, 24, 128, g, [1.0])
    x = torch.randint(-4, 5, (R, 128), generator=g).to(BF)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    moe.moe_grouped_mm_awq(x.cuda(), w, torch.tensor(off, dtype=torch.int32).cuda(), dev_status=st)
    assert st.tolist() == [0, 7]
    moe.moe_grouped_mm_awq(x.cuda(), w, torch.tensor(off, dtype=torch.int32).cuda())
    sizes = [1, 0, 4]
    y = moe.moe_grouped_mm_awq(x.cuda(), w, rr.offsets_of(sizes).cuda()).cpu()
    assert torch.equal(y, rr.mm(x, values, sizes)[0].to(BF))


def test_streams_graphs_and_many_experts():
    g = torch.Generator().manual_seed(6)
    E, N, K = 1024, 16, 128
    w, values = _weights(E, N, K, g, [1.0])
    sizes = [1 if e % 37 == 5 else 0 for e in range(E)]
    R = sum(sizes)
    x, off = torch.randint(-4, 5, (R, K), generator=g).to(BF), rr.offsets_of(sizes).cuda()
    want = rr.mm(x, values, sizes)[0].to(BF).cuda()
    xc = x.cuda()
    assert torch.equal(moe.moe_grouped_mm_awq(xc, w, off), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = moe.moe_grouped_mm_awq(xc, w, off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_grouped_mm_awq(xc, w, off, y=y)
    for shift in (0, 1, 500):
        new = [sizes[(e + shift) % E] for e in range(E)]
        off.copy_(rr.offsets_of(new))
        graph.replay()
        assert torch.equal(y, rr.mm(x, values, new)[0].to(BF).cuda())
    assert moe.moe_grouped_mm_awq(xc[:0], w, off).shape == (0, N)


def test_weights_past_two_gigabytes():
    """Offsets into the codes past 32 bits: the last of many experts."""
    E, N, K = 600, 2048, 4096                                       # 2.5 GB of codes, 5e9 weights
    q = torch.zeros((E, N, K // 8), dtype=torch.int32, device="cuda")
    s, z = torch.ones((E, N, K // 128), dtype=F16, device="cuda"), torch.zeros((E, N // 8, K // 128), dtype=torch.int32, device="cuda")
    q[-1], q[-2] = 0x33333333, 0x11111111
    w = moe.Weights(moe.MOE_W_AWQ4, q, s, z)
    sizes = [0] * (E - 2) + [2, 3]
    y = moe.moe_grouped_mm_awq(torch.ones((5, K), dtype=F16, device="cuda"), w, rr.offsets_of(sizes).cuda(), out_dtype=F32)
    assert (y[:2] == K).all() and (y[2:] == 3 * K).all()

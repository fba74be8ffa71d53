"""Ragged grouped products and their gradients against the 64-bit forms.

Small-integer inputs make every sum exact, so results must equal the rounded 64-bit ones bit for bit; normal inputs are
held to the bound of FP32 sums plus one rounding.
"""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

SIZES = {
    "one": [1],
    "one_of_many": [0, 0, 1, 0, 0],
    "decode": [1, 0, 1, 1, 0, 0, 1, 1, 0, 1, 1, 1, 0],
    "none": [0, 0, 0],
    "edges": [15, 16, 17, 31, 32, 33, 0, 63, 64, 65],
    "wide": [127, 128, 129, 0, 255, 256, 257],
    "long": [1, 700, 0, 515],
}
WIDTHS = [(8, 8), (128, 64), (136, 72), (264, 520), (512, 256), (1000, 200)]


def _ints(shape, g, dt, hi=2):
    return torch.randint(-hi, hi + 1, shape, generator=g).to(dt)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _same(got, want, what):
    got = got.cpu()
    want = want.to(got.dtype)
    bad = (got != want) & ~(got.isnan() & want.isnan())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("N,K", WIDTHS)
def test_exact_on_small_integers(name, N, K):
    sizes, g = SIZES[name], _gen(len(name) + 7 * N + K)
    dt = BF if (N + K) % 16 else HF
    R, E = sum(sizes) + 3, len(sizes)                       # three padding rows
    x, w, dy = _ints((R, K), g, dt), _ints((E, N, K), g, dt), _ints((R, N), g, dt)
    off = ref.offsets_of(sizes).cuda()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    xc, wc, dc = x.cuda(), w.cuda(), dy.cuda()
    junk = lambda *s, t=dt: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    _same(moe.moe_grouped_mm(xc, wc, off, y=junk(R, N), dev_status=st), ref.mm(x, w, sizes)[0], "y")
    _same(moe.moe_grouped_mm(xc, wc, off, y=junk(R, N, t=F32), dev_status=st), ref.mm(x, w, sizes)[0], "y fp32")
    _same(moe.moe_grouped_mm_dgrad(dc, wc, off, dx=junk(R, K), dev_status=st), ref.dgrad(dy, w, sizes)[0], "dx")
    _same(moe.moe_grouped_mm_dgrad(dc, wc, off, dx=junk(R, K, t=F32), dev_status=st), ref.dgrad(dy, w, sizes)[0], "dx fp32")
    want = ref.wgrad(dy, x, sizes)[0]
    _same(moe.moe_grouped_mm_wgrad(dc, xc, off, dw=junk(E, N, K, t=F32), dev_status=st), want, "dw fp32")
    _same(moe.moe_grouped_mm_wgrad(dc, xc, off, dw=junk(E, N, K), dev_status=st), want, "dw")
    old = _ints((E, N, K), g, F32, 50)
    _same(moe.moe_grouped_mm_wgrad(dc, xc, off, dw=old.cuda(), accumulate=True, dev_status=st), want + old, "dw +=")
    assert st.tolist() == [0, 0]


@pytest.mark.parametrize("sizes", [[1], [4], [0, 2, 0, 2], [1, 0, 3], [1, 1, 1, 1], [0, 0], [5], [2, 3]])
@pytest.mark.parametrize("N,K,pad", [(8, 8, 0), (136, 264, 1), (512, 2048, 0), (1000, 7176, 0)])
def test_few_rows_exact(sizes, N, K, pad):
    """The counts around the kernel for at most four rows, padding rows among them."""
    g = _gen(N + K)
    R, E = sum(sizes) + pad, len(sizes)
    for dt in (BF, HF):
        x, w = _ints((R, K), g, dt, 1), _ints((E, N, K), g, dt, 1)
        off = ref.offsets_of(sizes).cuda()
        want = ref.mm(x, w, sizes)[0]
        for out in (dt, F32):
            y = torch.full((R, N), float("nan"), dtype=out, device="cuda")
            st = torch.zeros(2, dtype=torch.int32, device="cuda")
            _same(moe.moe_grouped_mm(x.cuda(), w.cuda(), off, y=y, dev_status=st), want, "y")
            assert st.tolist() == [0, 0]


@pytest.mark.parametrize("bad", [[0, 3, 1, 4], [-2, 1, 2, 4], [0, 1, 9, 4]])
def test_few_rows_offsets_out_of_contract(bad):
    x, w = torch.ones((4, 64), dtype=BF, device="cuda"), torch.ones((3, 32, 64), dtype=BF, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    moe.moe_grouped_mm(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), dev_status=st)
    assert st.tolist() == [0, 7]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("out", [None, F32])
@pytest.mark.parametrize("sizes,N,K", [([40, 0, 3, 300], 256, 1024), ([1, 1, 0, 1], 768, 2048), ([513], 136, 264)])
def test_normal_inputs_within_the_sums_bound(dt, out, sizes, N, K):
    g = _gen(3 * N + K)
    R, E = sum(sizes), len(sizes)
    x = torch.randn((R, K), generator=g).to(dt)
    w = (torch.randn((E, N, K), generator=g) * 0.05).to(dt)
    dy = torch.randn((R, N), generator=g).to(dt)
    off = ref.offsets_of(sizes).cuda()
    o = out or dt
    for got, (want, mag), terms in (
            (moe.moe_grouped_mm(x.cuda(), w.cuda(), off, out_dtype=out), ref.mm(x, w, sizes), K),
            (moe.moe_grouped_mm_dgrad(dy.cuda(), w.cuda(), off, out_dtype=out), ref.dgrad(dy, w, sizes), N),
            (moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off, out_dtype=o), ref.wgrad(dy, x, sizes), max(sizes))):
        assert got.dtype == o
        err = (got.cpu().double() - want).abs()
        assert (err <= ref.tolerance(want, mag, terms, o)).all(), float((err / (mag + 1e-30)).max())


def test_nan_and_infinity_stay_with_their_rows_and_experts():
    """What one expert's rows or weights hold does not reach another's results, nor do the padding rows."""
    sizes, N, K = [5, 37, 0, 70, 130], 136, 72
    E, R, g = len(sizes), sum(sizes) + 9, _gen(5)
    x, w, dy = _ints((R, K), g, BF), _ints((E, N, K), g, BF), _ints((R, N), g, BF)
    lo, hi = 42, 112                                          # expert 3's rows
    xb, db, wb = x.clone(), dy.clone(), w.clone()
    xb[lo:hi:7, ::3], db[lo + 1:hi:9, ::5], wb[3, ::4, ::2] = float("inf"), float("nan"), float("nan")
    xb[sum(sizes):], db[sum(sizes):] = float("nan"), float("inf")
    off = ref.offsets_of(sizes).cuda()
    y = moe.moe_grouped_mm(xb.cuda(), wb.cuda(), off).cpu()
    dx = moe.moe_grouped_mm_dgrad(db.cuda(), wb.cuda(), off).cpu()
    dw = moe.moe_grouped_mm_wgrad(db.cuda(), xb.cuda(), off).cpu()
    keep = torch.ones(R, dtype=torch.bool)
    keep[lo:hi] = False
    _same(y[keep], ref.mm(x, w, sizes)[0][keep], "y")
    _same(dx[keep], ref.dgrad(dy, w, sizes)[0][keep], "dx")
    others = [0, 1, 2, 4]
    _same(dw[others], ref.wgrad(dy, x, sizes)[0][others], "dw")
    assert y[lo:hi].isnan().any() and dx[lo:hi].isnan().any() and dw[3].isnan().any()
    # inside the expert, a clean row with clean weight rows keeps its value
    clean = [r for r in range(lo, hi) if (r - lo) % 7]
    _same(y[clean][:, [1, 2, 3]], ref.mm(x, w, sizes)[0][clean][:, [1, 2, 3]], "y, clean rows and columns")


def test_long_sums_do_not_drift():
    """Sums of many terms of one sign.  A part of at most 512 terms is 32 accumulator updates, each off by at most 2^-23 of
    the part; the parts are added in FP32 rounded to nearest, each addition off by at most 2^-24 of the sum so far."""
    g = _gen(17)
    R, N, K = 40_000, 32, 24
    x, dy = torch.rand((R, K), generator=g).to(BF), torch.rand((R, N), generator=g).to(BF)
    off = ref.offsets_of([R]).cuda()
    got = moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off).cpu().double()
    want = ref.wgrad(dy, x, [R])[0]
    parts = -(-R // 512)
    assert ((got - want).abs() <= (32 * 2.0 ** -23 + parts * 2.0 ** -24) * want).all()
    w, xs = torch.rand((1, N, 20_000), generator=g).to(BF), torch.rand((40, 20_000), generator=g).to(BF)
    got = moe.moe_grouped_mm(xs.cuda(), w.cuda(), ref.offsets_of([40]).cuda(), out_dtype=F32).cpu().double()
    want = ref.mm(xs, w, [40])[0]
    assert ((got - want).abs() <= (32 * 2.0 ** -23 + 40 * 2.0 ** -24) * want).all()


@pytest.mark.parametrize("dt", [BF, HF])
def test_long_contractions_with_16_bit_results(dt):
    """Past 16384 contracted elements the 16-bit results take the kernels that add parts in registers; exact sums."""
    g = _gen(18)
    sizes, N, K = [16_500, 0, 37, 900], 136, 72
    R = sum(sizes)
    x, dy = _ints((R, K), g, dt, 1), _ints((R, N), g, dt, 1)
    off = ref.offsets_of(sizes).cuda()
    want = ref.wgrad(dy, x, sizes)[0]
    dw = torch.full((4, N, K), float("nan"), dtype=dt, device="cuda")
    _same(moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off, dw=dw), want, "dw")
    old = _ints((4, N, K), g, dt, 50)
    _same(moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off, dw=old.cuda(), accumulate=True), want + old, "dw +=")
    w, xs = _ints((2, 40, 16_400), g, dt, 1), _ints((75, 16_400), g, dt, 1)
    o2 = ref.offsets_of([33, 42]).cuda()
    _same(moe.moe_grouped_mm(xs.cuda(), w.cuda(), o2), ref.mm(xs, w, [33, 42])[0], "y")
    wt = _ints((2, 16_400, 40), g, dt, 1)
    _same(moe.moe_grouped_mm_dgrad(xs.cuda(), wt.cuda(), o2), ref.dgrad(xs, wt, [33, 42])[0], "dx")


def test_same_bits_again_and_alone():
    """The same call gives the same bits, and past four rows a row's bits do not depend on the rows it is with."""
    g = _gen(11)
    sizes, N, K = [300, 20, 0, 77], 384, 640
    x, w = torch.randn((397, K), generator=g).to(BF).cuda(), torch.randn((4, N, K), generator=g).to(BF).cuda()
    off = ref.offsets_of(sizes).cuda()
    y = moe.moe_grouped_mm(x, w, off, out_dtype=F32)
    assert torch.equal(y, moe.moe_grouped_mm(x, w, off, out_dtype=F32))
    dw = moe.moe_grouped_mm_wgrad(y.to(BF), x, off)
    assert torch.equal(dw, moe.moe_grouped_mm_wgrad(y.to(BF), x, off))
    part = moe.moe_grouped_mm(x[100:330].contiguous(), w, ref.offsets_of([200, 20, 0, 10]).cuda(), out_dtype=F32)
    assert torch.equal(part, y[100:330])


def test_other_stream_and_graph_capture():
    g = _gen(12)
    sizes, N, K = [64, 1, 0, 40], 256, 128
    x, w, dy = _ints((105, K), g, BF).cuda(), _ints((4, N, K), g, BF).cuda(), _ints((105, N), g, BF).cuda()
    off = ref.offsets_of(sizes).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, dx = torch.empty((105, N), dtype=BF, device="cuda"), torch.empty((105, K), dtype=BF, device="cuda")
    dw = torch.empty((4, N, K), device="cuda")
    moe.moe_grouped_mm(x, w, off, y=y, stream=s)
    own = moe.moe_grouped_mm(x, w, off, stream=s)              # its result is allocated for that stream
    torch.cuda.current_stream().wait_stream(s)
    _same(y, ref.mm(x.cpu(), w.cpu(), sizes)[0], "y on another stream")
    _same(own, ref.mm(x.cpu(), w.cpu(), sizes)[0], "a new y on another stream")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        moe.moe_grouped_mm(x, w, off, y=y)
        moe.moe_grouped_mm_dgrad(dy, w, off, dx=dx)
        moe.moe_grouped_mm_wgrad(dy, x, off, dw=dw)
    # the graph reads the offsets and rows of the replay, not of the capture
    sizes = [0, 50, 55, 0]
    off.copy_(ref.offsets_of(sizes))
    x.copy_(_ints((105, K), g, BF))
    for t in (y, dx, dw):
        t.fill_(float("nan"))
    gr.replay()
    _same(y, ref.mm(x.cpu(), w.cpu(), sizes)[0], "y replayed")
    _same(dx, ref.dgrad(dy.cpu(), w.cpu(), sizes)[0], "dx replayed")
    _same(dw, ref.wgrad(dy.cpu(), x.cpu(), sizes)[0], "dw replayed")


def test_two_streams_at_once():
    """Calls that overlap on two streams, forward, gradients and few rows, each with the result it has alone."""
    g = _gen(19)
    jobs = []
    for sizes, N, K in (([300, 0, 77], 512, 640), ([3], 1024, 2048), ([40] * 9, 256, 512), ([1, 0, 700], 768, 256)):
        R, E = sum(sizes), len(sizes)
        x, w, dy = _ints((R, K), g, BF).cuda(), _ints((E, N, K), g, BF).cuda(), _ints((R, N), g, BF).cuda()
        jobs.append((x, w, dy, ref.offsets_of(sizes).cuda()))

    def run(job, stream=None):
        x, w, dy, off = job
        return (moe.moe_grouped_mm(x, w, off, stream=stream), moe.moe_grouped_mm_dgrad(dy, w, off, stream=stream),
                moe.moe_grouped_mm_wgrad(dy, x, off, stream=stream))

    alone = [run(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(40):
        got.append((i % 4, run(jobs[i % 4], streams[(i // 2) % 2])))
    torch.cuda.synchronize()
    for j, out in got:
        for a, b in zip(out, alone[j]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [[0, 10, 5, 20], [-3, 4, 9, 20], [0, 8, 12, 4000], [2, 8, 12, 20]])
def test_offsets_out_of_contract_are_clamped_and_reported(bad):
    g = _gen(13)
    N, K, R = 64, 128, 24
    x, w = _ints((R, K), g, BF).cuda(), _ints((3, N, K), g, BF).cuda()
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for call in (lambda st: moe.moe_grouped_mm(x, w, off, dev_status=st),
                 lambda st: moe.moe_grouped_mm_dgrad(x[:, :N].contiguous(), w, off, dev_status=st),
                 lambda st: moe.moe_grouped_mm_wgrad(x[:, :N].contiguous(), x, off, dev_status=st)):
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        call(st)
        assert st.tolist() == [0, 7]


def test_no_rows():
    w = torch.ones((3, 64, 32), dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty((0, 32), dtype=BF, device="cuda"), torch.empty((0, 64), dtype=BF, device="cuda")
    assert moe.moe_grouped_mm(x, w, off).shape == (0, 64) and moe.moe_grouped_mm_dgrad(dy, w, off).shape == (0, 32)
    dw = torch.full((3, 64, 32), 7.0, device="cuda")
    moe.moe_grouped_mm_wgrad(dy, x, off, dw=dw, accumulate=True)
    assert (dw == 7).all()
    assert (moe.moe_grouped_mm_wgrad(dy, x, off, dw=dw) == 0).all()


def test_many_experts():
    """The largest expert count, most of them without rows."""
    g = _gen(14)
    E, N, K = 1024, 16, 24
    sizes = [0] * E
    for e in (0, 5, 511, 512, 1000, 1023):
        sizes[e] = 1 + e % 40
    R = sum(sizes)
    x, w, dy = _ints((R, K), g, HF), _ints((E, N, K), g, HF), _ints((R, N), g, HF)
    off = ref.offsets_of(sizes).cuda()
    _same(moe.moe_grouped_mm(x.cuda(), w.cuda(), off), ref.mm(x, w, sizes)[0], "y")
    _same(moe.moe_grouped_mm_dgrad(dy.cuda(), w.cuda(), off), ref.dgrad(dy, w, sizes)[0], "dx")
    _same(moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off), ref.wgrad(dy, x, sizes)[0], "dw")


def test_offsets_past_32_bits_of_elements():
    """Rows and weights whose element index passes 2^31."""
    g = _gen(15)
    R, N, K, E = 300_000, 8192, 8192, 33                      # R*K and E*N*K > 2^31
    x = torch.zeros((R, K), dtype=BF, device="cuda")
    w = torch.zeros((E, N, K), dtype=BF, device="cuda")
    xt, wt = _ints((5, K), g, BF), _ints((N, K), g, BF)
    x[-5:], w[-1] = xt.cuda(), wt.cuda()
    sizes = [R - 5] + [0] * (E - 2) + [5]
    off = ref.offsets_of(sizes).cuda()
    y = moe.moe_grouped_mm(x, w, off)
    want = xt.double() @ wt.double().T
    _same(y[-5:], want, "y")
    assert not y[-4096:-5].any()
    dy = torch.zeros((R, N), dtype=BF, device="cuda")
    dt = _ints((5, N), g, BF)
    dy[-5:] = dt.cuda()
    del y
    dx = moe.moe_grouped_mm_dgrad(dy, w, off)
    _same(dx[-5:], dt.double() @ wt.double(), "dx")
    del dx
    dw = moe.moe_grouped_mm_wgrad(dy, x, off, out_dtype=BF)
    _same(dw[-1], dt.double().T @ xt.double(), "dw")
    assert not dw[0].any() and not dw[1].any()


def test_gradients_match_differences():
    """dx and dw against central differences of the 64-bit loss sum(y * dy): the loss is linear in x and in w, so the
    difference is the derivative itself."""
    g = _gen(16)
    sizes, N, K = [3, 0, 6], 16, 24
    x, w, dy = _ints((9, K), g, BF), _ints((3, N, K), g, BF), _ints((9, N), g, BF)
    off = ref.offsets_of(sizes).cuda()
    dx = moe.moe_grouped_mm_dgrad(dy.cuda(), w.cuda(), off, out_dtype=F32).cpu().double()
    dw = moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off).cpu().double()
    loss = lambda x_, w_: float((ref.mm(x_, w_, sizes)[0] * dy.double()).sum())  # noqa: E731
    for r, k in ((0, 0), (2, 5), (8, 23)):
        h = torch.zeros_like(x, dtype=torch.float64)
        h[r, k] = 1.0
        assert loss(x.double() + h, w) - loss(x.double() - h, w) == 2 * float(dx[r, k])
    for e, n, k in ((0, 0, 0), (1, 3, 3), (2, 15, 23)):
        h = torch.zeros_like(w, dtype=torch.float64)
        h[e, n, k] = 1.0
        assert loss(x, w.double() + h) - loss(x, w.double() - h) == 2 * float(dw[e, n, k])

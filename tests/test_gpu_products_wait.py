"""A wait that runs out in the ragged and 4-bit products is reported, whichever role's it is.  The debug build makes the
thread that issues the MMAs wait, from its pair's second tile on, for a barrier that nothing arrives on: the wait gives up
after its limit (about 2 s), the call ends with MOE_ERR_TIMEOUT in dev_status[1], and the context stays usable."""
import pytest
import torch

import top_moe_expert_gb300 as moe
from tests import gpu_setup as gs
from tests import ragged_ref as ref
from top_moe_expert_gb300 import build

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MOE_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def debug():
    gs.need_gpu()
    moe.use_library(build.build(debug=True))
    yield moe.lib()
    moe.use_library(build.LIB)


def _calls():
    """Products of two tiles for some pairs of CTAs (and one for the rest), each (call, its result)."""
    g = torch.Generator().manual_seed(1)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    C, J = 256 * (sms // 2 + 4), 256                          # 4 tiles more than pairs
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(BF)  # noqa: E731
    sizes = [40]
    off = ref.offsets_of(sizes).cuda()
    x, w, wt, dy = ints(40, J), ints(1, C, J), ints(1, J, C), ints(40, C)
    for out in (BF, F32):
        yield lambda st, out=out: moe.moe_grouped_mm(x.cuda(), w.cuda(), off, out_dtype=out, dev_status=st), ref.mm(x, w, sizes)[0]
        yield (lambda st, out=out: moe.moe_grouped_mm_dgrad(x.cuda(), wt.cuda(), off, out_dtype=out, dev_status=st),
               ref.dgrad(x, wt, sizes)[0])
        yield (lambda st, out=out: moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), off, out_dtype=out, dev_status=st),
               ref.wgrad(dy, x, sizes)[0])
    xq, wq = (torch.randint(0, 256, s, generator=g, dtype=torch.int32).to(torch.uint8) for s in ((40, J // 2), (1, C, J // 2)))
    xs, ws = torch.full((40, 16), 127, dtype=torch.uint8), torch.full((1, C, 16), 127, dtype=torch.uint8)
    xs[:, J // 32:], ws[:, :, J // 32:] = 0, 0
    mx = moe.MOE_FP4_MXFP4
    want = ref.mm(torch.from_numpy(ref.values(xq, xs, mx)), torch.from_numpy(ref.values(wq, ws, mx)), sizes)[0]
    yield (lambda st: moe.moe_grouped_mm_fp4(moe.Fp4(mx, xq.cuda(), xs.cuda()), moe.Fp4(mx, wq.cuda(), ws.cuda()), off,
                                             out_dtype=F32, dev_status=st), want)


def test_an_expired_wait_is_reported(debug):
    for i, (call, want) in enumerate(_calls()):
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        assert debug.moe_debug_products_stall(1) == 0
        try:
            call(st)
            torch.cuda.synchronize()
        finally:
            debug.moe_debug_products_stall(0)
        assert st.tolist() == [0, MOE_ERR_TIMEOUT], i
        st.zero_()
        y = call(st)
        assert st.tolist() == [0, 0], i
        assert torch.equal(y.cpu(), want.to(y.dtype)), i


def test_the_hook_checks_its_argument(debug):
    assert debug.moe_debug_products_stall(2) == 1 and debug.moe_debug_products_stall(-1) == 1


def test_ragged_tails_far_apart():
    """A weight gradient whose ragged experts come after hundreds of tiles without a tail (the release build)."""
    moe.use_library(build.LIB)
    g = torch.Generator().manual_seed(2)
    sizes = ([64] * 200 + [37] + [0] * 50 + [16] * 100 + [1]) * 2
    R, E, N, K = sum(sizes) + 5, len(sizes), 256, 264
    x, dy = (torch.randint(-2, 3, (R, c), generator=g).to(BF) for c in (K, N))
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    for out in (BF, F32):
        dw = moe.moe_grouped_mm_wgrad(dy.cuda(), x.cuda(), ref.offsets_of(sizes).cuda(), out_dtype=out, dev_status=st)
        assert torch.equal(dw.cpu(), ref.wgrad(dy, x, sizes)[0].to(out))
    assert st.tolist() == [0, 0]

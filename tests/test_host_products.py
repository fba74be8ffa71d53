"""Arithmetic that the ragged and 4-bit products share between host and device, run on the CPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_products.cu")
CSRC = os.path.join(ROOT, "top_moe_expert_gb300", "csrc")
INCLUDE = os.path.join(ROOT, "include")
DEPS = [SRC, *(os.path.join(CSRC, n) for n in ("fp4.cuh", "ragged.cuh", "common.cuh"))]
OUT = os.path.join(ROOT, "top_moe_expert_gb300", "_build", "host_products.so")


@pytest.fixture(scope="module")
def emu():
    nvcc = next((c for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc")
                 if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    t = max(os.path.getmtime(p) for p in DEPS)
    if not os.path.exists(OUT) or os.path.getmtime(OUT) < t:
        os.makedirs(os.path.dirname(OUT), exist_ok=True)
        subprocess.run([nvcc, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared",
                        "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC, "-I", INCLUDE, SRC, "-o", OUT],
                       check=True, capture_output=True)
    return ctypes.CDLL(OUT)


def _factors(emu, a, b):
    f, g = np.empty_like(a), np.empty_like(a)
    p = lambda t: t.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    emu.fp4_factors(ctypes.c_int64(a.size), p(a), p(b), p(f), p(g))
    return f, g


def test_two_constants_over_their_whole_range(emu):
    """v * f * g of sums v (2^-20 .. 2^54) and constants from 2^-100 to 2^100: the value to three roundings wherever FP32
    holds it, the bits of v * (a * b) where nothing on the way leaves FP32's normal range, 0 for 0."""
    r = np.random.default_rng(1)
    n = 400_000
    f32 = np.float32
    a, b = (np.ldexp(1 + r.random(n), r.integers(-100, 100, n)).astype(f32) for _ in range(2))
    v = (np.ldexp(1 + r.random(n), r.integers(-20, 54, n)) * r.choice([-1, 1], n)).astype(f32)
    f, g = _factors(emu, a, b)
    with np.errstate(over="ignore", under="ignore"):
        got = v * f * g
        plain = v * (a * b)
        want = v.astype(np.float64) * a.astype(np.float64) * b.astype(np.float64)
        ab = a.astype(np.float64) * b
        fits = np.abs(want) < 3.4e38
        tol = 3.01 * 2.0 ** -24 * np.abs(want) + 2.0 ** -150
        assert (np.abs(got - want) <= tol)[fits].all()
        assert np.isinf(got[np.abs(want) > 3.41e38]).all()
        normal = fits & (np.abs(want) > 2.0 ** -125) & (ab > 2.0 ** -125) & (ab < 2.0 ** 127)
        assert normal.sum() > n // 4 and np.array_equal(got[normal], plain[normal])
        lost = fits & (np.abs(want) > 2.0 ** -125) & ~normal
        assert lost.sum() > n // 50                          # a * b alone would have left FP32's normal range
        assert not (f32(0) * f * g).any()


def test_zero_and_special_constants(emu):
    a = np.array([0, 0, 1, np.nan, np.inf, 2.0 ** -126, 2.0 ** 127], dtype=np.float32)
    b = np.array([0, 2.0 ** 100, 0, 1, 2.0 ** -100, 1, 2.0 ** -100], dtype=np.float32)
    f, g = _factors(emu, a, b)
    y = np.float32(3) * f * g
    assert not y[:3].any() and np.isnan(y[3]) and np.isposinf(y[4])
    assert y[5] == np.float32(3 * 2.0 ** -126) and y[6] == np.float32(3 * 2.0 ** 27)


def test_a_limit_runs_from_the_last_progress(emu):
    """A wait much longer than the limit goes on while the other role moves, however slowly, and ends a limit after it
    last did."""
    emu.limit_expires.restype = ctypes.c_int64
    limit, n = 5_000_000_000, 4000
    now = np.arange(n, dtype=np.int64) * 100_000_000            # 80 limits
    p = lambda t: t.ctypes.data_as(ctypes.c_void_p)  # noqa: E731

    def expires(progress):
        t = progress.astype(np.int32)
        return emu.limit_expires(ctypes.c_int64(n), p(now), p(t), ctypes.c_int64(limit))

    assert expires(np.zeros(n)) == 51
    assert expires(np.arange(n)) == n and expires(np.arange(n) // 50) == n
    assert expires(np.minimum(np.arange(n), 1000)) == 1051
    assert expires(np.arange(n) // 60) == 51                    # a role that rests for longer than the limit
    wrap = (np.arange(n) + 2 ** 31 - 100).astype(np.int64).astype(np.uint32).astype(np.int64)
    assert expires(np.where(wrap >= 2 ** 31, wrap - 2 ** 32, wrap)) == n


def test_arrivals_on_another_cta_name_their_scope():
    """An mbarrier arrival without a scope is ordered at CTA scope, which on a barrier of another CTA of the cluster does not
    order what it announces for the thread that waits there: each says which one it means, and wgrad's takes the cluster's."""
    import glob
    import re
    arrivals = []
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        code = re.sub(r"//[^\n]*", "", open(path).read())
        arrivals += [(os.path.basename(path), m) for m in re.findall(r"mbarrier\.arrive[\w.:]*", code) if "shared::cluster" in m]
    assert arrivals
    for path, a in arrivals:
        assert re.search(r"\.(release|relaxed)\.(cta|cluster)\.", a) or "commit" in a, (path, a)
    assert "mbar_arrive_cluster_smem" not in open(os.path.join(CSRC, "gmm.cu")).read()

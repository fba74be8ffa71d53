"""The grouped products' tile order, run on the CPU: every tile of a grid exactly once, and tiles that follow one another
near each other (within a band of eight along the weights' rows)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_ragged.cu")
CSRC = os.path.join(ROOT, "top_moe_expert_gb300", "csrc")
INCLUDE = os.path.join(ROOT, "include")
DEPS = [SRC, os.path.join(CSRC, "ragged.cuh"), os.path.join(CSRC, "common.cuh")]
OUT = os.path.join(ROOT, "top_moe_expert_gb300", "_build", "host_ragged.so")


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
    L = ctypes.CDLL(OUT)
    L.place_all.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return L


@pytest.mark.parametrize("n_mt", [*range(1, 27), 32, 33, 255])
def test_every_tile_once_in_bands(emu, n_mt):
    for n_nt in (1, 2, 3, 7, 8, 40):
        out = np.full((n_mt * n_nt, 2), -1, dtype=np.int32)
        emu.place_all(n_mt, n_nt, out.ctypes.data_as(ctypes.c_void_p))
        seen = out[:, 0].astype(np.int64) * n_nt + out[:, 1]
        assert np.array_equal(np.sort(seen), np.arange(n_mt * n_nt))
        assert out.min() >= 0 and (out[:, 0] < n_mt).all() and (out[:, 1] < n_nt).all()
        band = out[:, 0] // 8
        assert (np.diff(band) >= 0).all()
        for b in np.unique(band):                          # inside a band: along nt, every mt of the band each time
            nt = out[band == b, 1]
            width = min(8, n_mt - 8 * b)
            assert np.array_equal(nt, np.repeat(np.arange(n_nt), width))

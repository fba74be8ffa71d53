"""Plain 64-bit forms of the ragged grouped products and of NVFP4 / MXFP4, for the tests (torch on the CPU)."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NVFP4, MXFP4 = 0, 1
BLOCK = {NVFP4: 16, MXFP4: 32}


def offsets_of(sizes) -> torch.Tensor:
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32)


def mm(x, w, sizes):
    """(y, sum of the terms' magnitudes): rows of x [R, K] by w [E, N, K]; rows past the groups are zero."""
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64)
    a = torch.zeros_like(y)
    lo = 0
    for e, n in enumerate(sizes):
        if n:
            y[lo:lo + n] = x[lo:lo + n].double() @ w[e].double().T
            a[lo:lo + n] = x[lo:lo + n].double().abs() @ w[e].double().abs().T
        lo += n
    return y, a


def dgrad(dy, w, sizes):
    return mm(dy, w.transpose(1, 2), sizes)


def wgrad(dy, x, sizes):
    E = len(sizes)
    dw = torch.zeros((E, dy.shape[1], x.shape[1]), dtype=torch.float64)
    a = torch.zeros_like(dw)
    lo = 0
    for e, n in enumerate(sizes):
        d, v = dy[lo:lo + n].double(), x[lo:lo + n].double()
        dw[e] = d.T @ v
        a[e] = d.abs().T @ v.abs()
        lo += n
    return dw, a


def tolerance(ref, mag, terms, dtype):
    """terms FP32 additions in any order, each off by at most one unit of 2^-23 of the magnitudes' sum, then one
    rounding to dtype (half a step, and half of the smallest subnormal step of fp16)."""
    tol = terms * 2.0 ** -23 * mag
    if dtype != torch.float32:
        tol = tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol)
        if dtype == torch.float16:
            tol = tol + 2.0 ** -25
    return tol + 1e-37


# ---------------------------------------------------------------- 4-bit floats

def _round_grid(a, mantissa, emin, top):
    """Nearest value, ties to even, of the float grid with `mantissa` fraction bits and smallest exponent emin."""
    a = np.asarray(a, dtype=np.float64)
    _, e = np.frexp(np.where(a > 0, a, 1.0))
    step = np.ldexp(1.0, np.maximum(e - 1, emin) - mantissa)
    return np.minimum(np.rint(a / step) * step, top)


def ue4m3_byte(v):
    """Byte of a value that is on the UE4M3 grid."""
    v = np.asarray(v, dtype=np.float64)
    m, e = np.frexp(np.where(v > 0, v, 1.0))
    e = e - 1
    sub = v < 2.0 ** -6
    return np.where(sub, np.rint(v * 512), ((e + 7) << 3) + np.rint((2 * m - 1) * 8)).astype(np.int64)


def ue4m3_value(b):
    b = np.asarray(b, dtype=np.int64)
    e, m = b >> 3, b & 7
    v = np.where(e > 0, (1 + m / 8) * np.ldexp(1.0, e - 7), m / 512)
    return np.where(b == 0x7F, np.nan, v)


def quantize(v, fmt, alpha=None):
    """(q [rows, K/2], s [rows, Ks]) of v [rows, K] (float64 holding the input type's values); alpha [groups] float32."""
    rows, K = v.shape
    b = BLOCK[fmt]
    x = np.asarray(v, dtype=np.float64).reshape(rows, K // b, b)
    bad = ~np.isfinite(x).all(axis=2)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(axis=2)
    if fmt == NVFP4:
        f32 = np.float32
        a = np.repeat(np.asarray(alpha, dtype=f32), rows // len(alpha))[:, None]
        with np.errstate(all="ignore"):
            r = f32(1) / (f32(6) * a)
            S = _round_grid((amax.astype(f32) * r).astype(np.float64), 3, -6, 448.0)
            S = np.where(amax > 0, S, 0.0)
            inv = np.where(S > 0, f32(1) / (a * S.astype(f32)), f32(0)).astype(f32)
            t = (x.astype(f32) * inv[..., None]).astype(np.float64)
        byte = ue4m3_byte(S)
        byte = np.where(bad, 0x7F, byte)
    else:
        _, e = np.frexp(np.where(amax > 0, amax, 1.0))
        X = np.where(amax > 0, np.clip(e - 3, -127, 127), -127)
        t = np.ldexp(x, -X[..., None])
        byte = np.where(bad, 0xFF, X + 127)
    code = np.searchsorted(E2M1, _round_grid(np.abs(t), 1, 0, 6.0))
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(x)).reshape(rows, K // 2, 2)
    s = np.zeros((rows, (K // b + 15) // 16 * 16), dtype=np.uint8)
    s[:, :K // b] = byte
    return (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8), s


def values(q, s, fmt):
    """Scale times code (float64, exact; NaN scales give NaN), without alpha."""
    q, s = np.asarray(q), np.asarray(s)
    K, b = q.shape[-1] * 2, BLOCK[fmt]
    nib = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], K)
    v = E2M1[nib & 7] * np.where(nib >= 8, -1.0, 1.0)
    sb = s[..., :K // b].astype(np.int64)
    f = ue4m3_value(sb) if fmt == NVFP4 else np.where(sb == 255, np.nan, np.ldexp(1.0, sb - 127))
    return v * np.repeat(f, b, axis=-1)

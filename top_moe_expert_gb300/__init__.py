"""top_moe_expert_gb300 -- GB300 (sm_103a) routed MoE expert-FFN layer.

A thin ctypes binding over the C ABI of ``libmoe_ffn.so`` (declared in
``include/moe_ffn.h``).  The functions here carry the same names as the C
entry points and only marshal arguments: PyTorch supplies device memory and
the current CUDA stream; every step of the layer runs in the library's CUDA
kernels.  There is no fallback: if the library is not built, or no GPU is
present, calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_ffn.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_CAPACITY", 4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA",
                6: "MOE_ERR_TIMEOUT", 7: "MOE_ERR_BOUNDS"}
MOE_W_MXFP8, MOE_W_AWQ4, MOE_W_NVFP4S = 0, 1, 3
MOE_BF16, MOE_FP16, MOE_FP32 = 0, 1, 2
MOE_PATH_DECODE, MOE_PATH_GROUPED = 0, 1
MOE_FP4_NVFP4, MOE_FP4_MXFP4 = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1

_DT = {torch.bfloat16: MOE_BF16, torch.float16: MOE_FP16, torch.float32: MOE_FP32}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class moe_weights_t(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("zero", ctypes.c_void_p), ("alpha", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None

_I32, _I64, _P, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_PROTOS = {
    "moe_status_string": (ctypes.c_char_p, [_I32]),
    "moe_abi_version": (_I32, []),
    "moe_ffn_select_path": (_I32, [_I32, _I32, _I32, _I32, _I32, _I32, _P, _P]),
    "moe_topk_softmax": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_align_capacity": (_I32, [_I32, _I32, _I32, _I32, _P, _P]),
    "moe_align_workspace_size": (_I32, [_I32, _I32, _I32, _I32, _P]),
    "moe_align_block_size": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _I32, _I32, _P, _SZ, _P, _P]),
    "moe_mxfp8_quantize": (_I32, [_P, _I32, _I64, _I32, _P, _P, _P]),
    "moe_ffn_decode_workspace_size": (_I32, [_I32, _I32, _I32, _I32, _P]),
    "moe_ffn_decode": (_I32, [_P, _I32, _I32, _I32, _P, _P, _I32, ctypes.POINTER(moe_weights_t),
                              ctypes.POINTER(moe_weights_t), _P, _I32, _P, _SZ, _P, _P]),
    "moe_ffn_decode_logits": (_I32, [_P, _P, _I32, _I32, _I32, _I32, ctypes.POINTER(moe_weights_t),
                                     ctypes.POINTER(moe_weights_t), _P, _P, _P, _I32, _P, _SZ, _P, _P]),
    "moe_grouped_prepare_size": (_I32, [ctypes.POINTER(moe_weights_t), ctypes.POINTER(moe_weights_t), _P, _P]),
    "moe_grouped_prepare": (_I32, [ctypes.POINTER(moe_weights_t), ctypes.POINTER(moe_weights_t), _P, _P, _P]),
    "moe_grouped_prepare_nvfp4s": (_I32, [ctypes.POINTER(moe_weights_t), ctypes.POINTER(moe_weights_t),
                                          ctypes.c_float, ctypes.c_float, _P, _P, _P]),
    "moe_ffn_grouped_workspace_size": (_I32, [_I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "moe_ffn_grouped": (_I32, [_P, _I32, _I32, _I32, _P, _P, _I32, ctypes.POINTER(moe_weights_t),
                               ctypes.POINTER(moe_weights_t), _P, _P, _P, _P, _P, _I32, _I32, _P, _I32,
                               _P, _SZ, _P, _P]),
    "moe_ffn_decode_noalloc": (_I32, [_P, _I32, _I32, _I32, _P, _P, _I32, ctypes.POINTER(moe_weights_t),
                                      ctypes.POINTER(moe_weights_t), _P, _I32, _P, _P]),
    "moe_debug_exchange_stall": (_I32, [_I32]),
    "moe_ep_local_routes": (_I32, [_P, _I64, _I32, _I32, _P, _P]),
    "moe_align_fixed_capacity": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P]),
    "moe_ffn_grouped_batched": (_I32, [_P, _I32, _I32, _I32, _P, _P, _I32, ctypes.POINTER(moe_weights_t),
                                       ctypes.POINTER(moe_weights_t), _P, _P, _P, _P, _P, _P, _I32, _I32, _P,
                                       _I32, _P, _SZ, _P, _P]),
    "moe_grouped_mm": (_I32, [_P, _P, _I32, _P, _I32, _I32, _I32, _I32, _P, _I32, _P, _P]),
    "moe_grouped_mm_dgrad": (_I32, [_P, _P, _I32, _P, _I32, _I32, _I32, _I32, _P, _I32, _P, _P]),
    "moe_grouped_mm_wgrad": (_I32, [_P, _P, _I32, _P, _I32, _I32, _I32, _I32, _P, _I32, _I32, _P, _P]),
    "moe_route": (_I32, [_P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _P, _P, _P]),
    "moe_route_bwd": (_I32, [_P, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _P]),
    "moe_swiglu_dropout": (_I32, [_P, _I32, _I32, _I32, ctypes.c_double, _P, _P, _P]),
    "moe_swiglu_dropout_bwd": (_I32, [_P, _P, _I32, _I32, _I32, ctypes.c_double, _P, _P, _P]),
    "moe_grouped_mm_awq": (_I32, [_P, _I32, ctypes.POINTER(moe_weights_t), _P, _I32, _P, _I32, _P, _P]),
    "moe_fp4_scale_cols": (_I32, [_I32, _I32, _P]),
    "moe_fp4_quantize": (_I32, [_P, _I32, _I64, _I32, _I32, _P, _I64, _P, _P, _P]),
    "moe_fp4_dequantize": (_I32, [_P, _P, _I64, _I32, _I32, _P, _I64, _P, _I32, _P]),
    "moe_grouped_mm_fp4": (_I32, [_P, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _I32, _I32, _P, _I32, _P, _P]),
}


def use_library(path: str) -> None:
    """Load the library at `path` for the calls that follow (for example the
    debug bounds-check build, build.LIB_DEBUG); the same entry points."""
    global _lib, LIB_PATH
    with _lock:
        LIB_PATH = path
        _lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe_ffn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m top_moe_expert_gb300.build` (no CPU fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _PROTOS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


# Every pointer handed to the library is checked first: a host tensor, a
# tensor on another GPU, a strided view, a wrong element type or a short
# output buffer would otherwise reach a kernel as a bad address or a bad
# size.  The checks raise ValueError; nothing is launched.

def _is_gpu(t: torch.Tensor) -> bool:
    return t.is_cuda


def _need(t, name: str, dtypes=None, shape=None, min_numel=None, device=None):
    """Check one tensor argument: a contiguous CUDA tensor on `device`, of one
    of `dtypes`, of exactly `shape` or at least `min_numel` elements."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor, not {type(t).__name__}")
    if not _is_gpu(t):
        raise ValueError(f"{name} must be a CUDA tensor (it is on {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}; the call's tensors are on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements; the call needs at least {min_numel}")
    return t


def _dev(t: torch.Tensor, name: str):
    _need(t, name)


def _opt(t, name: str, **kw):
    """_need for an optional argument (None passes)."""
    if t is not None:
        _need(t, name, **kw)
    return t


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _guard(device):
    """Make the tensors' GPU current for the call (the library launches on
    the current device)."""
    if device.type != "cuda" or device.index == torch.cuda.current_device():
        return _NO_GUARD
    return torch.cuda.device(device)


_NO_GUARD = contextlib.nullcontext()


# torch's own handles without the objects around them; a torch without CUDA, on
# which the host-only functions run, has neither.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda gpu: torch.cuda.current_stream(gpu).cuda_stream)
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None, device=None):
    """The stream handle: `stream`, or the current stream of `device`."""
    if stream is None:
        # the handle alone: a Stream object costs more than a small launch
        return _raw_stream(torch.cuda.current_device() if device is None else device.index)
    sd = getattr(stream, "device", None)
    if device is not None and sd is not None and sd != device:
        raise ValueError(f"stream is on {sd}; the call's tensors are on {device}")
    return stream.cuda_stream


_IDS = (torch.int32,)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_YDT = (torch.bfloat16, torch.float32)


@dataclasses.dataclass(frozen=True)
class Weights:
    """One projection of all experts: MXFP8 (q uint8 [E,N,K], scale uint8
    [E,N,K/32]) or AWQ4 (q int32 [E,N,K/8], scale fp16 [E,N,K/128],
    zero int32 [E,N/8,K/128]) or NVFP4S, paired 4:8 sparse NVFP4 (q uint8
    [E,N,K/4] kept E2M1 codes, scale uint8 [E,N,K/32] UE4M3, zero uint8
    [E,N,K/16] pattern nibbles, alpha float32 [E]).  The tensors are checked against the format
    when the object is made (device, contiguity, dtype, shapes), and the
    object is immutable, so the layer calls only compare its device."""
    fmt: int
    q: torch.Tensor
    scale: torch.Tensor
    zero: torch.Tensor | None = None
    alpha: torch.Tensor | None = None

    def __post_init__(self):
        object.__setattr__(self, "device", self._check())
        object.__setattr__(self, "_struct", moe_weights_t(
            self.fmt, self.E, self.N, self.K, self.q.data_ptr(), self.scale.data_ptr(),
            self.zero.data_ptr() if self.zero is not None else None,
            self.alpha.data_ptr() if self.alpha is not None else None))

    @property
    def E(self):
        return self.q.shape[0]

    @property
    def N(self):
        return self.q.shape[1]

    @property
    def K(self):
        return self.q.shape[2] * {MOE_W_AWQ4: 8, MOE_W_NVFP4S: 4}.get(self.fmt, 1)

    def _check(self):
        q = _need(self.q, "weights.q")
        device = q.device
        if q.dim() != 3:
            raise ValueError(f"weights.q must be 3-D [E, ., .], not {tuple(q.shape)}")
        E, N, K = self.E, self.N, self.K
        if self.fmt == MOE_W_MXFP8:
            _need(q, "weights.q", _U8)
            if K % 32:
                raise ValueError(f"weights: K = {K} is not a multiple of 32")
            _need(self.scale, "weights.scale", _U8, (E, N, K // 32), device=device)
        elif self.fmt == MOE_W_AWQ4:
            _need(q, "weights.q", _IDS)
            if K % 128 or N % 8:
                raise ValueError(f"weights: AWQ needs K % 128 == 0 and N % 8 == 0 (K = {K}, N = {N})")
            _need(self.scale, "weights.scale", (torch.float16,), (E, N, K // 128), device=device)
            if self.zero is None:
                raise ValueError("weights.zero is required for AWQ weights")
            _need(self.zero, "weights.zero", _IDS, (E, N // 8, K // 128), device=device)
        elif self.fmt == MOE_W_NVFP4S:
            _need(q, "weights.q", _U8)
            if K % 64:
                raise ValueError(f"weights: NVFP4S needs K % 64 == 0 (K = {K})")
            _need(self.scale, "weights.scale", _U8, (E, N, K // 32), device=device)
            if self.zero is None or self.alpha is None:
                raise ValueError("weights.zero (patterns) and weights.alpha are required for NVFP4S weights")
            _need(self.zero, "weights.zero", _U8, (E, N, K // 16), device=device)
            _need(self.alpha, "weights.alpha", _F32, (E,), device=device)
        else:
            raise ValueError(f"weights: unknown format {self.fmt}")
        if self.fmt not in (MOE_W_AWQ4, MOE_W_NVFP4S) and self.zero is not None:
            raise ValueError("weights.zero must be None for MXFP8 weights")
        if self.fmt != MOE_W_NVFP4S and self.alpha is not None:
            raise ValueError("weights.alpha is only for NVFP4S weights")
        return device

    def on(self, name: str, device):
        """Raise unless the weights live on `device`."""
        if self.device != device:
            raise ValueError(f"{name} is on {self.device}; the call's tensors are on {device}")

    def c_struct(self) -> moe_weights_t:
        return self._struct


# ---------------------------------------------------------------- routing

def moe_topk_softmax(logits: torch.Tensor, k: int, topk_ids=None, topk_w=None, stream=None):
    _need(logits, "logits", _F32)
    if logits.dim() != 2:
        raise ValueError(f"logits must be [M, E], not {tuple(logits.shape)}")
    dev = logits.device
    M, E = logits.shape
    ids = topk_ids if topk_ids is not None else torch.empty((M, k), dtype=torch.int32, device=dev)
    w = topk_w if topk_w is not None else torch.empty((M, k), dtype=torch.float32, device=dev)
    _need(ids, "topk_ids", _IDS, (M, k), device=dev)
    _need(w, "topk_w", _F32, (M, k), device=dev)
    with _guard(dev):
        _check(lib().moe_topk_softmax(_ptr(logits), M, E, k, _ptr(ids), _ptr(w), _stream(stream, dev)),
               "moe_topk_softmax")
    return ids, w


def moe_ep_local_routes(topk_ids: torch.Tensor, e_lo: int, e_hi: int, local_ids=None, stream=None):
    """The routing as seen by the rank that owns experts [e_lo, e_hi): ids
    of its experts shifted to 0 .. e_hi - e_lo - 1, every other id -1 (an
    invalid route the layer skips)."""
    _need(topk_ids, "topk_ids", _IDS)
    dev = topk_ids.device
    out = local_ids if local_ids is not None else torch.empty_like(topk_ids)
    _need(out, "local_ids", _IDS, tuple(topk_ids.shape), device=dev)
    with _guard(dev):
        _check(lib().moe_ep_local_routes(_ptr(topk_ids), topk_ids.numel(), int(e_lo), int(e_hi), _ptr(out),
                                         _stream(stream, dev)), "moe_ep_local_routes")
    return out


# ---------------------------------------------------------------- alignment

def moe_ffn_select_path(M: int, k: int, E: int, d: int, I: int, fmt: int = None):
    """(path, b): MOE_PATH_DECODE with b = 0, or MOE_PATH_GROUPED with the
    block size for alignment, at the measured crossover of the two paths."""
    fmt = MOE_W_MXFP8 if fmt is None else fmt
    p, b = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_ffn_select_path(M, k, E, d, I, fmt, ctypes.byref(p), ctypes.byref(b)), "moe_ffn_select_path")
    return p.value, b.value


def moe_debug_exchange_stall(on: bool) -> None:
    """Failure-detection test hook: the single-token one-kernel launches that
    follow wait for h values tagged with a tag no CTA writes, so their bounded
    wait runs out and reports MOE_ERR_TIMEOUT in dev_status[1]; False
    restores normal operation."""
    _check(lib().moe_debug_exchange_stall(1 if on else 0), "moe_debug_exchange_stall")


def moe_align_capacity(M: int, k: int, E: int, b: int):
    cr, cb = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_align_capacity(M, k, E, b, ctypes.byref(cr), ctypes.byref(cb)), "moe_align_capacity")
    return cr.value, cb.value


def moe_align_workspace_size(M: int, k: int, E: int, b: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_align_workspace_size(M, k, E, b, ctypes.byref(n)), "moe_align_workspace_size")
    return n.value


def moe_align_block_size(topk_ids: torch.Tensor, E: int, b: int, cap_rows=None, cap_blocks=None,
                         out=None, ws=None, dev_status=None, stream=None):
    """Returns (sorted_route_ids [cap_rows], expert_ids [cap_blocks],
    num_rows_post_pad [1]) as int32 device tensors."""
    _need(topk_ids, "topk_ids", _IDS)
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids must be [M, k], not {tuple(topk_ids.shape)}")
    M, k = topk_ids.shape
    dev = topk_ids.device
    if out is None:
        cr, cb = moe_align_capacity(M, k, E, b)
        cap_rows = cr if cap_rows is None else cap_rows
        cap_blocks = cb if cap_blocks is None else cap_blocks
        out = (torch.empty(cap_rows, dtype=torch.int32, device=dev),
               torch.empty(cap_blocks, dtype=torch.int32, device=dev),
               torch.empty(1, dtype=torch.int32, device=dev))
    else:
        # capacities default to the given buffers' lengths
        cap_rows = out[0].numel() if cap_rows is None else cap_rows
        cap_blocks = out[1].numel() if cap_blocks is None else cap_blocks
    _need(out[0], "sorted_route_ids", _IDS, min_numel=cap_rows, device=dev)
    _need(out[1], "expert_ids", _IDS, min_numel=cap_blocks, device=dev)
    _need(out[2], "num_rows_post_pad", _IDS, min_numel=1, device=dev)
    need = moe_align_workspace_size(M, k, E, b)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _opt(ws, "ws", device=dev)
    _opt(dev_status, "dev_status", dtypes=_IDS, min_numel=2, device=dev)
    with _guard(dev):
        _check(lib().moe_align_block_size(_ptr(topk_ids), M, k, E, b, _ptr(out[0]), _ptr(out[1]), _ptr(out[2]),
                                          cap_rows, cap_blocks, _ptr(ws), _nbytes(ws), _ptr(dev_status),
                                          _stream(stream, dev)), "moe_align_block_size")
    return out


def moe_align_fixed_capacity(topk_ids: torch.Tensor, E: int, b: int, C: int, out=None, dev_status=None,
                             stream=None):
    """Fixed-capacity layout: returns (sorted_route_ids [E*C], expert_ids
    [E*C/b], block_rows [E*C/b], num_rows_post_pad [1]) as int32 device
    tensors; C (a multiple of b) must be at least every expert's route count."""
    _need(topk_ids, "topk_ids", _IDS)
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids must be [M, k], not {tuple(topk_ids.shape)}")
    if b < 1 or C < b or C % b:
        raise ValueError(f"capacity C = {C} must be a positive multiple of b = {b}")
    M, k = topk_ids.shape
    dev = topk_ids.device
    rows, blocks = E * C, E * C // b
    if out is None:
        out = (torch.empty(rows, dtype=torch.int32, device=dev), torch.empty(blocks, dtype=torch.int32, device=dev),
               torch.empty(blocks, dtype=torch.int32, device=dev), torch.empty(1, dtype=torch.int32, device=dev))
    _need(out[0], "sorted_route_ids", _IDS, (rows,), device=dev)
    _need(out[1], "expert_ids", _IDS, (blocks,), device=dev)
    _need(out[2], "block_rows", _IDS, (blocks,), device=dev)
    _need(out[3], "num_rows_post_pad", _IDS, min_numel=1, device=dev)
    _opt(dev_status, "dev_status", dtypes=_IDS, min_numel=2, device=dev)
    with _guard(dev):
        _check(lib().moe_align_fixed_capacity(_ptr(topk_ids), M, k, E, b, C, _ptr(out[0]), _ptr(out[1]),
                                              _ptr(out[2]), _ptr(out[3]), _ptr(dev_status), _stream(stream, dev)),
               "moe_align_fixed_capacity")
    return out


# ---------------------------------------------------------------- quantization

def moe_mxfp8_quantize(v: torch.Tensor, q=None, s=None, stream=None):
    """MXFP8 codes and E8M0 scales of v [rows, K] (fp32 or bf16)."""
    _need(v, "v", (torch.float32, torch.bfloat16))
    dev = v.device
    K = v.shape[-1]
    if K % 32:
        raise ValueError(f"v's last dimension ({K}) is not a multiple of 32")
    rows = v.numel() // K if K else 0
    q = q if q is not None else torch.empty(v.shape, dtype=torch.uint8, device=dev)
    s = s if s is not None else torch.empty((*v.shape[:-1], K // 32), dtype=torch.uint8, device=dev)
    _need(q, "q", _U8, min_numel=rows * K, device=dev)
    _need(s, "s", _U8, min_numel=rows * (K // 32), device=dev)
    with _guard(dev):
        _check(lib().moe_mxfp8_quantize(_ptr(v), _DT[v.dtype], rows, K, _ptr(q), _ptr(s), _stream(stream, dev)),
               "moe_mxfp8_quantize")
    return q, s


def _layer_args(x, topk_ids, topk_w, w13: Weights, w2: Weights, y, out_dtype, dev_status):
    """Check the common arguments of the layer calls; returns (device, M, d,
    k, y) with y allocated when not given."""
    _need(x, "x", tuple(_DT))
    if x.dim() != 2:
        raise ValueError(f"x must be [M, d], not {tuple(x.shape)}")
    dev = x.device
    M, d = x.shape
    _need(topk_ids, "topk_ids", _IDS, device=dev)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != M:
        raise ValueError(f"topk_ids must be [M={M}, k], not {tuple(topk_ids.shape)}")
    k = topk_ids.shape[1]
    _need(topk_w, "topk_w", _F32, (M, k), device=dev)
    w13.on("w13", dev)
    w2.on("w2", dev)
    y = y if y is not None else torch.empty((M, d), dtype=out_dtype, device=dev)
    _need(y, "y", _YDT, (M, d), device=dev)
    _opt(dev_status, "dev_status", dtypes=_IDS, min_numel=2, device=dev)
    return dev, M, d, k, y


def moe_ffn_decode_workspace_size(M: int, k: int, d: int, I: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_ffn_decode_workspace_size(M, k, d, I, ctypes.byref(n)), "moe_ffn_decode_workspace_size")
    return n.value


def moe_ffn_decode(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, w13: Weights, w2: Weights,
                   out_dtype=torch.bfloat16, y=None, ws=None, dev_status=None, stream=None):
    """Output-centric decode path: y [M, d] = sum_j w_j * FFN_{e_j}(x)."""
    dev, M, d, k, y = _layer_args(x, topk_ids, topk_w, w13, w2, y, out_dtype, dev_status)
    I = w2.K
    if ws is None:
        # zeroed: the single-token path keeps its grid-barrier counters in the
        # first 256 bytes and needs them zero before the first call
        ws = torch.zeros(moe_ffn_decode_workspace_size(M, k, d, I), dtype=torch.uint8, device=dev)
    _need(ws, "ws", device=dev)
    a, b = w13.c_struct(), w2.c_struct()
    with _guard(dev):
        _check(lib().moe_ffn_decode(_ptr(x), _DT[x.dtype], M, d, _ptr(topk_ids), _ptr(topk_w), k,
                                    ctypes.byref(a), ctypes.byref(b), _ptr(y), _DT[y.dtype], _ptr(ws),
                                    _nbytes(ws), _ptr(dev_status), _stream(stream, dev)), "moe_ffn_decode")
    return y


def moe_ffn_decode_logits(logits: torch.Tensor, x: torch.Tensor, k: int, w13: Weights, w2: Weights,
                          out_dtype=torch.bfloat16, y=None, topk_ids=None, topk_w=None, ws=None, dev_status=None,
                          stream=None):
    """Routing + decode layer in one call (one kernel for a single token on the
    single-pass layout): returns (y, topk_ids, topk_w), identical to
    moe_topk_softmax followed by moe_ffn_decode."""
    _need(x, "x", tuple(_DT))
    if x.dim() != 2:
        raise ValueError(f"x must be [M, d], not {tuple(x.shape)}")
    dev = x.device
    M, d = x.shape
    _need(logits, "logits", _F32, device=dev)
    if logits.dim() != 2 or logits.shape[0] != M or logits.shape[1] != w13.E:
        raise ValueError(f"logits must be [M={M}, E={w13.E}], not {tuple(logits.shape)}")
    topk_ids = topk_ids if topk_ids is not None else torch.empty((M, k), dtype=torch.int32, device=dev)
    topk_w = topk_w if topk_w is not None else torch.empty((M, k), dtype=torch.float32, device=dev)
    _need(topk_ids, "topk_ids", _IDS, (M, k), device=dev)
    dev, M, d, k, y = _layer_args(x, topk_ids, topk_w, w13, w2, y, out_dtype, dev_status)
    I = w2.K
    if ws is None:
        ws = torch.zeros(moe_ffn_decode_workspace_size(M, k, d, I), dtype=torch.uint8, device=dev)
    _need(ws, "ws", device=dev)
    a, b = w13.c_struct(), w2.c_struct()
    with _guard(dev):
        _check(lib().moe_ffn_decode_logits(_ptr(logits), _ptr(x), _DT[x.dtype], M, d, k, ctypes.byref(a),
                                           ctypes.byref(b), _ptr(topk_ids), _ptr(topk_w), _ptr(y), _DT[y.dtype],
                                           _ptr(ws), _nbytes(ws), _ptr(dev_status), _stream(stream, dev)),
               "moe_ffn_decode_logits")
    return y, topk_ids, topk_w


def moe_ffn_decode_noalloc(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, w13: Weights,
                           w2: Weights, out_dtype=torch.bfloat16, y=None, dev_status=None, stream=None):
    """moe_ffn_decode without a workspace, for callers that cannot give the
    library device memory: the intermediate lives in a fixed 4 MiB array
    inside the library (MXFP8 two-kernel path only; first call on a device
    outside stream capture; calls must not overlap on the GPU)."""
    dev, M, d, k, y = _layer_args(x, topk_ids, topk_w, w13, w2, y, out_dtype, dev_status)
    a, b = w13.c_struct(), w2.c_struct()
    with _guard(dev):
        _check(lib().moe_ffn_decode_noalloc(_ptr(x), _DT[x.dtype], M, d, _ptr(topk_ids), _ptr(topk_w), k,
                                            ctypes.byref(a), ctypes.byref(b), _ptr(y), _DT[y.dtype],
                                            _ptr(dev_status), _stream(stream, dev)), "moe_ffn_decode_noalloc")
    return y


# ---------------------------------------------------------------- grouped path

def moe_grouped_prepare(w13: Weights, w2: Weights, stream=None):
    """Scale atoms of both projections in the tensor-core layout."""
    dev = w13.device
    w2.on("w2", dev)
    a, b = w13.c_struct(), w2.c_struct()
    n13, n2 = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_grouped_prepare_size(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n13), ctypes.byref(n2)),
           "moe_grouped_prepare_size")
    sfa13 = torch.empty(n13.value, dtype=torch.uint8, device=dev)
    sfa2 = torch.empty(n2.value, dtype=torch.uint8, device=dev)
    with _guard(dev):
        _check(lib().moe_grouped_prepare(ctypes.byref(a), ctypes.byref(b), _ptr(sfa13), _ptr(sfa2),
                                         _stream(stream, dev)), "moe_grouped_prepare")
    return sfa13, sfa2


def moe_grouped_prepare_nvfp4s(w13: Weights, w2: Weights, alpha_x: float, alpha_h: float, stream=None):
    """Prepared buffers (p13, p2) of paired 4:8 sparse NVFP4 weights for the
    W4A4 grouped path: the activations' tensor-wide scales alpha_x (block
    input) and alpha_h (SwiGLU output), the per-expert factors and the
    per-k-step side records; pass them to moe_ffn_grouped as sfa13 / sfa2."""
    dev = w13.device
    w2.on("w2", dev)
    if w13.fmt != MOE_W_NVFP4S or w2.fmt != MOE_W_NVFP4S:
        raise ValueError("moe_grouped_prepare_nvfp4s takes NVFP4S weights")
    if not (alpha_x > 0 and alpha_h > 0 and math.isfinite(alpha_x) and math.isfinite(alpha_h)):
        raise ValueError(f"alpha_x = {alpha_x}, alpha_h = {alpha_h}: both must be finite and > 0")
    a, b = w13.c_struct(), w2.c_struct()
    n13, n2 = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_grouped_prepare_size(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n13), ctypes.byref(n2)),
           "moe_grouped_prepare_size")
    p13 = torch.empty(n13.value, dtype=torch.uint8, device=dev)
    p2 = torch.empty(n2.value, dtype=torch.uint8, device=dev)
    with _guard(dev):
        _check(lib().moe_grouped_prepare_nvfp4s(ctypes.byref(a), ctypes.byref(b), float(alpha_x), float(alpha_h),
                                                _ptr(p13), _ptr(p2), _stream(stream, dev)),
               "moe_grouped_prepare_nvfp4s")
    return p13, p2


def _round256(n):
    return (n + 255) // 256 * 256


def grouped_workspace_layout(M, k, d, I, b, cap_rows):
    """Byte offsets of Xq, Xs, Hq, Hs, Yr and D inside the MXFP8 grouped
    workspace (the layout include/moe_ffn.h documents) and its total."""
    n_mma = (b + 15) // 16 * 16
    nsf = (n_mma + 127) // 128
    cap_blocks = cap_rows // b
    off, out = 0, {}
    for name, size in (("xq", cap_rows * d), ("xs", cap_blocks * (d // 128) * nsf * 512),
                       ("hq", cap_rows * I), ("hs", cap_blocks * (I // 128) * nsf * 512),
                       ("yr", M * k * d * 4), ("done", cap_blocks * 4)):
        out[name] = off
        off += _round256(size)
    out["total"] = off
    out["nsf"] = nsf
    return out


def moe_ffn_grouped_workspace_size(M, k, d, I, b, cap_rows) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_ffn_grouped_workspace_size(M, k, d, I, b, cap_rows, ctypes.byref(n)),
           "moe_ffn_grouped_workspace_size")
    return n.value


def moe_ffn_grouped(x, topk_ids, topk_w, w13: Weights, w2: Weights, sfa13, sfa2, aligned, b: int,
                    out_dtype=torch.bfloat16, y=None, ws=None, dev_status=None, stream=None):
    """Expert-centric grouped path; `aligned` = (sorted_route_ids,
    expert_ids, num_rows_post_pad) from moe_align_block_size with the same b,
    or (sorted_route_ids, expert_ids, block_rows, num_rows_post_pad) from
    moe_align_fixed_capacity (the fixed-capacity layout, MXFP8 only)."""
    dev, M, d, k, y = _layer_args(x, topk_ids, topk_w, w13, w2, y, out_dtype, dev_status)
    I = w2.K
    if b < 1:
        raise ValueError(f"block size b = {b} must be positive")
    if len(aligned) == 4:
        sorted_ids, expert_ids, block_rows, npp = aligned
    else:
        (sorted_ids, expert_ids, npp), block_rows = aligned, None
    _need(sorted_ids, "sorted_route_ids", _IDS, device=dev)
    cap_rows = sorted_ids.numel()
    _need(expert_ids, "expert_ids", _IDS, min_numel=cap_rows // b, device=dev)
    _opt(block_rows, "block_rows", dtypes=_IDS, min_numel=cap_rows // b, device=dev)
    _need(npp, "num_rows_post_pad", _IDS, min_numel=1, device=dev)
    a, bb = w13.c_struct(), w2.c_struct()
    if w13.fmt == w2.fmt and w13.fmt in (MOE_W_MXFP8, MOE_W_NVFP4S):
        # the block-scaled MMA reads the scale atoms moe_grouped_prepare wrote;
        # the NVFP4S path, what moe_grouped_prepare_nvfp4s wrote
        n13, n2 = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().moe_grouped_prepare_size(ctypes.byref(a), ctypes.byref(bb), ctypes.byref(n13),
                                              ctypes.byref(n2)), "moe_grouped_prepare_size")
        _need(sfa13, "sfa13", _U8, min_numel=n13.value, device=dev)
        _need(sfa2, "sfa2", _U8, min_numel=n2.value, device=dev)
    else:
        _opt(sfa13, "sfa13", device=dev)
        _opt(sfa2, "sfa2", device=dev)
    if ws is None:
        ws = torch.empty(moe_ffn_grouped_workspace_size(M, k, d, I, b, cap_rows), dtype=torch.uint8, device=dev)
    _need(ws, "ws", device=dev)
    with _guard(dev):
        if block_rows is None:
            _check(lib().moe_ffn_grouped(_ptr(x), _DT[x.dtype], M, d, _ptr(topk_ids), _ptr(topk_w), k,
                                         ctypes.byref(a), ctypes.byref(bb), _ptr(sfa13), _ptr(sfa2),
                                         _ptr(sorted_ids), _ptr(expert_ids), _ptr(npp), b, cap_rows,
                                         _ptr(y), _DT[y.dtype], _ptr(ws), _nbytes(ws), _ptr(dev_status),
                                         _stream(stream, dev)), "moe_ffn_grouped")
        else:
            _check(lib().moe_ffn_grouped_batched(_ptr(x), _DT[x.dtype], M, d, _ptr(topk_ids), _ptr(topk_w), k,
                                                 ctypes.byref(a), ctypes.byref(bb), _ptr(sfa13), _ptr(sfa2),
                                                 _ptr(sorted_ids), _ptr(expert_ids), _ptr(block_rows), _ptr(npp),
                                                 b, cap_rows, _ptr(y), _DT[y.dtype], _ptr(ws), _nbytes(ws),
                                                 _ptr(dev_status), _stream(stream, dev)), "moe_ffn_grouped_batched")
    return y


# ---------------------------------------------------------------- ragged grouped products

_DT16 = (torch.bfloat16, torch.float16)


def _arg(t, name: str, dtypes, dim, device=None):
    """_need plus the number of dimensions (None: any but 0), in one pass;
    returns the shape."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == dim and t.is_contiguous()
            and (device is None or t.device == device)):
        _need(t, name, dtypes, device=device)
        if t.dim() != dim and (dim is not None or t.dim() == 0):
            raise ValueError(f"{name} must have {dim or 'at least 1'} dimensions, not {tuple(t.shape)}")
    return t.shape


# The calls of a single token take about as long on the host as on the GPU, so
# the functions below check their arguments in one expression where all is in
# order, and go to the checks that name what is not only when it fails.


def _launch(gpu: int, name: str, *args) -> None:
    """The entry point `name` on the GPU of that index; raises on a refusal."""
    fn = getattr(lib(), name)
    if gpu >= 0 and gpu != _current_gpu():
        with torch.cuda.device(gpu):
            status = fn(*args)
    else:
        status = fn(*args)
    if status != MOE_OK:
        raise MoeError(status, name)


def _on(stream, gpu: int, dev):
    """The handle of the stream to launch on."""
    return _raw_stream(gpu) if stream is None and gpu >= 0 else _stream(stream, dev)


def _fit(a, b, b_dim: int, offsets) -> bool:
    """Whether a [., .] and b are 16-bit tensors of one type and offsets [.]
    int32, all contiguous and on one GPU."""
    try:
        gpu, dt = a.get_device(), a.dtype
        return (gpu >= 0 and dt in _DT16 and b.dtype is dt and offsets.dtype is torch.int32 and b.get_device() == gpu
                and offsets.get_device() == gpu and a.is_contiguous() and b.is_contiguous() and offsets.is_contiguous()
                and a.dim() == 2 and b.dim() == b_dim and offsets.dim() == 1)
    except AttributeError:
        return False


def _status(dev_status, dev):
    """Check dev_status; returns its address (None without one)."""
    if dev_status is None:
        return None
    return _need(dev_status, "dev_status", _IDS, min_numel=2, device=dev).data_ptr()


def _need_pair(a, a_name: str, b, b_name: str, b_dim: int, offsets) -> None:
    """What _fit asks, with the reason why not."""
    _arg(a, a_name, _DT16, 2)
    _arg(b, b_name, (a.dtype,), b_dim, a.device)
    _arg(offsets, "offsets", _IDS, 1, a.device)


def _experts(offsets) -> int:
    n = offsets.shape[0]
    if n < 2:
        raise ValueError(f"offsets must be [E + 1], not [{n}]")
    return n - 1


def _too_long(*sizes) -> None:
    raise ValueError(f"sizes {sizes} do not fit in 32 bits")          # the C call would get them cut


def _result(t, name: str, shape, dtype, dtypes, dev, stream):
    """The output: a new one of `dtype`, or the caller's after its check.  One
    that is first written on a given stream comes from that stream's memory,
    and is not reused before the current stream, which gets it, is past it."""
    if t is not None:
        return _need(t, name, dtypes, shape, device=dev)
    if stream is None and dtype in dtypes:
        return torch.empty(shape, dtype=dtype, device=dev)
    if dtype not in dtypes:
        raise ValueError(f"{name} cannot be {dtype}; expected {' or '.join(str(d) for d in dtypes)}")
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def moe_grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out_dtype=None, y=None, dev_status=None,
                   stream=None):
    """y [R, N]: rows offsets[e] .. offsets[e+1] - 1 of x [R, K] times w[e]^T,
    w [E, N, K] of x's type (bf16 or fp16); rows past offsets[E] give zeros.
    out_dtype: x's type (default) or float32."""
    if not _fit(x, w, 3, offsets):
        _need_pair(x, "x", w, "w", 3, offsets)
    (R, K), (e, N, k), E = x.shape, w.shape, _experts(offsets)
    if e != E or k != K:
        raise ValueError(f"w must be [E={E}, N, K={K}], not {tuple(w.shape)}")
    if (R | E | N | K) >> 31:
        _too_long(R, E, N, K)
    gpu, dev, dt = x.get_device(), x.device, x.dtype
    y = _result(y, "y", (R, N), out_dtype or dt, (dt, torch.float32), dev, stream)
    _launch(gpu, "moe_grouped_mm", x.data_ptr(), w.data_ptr(), _DT[dt], offsets.data_ptr(), R, E, N, K, y.data_ptr(),
            _DT[y.dtype], _status(dev_status, dev), _on(stream, gpu, dev))
    return y


def moe_grouped_mm_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out_dtype=None, dx=None,
                         dev_status=None, stream=None):
    """dx [R, K], the gradient of moe_grouped_mm's x: rows of dy [R, N] times
    their expert's w[e] [N, K]; rows past offsets[E] give zeros."""
    if not _fit(dy, w, 3, offsets):
        _need_pair(dy, "dy", w, "w", 3, offsets)
    (R, N), (e, n, K), E = dy.shape, w.shape, _experts(offsets)
    if e != E or n != N:
        raise ValueError(f"w must be [E={E}, N={N}, K], not {tuple(w.shape)}")
    if (R | E | N | K) >> 31:
        _too_long(R, E, N, K)
    gpu, dev, dt = dy.get_device(), dy.device, dy.dtype
    dx = _result(dx, "dx", (R, K), out_dtype or dt, (dt, torch.float32), dev, stream)
    _launch(gpu, "moe_grouped_mm_dgrad", dy.data_ptr(), w.data_ptr(), _DT[dt], offsets.data_ptr(), R, E, N, K,
            dx.data_ptr(), _DT[dx.dtype], _status(dev_status, dev), _on(stream, gpu, dev))
    return dx


def moe_grouped_mm_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out_dtype=torch.float32, dw=None,
                         accumulate: bool = False, dev_status=None, stream=None):
    """dw [E, N, K], the gradient of moe_grouped_mm's w: over each expert's
    rows the sum of dy [R, N] outer x [R, K].  accumulate adds it to the dw
    given."""
    if not _fit(dy, x, 2, offsets):
        _need_pair(dy, "dy", x, "x", 2, offsets)
    (R, N), (r, K), E = dy.shape, x.shape, _experts(offsets)
    if r != R:
        raise ValueError(f"x must be [R={R}, K], not {tuple(x.shape)}")
    if (R | E | N | K) >> 31:
        _too_long(R, E, N, K)
    gpu, dev, dt = dy.get_device(), dy.device, dy.dtype
    if accumulate and dw is None:
        raise ValueError("accumulate needs the dw to add to")
    dw = _result(dw, "dw", (E, N, K), out_dtype, (dt, torch.float32), dev, stream)
    _launch(gpu, "moe_grouped_mm_wgrad", dy.data_ptr(), x.data_ptr(), _DT[dt], offsets.data_ptr(), R, E, N, K,
            dw.data_ptr(), _DT[dw.dtype], 1 if accumulate else 0, _status(dev_status, dev), _on(stream, gpu, dev))
    return dw


def moe_grouped_mm_awq(x: torch.Tensor, w: Weights, offsets: torch.Tensor, out_dtype=None, y=None, dev_status=None,
                       stream=None):
    """y [R, N]: moe_grouped_mm with 4-bit AWQ weights, for few rows per expert:
    x [R, K] bf16 or fp16, w of E experts (offsets [0, R] with E = 1: the dense
    product).  out_dtype: x's type (default) or float32."""
    if not isinstance(w, Weights) or w.fmt != MOE_W_AWQ4:
        raise ValueError("w must be AWQ4 Weights")
    try:
        gpu, dt = x.get_device(), x.dtype
        ok = (gpu >= 0 and dt in _DT16 and x.is_contiguous() and x.dim() == 2 and offsets.dtype is torch.int32
              and offsets.get_device() == gpu and offsets.is_contiguous() and offsets.dim() == 1)
    except AttributeError:
        ok = False
    if not ok:
        _arg(x, "x", _DT16, 2)
        _arg(offsets, "offsets", _IDS, 1, x.device)
    dev, dt, c = x.device, x.dtype, w.c_struct()
    w.on("w", dev)
    (R, k), E, N = x.shape, _experts(offsets), c.N
    if c.E != E or c.K != k:
        raise ValueError(f"w is [{c.E}, {N}, {c.K}]; offsets are for {E} experts and x has K = {k}")
    if (R | E | N | k) >> 31:
        _too_long(R, E, N, k)
    y = _result(y, "y", (R, N), out_dtype or dt, (dt, torch.float32), dev, stream)
    _launch(gpu, "moe_grouped_mm_awq", x.data_ptr(), _DT[dt], c, offsets.data_ptr(), R, y.data_ptr(),
            _DT[y.dtype], _status(dev_status, dev), _on(stream, gpu, dev))
    return y


# ---------------------------------------------------------------- general routing, activation with dropout

_SCORES = (MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID)


def _route_how(k, E, score, scale) -> None:
    if score not in _SCORES:
        raise ValueError(f"unknown score {score}")
    if not 0 < k <= E:
        raise ValueError(f"k = {k} is not in 1 .. E = {E}")
    if not 0.0 < scale < math.inf:
        raise ValueError(f"scale must be finite and positive, not {scale}")


def moe_route(logits: torch.Tensor, k: int, score: int = MOE_SCORE_SOFTMAX, bias=None, groups: int = 1,
              topk_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0, topk_ids=None,
              topk_w=None, load=None, stream=None):
    """(topk_ids int32 [M, k], topk_w float32 [M, k]) of logits [M, E] (fp32, bf16
    or fp16): experts by score + bias (float32 [E]; by logit without one) from the
    topk_groups best of `groups` groups, each worth its group_top (1 or 2) best
    values; weights scale * score, over their sum with renorm.  load int32 [E] is
    increased by each expert's slots.  ragged.route has the gradient."""
    try:
        gpu, (M, E) = logits.get_device(), logits.shape
        ok = (gpu >= 0 and logits.dtype in _DT and logits.is_contiguous() and score in _SCORES and 0 < k <= E
              and 0.0 < scale < math.inf and 0 < topk_groups <= groups <= E and E % groups == 0
              and k <= topk_groups * (E // groups) and 0 < group_top < 3 and (M * k) >> 31 == 0
              and (bias is None or bias.dtype is torch.float32 and bias.get_device() == gpu and bias.is_contiguous()
                   and bias.dim() == 1 and bias.shape[0] == E)
              and (load is None or load.dtype is torch.int32 and load.get_device() == gpu and load.is_contiguous()
                   and load.dim() == 1 and load.shape[0] == E))
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        _need_route(logits, k, score, bias, groups, topk_groups, group_top, scale, load)
    dev = logits.device
    ids = _result(topk_ids, "topk_ids", (M, k), torch.int32, _IDS, dev, stream)
    w = _result(topk_w, "topk_w", (M, k), torch.float32, _F32, dev, stream)
    _launch(gpu, "moe_route", logits.data_ptr(), _DT[logits.dtype], _ptr(bias), M, E, k, score, groups, topk_groups,
            group_top, 1 if renorm else 0, scale, ids.data_ptr(), w.data_ptr(), _ptr(load), _on(stream, gpu, dev))
    return ids, w


def _need_route(logits, k, score, bias, groups, topk_groups, group_top, scale, load) -> None:
    """What moe_route asks of its arguments, with the reason why not."""
    M, E = _arg(logits, "logits", _DT, 2)
    dev = logits.device
    _route_how(k, E, score, scale)
    if not 1 <= groups <= E or E % groups or not 1 <= topk_groups <= groups or group_top not in (1, 2):
        raise ValueError(f"groups = {groups}, topk_groups = {topk_groups}, group_top = {group_top} do not fit E = {E}")
    if k > topk_groups * (E // groups):
        raise ValueError(f"k = {k} of {topk_groups} groups of {E // groups}")
    if (M * k) >> 31:
        _too_long(M, k)
    _opt(bias, "bias", dtypes=_F32, shape=(E,), device=dev)
    _opt(load, "load", dtypes=_IDS, shape=(E,), device=dev)


def moe_route_bwd(dw: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, score: int = MOE_SCORE_SOFTMAX,
                  renorm: bool = True, scale: float = 1.0, dlogits=None, stream=None):
    """dlogits [M, E], of logits' type: the gradient of moe_route's logits from
    that of its weights, dw float32 [M, k], at the ids it gave."""
    try:
        gpu, (M, E), (m, k) = logits.get_device(), logits.shape, topk_ids.shape
        ok = (gpu >= 0 and logits.dtype in _DT and logits.is_contiguous() and topk_ids.dtype is torch.int32
              and topk_ids.get_device() == gpu and topk_ids.is_contiguous() and dw.dtype is torch.float32
              and dw.get_device() == gpu and dw.is_contiguous() and dw.shape == topk_ids.shape and m == M
              and score in _SCORES and 0 < k <= E and 0.0 < scale < math.inf and (M * k) >> 31 == 0)
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:                                                        # the same, with the reason why not
        M, E = _arg(logits, "logits", _DT, 2)
        m, k = _arg(topk_ids, "topk_ids", _IDS, 2, logits.device)
        if m != M:
            raise ValueError(f"topk_ids is for {m} tokens, logits for {M}")
        _route_how(k, E, score, scale)
        if _arg(dw, "dw", _F32, 2, logits.device) != (M, k):
            raise ValueError(f"dw has shape {tuple(dw.shape)}; expected {(M, k)}")
        if (M * k) >> 31:
            _too_long(M, k)
    dev = logits.device
    dl = _result(dlogits, "dlogits", (M, E), logits.dtype, (logits.dtype,), dev, stream)
    _launch(gpu, "moe_route_bwd", dw.data_ptr(), logits.data_ptr(), _DT[logits.dtype], topk_ids.data_ptr(), M, E, k,
            score, 1 if renorm else 0, scale, dl.data_ptr(), _on(stream, gpu, dev))
    return dl


def _swiglu_args(gu, p, rng):
    """Check gu, p and rng; returns R, I and the GPU's index."""
    try:
        gpu, (R, cols) = gu.get_device(), gu.shape
        if (gpu >= 0 and gu.dtype in _DT and gu.is_contiguous() and cols > 0 and cols % 2 == 0 and (R | cols // 2) >> 31 == 0
                and 0.0 <= p < 1.0 - 2.0 ** -17
                and (p < 2.0 ** -17 if rng is None else rng.dtype is torch.int64 and rng.get_device() == gpu
                     and rng.is_contiguous() and rng.dim() == 1 and rng.shape[0] == 2)):
            return R, cols // 2, gpu
    except (AttributeError, TypeError, ValueError):
        pass
    R, cols = _arg(gu, "gu", _DT, 2)                                  # the same, with the reason why not
    if cols < 2 or cols % 2:
        raise ValueError(f"gu must be [R, 2 I], not {tuple(gu.shape)}")
    if (R | cols // 2) >> 31:
        _too_long(R, cols // 2)
    if not 0.0 <= p < 1.0 - 2.0 ** -17:
        raise ValueError(f"p = {p} is not in [0, 1 - 2^-17)")
    if rng is not None:
        _need(rng, "rng", (torch.int64,), (2,), device=gu.device)
    elif p >= 2.0 ** -17:
        raise ValueError("dropout needs rng, int64 [2]: seed and offset")
    return R, cols // 2, gu.get_device()


def moe_swiglu_dropout(gu: torch.Tensor, p: float = 0.0, rng=None, h=None, stream=None):
    """h [R, I] of gu [R, 2 I] = [g | u] (fp32, bf16 or fp16): silu(g) u, dropped
    with chance p (in steps of 2^-16) and divided by what is kept of 1.  rng int64
    [2] on the GPU: {seed, offset}; each call of a step takes its own offset."""
    R, I, gpu = _swiglu_args(gu, p, rng)
    dev = gu.device
    h = _result(h, "h", (R, I), gu.dtype, (gu.dtype,), dev, stream)
    _launch(gpu, "moe_swiglu_dropout", gu.data_ptr(), _DT[gu.dtype], R, I, p, _ptr(rng), h.data_ptr(),
            _on(stream, gpu, dev))
    return h


def moe_swiglu_dropout_bwd(dh: torch.Tensor, gu: torch.Tensor, p: float = 0.0, rng=None, dgu=None, stream=None):
    """dgu [R, 2 I], the gradient of moe_swiglu_dropout's gu from dh [R, I], with
    the p and rng of that call.  dgu may be gu."""
    R, I, gpu = _swiglu_args(gu, p, rng)
    dev = gu.device
    if _arg(dh, "dh", (gu.dtype,), 2, dev) != (R, I):
        raise ValueError(f"dh has shape {tuple(dh.shape)}; expected {(R, I)}")
    dgu = _result(dgu, "dgu", (R, 2 * I), gu.dtype, (gu.dtype,), dev, stream)
    _launch(gpu, "moe_swiglu_dropout_bwd", dh.data_ptr(), gu.data_ptr(), _DT[gu.dtype], R, I, p, _ptr(rng),
            dgu.data_ptr(), _on(stream, gpu, dev))
    return dgu


# ---------------------------------------------------------------- microscaled 4-bit floats

_FP4_BLOCK = {MOE_FP4_NVFP4: 16, MOE_FP4_MXFP4: 32}


def moe_fp4_scale_cols(K: int, fmt: int) -> int:
    """Scale bytes of a row of K elements (K / block rounded up to 16)."""
    n = ctypes.c_int32()
    _check(lib().moe_fp4_scale_cols(K, fmt, ctypes.byref(n)), "moe_fp4_scale_cols")
    return n.value


def _fp4_shape(K: int, fmt: int, what: str) -> int:
    b = _FP4_BLOCK.get(fmt)
    if b is None:
        raise ValueError(f"{what}: unknown format {fmt}")
    if K < 1 or K % 32:
        raise ValueError(f"{what}: K = {K} is not a positive multiple of 32")
    if K >> 31:
        _too_long(K)
    return (K // b + 15) // 16 * 16


def _fp4_alpha(alpha, fmt, rows, dev):
    """Check alpha ([groups] for NVFP4, None for MXFP4); returns groups."""
    if fmt != MOE_FP4_NVFP4:
        if alpha is not None:
            raise ValueError("alpha is only for NVFP4")
        return 1
    n, = _arg(alpha, "alpha", _F32, 1, dev)
    if n < 1 or rows % n:
        raise ValueError(f"alpha holds {n} entries, which do not divide the {rows} rows")
    return n


class Fp4:
    """Rows in NVFP4 or MXFP4: q uint8 [..., K/2], s uint8 [..., Ks] and, for
    NVFP4, alpha float32 (one for activations [R, .], one per expert for
    weights [E, N, .]), as moe_fp4_quantize returns them.  Checked when the
    object is made, for every launch that takes it: its fields are fixed."""
    __slots__ = ("fmt", "q", "s", "alpha")

    def __init__(self, fmt: int, q: torch.Tensor, s: torch.Tensor, alpha: torch.Tensor | None = None):
        put = object.__setattr__
        put(self, "fmt", fmt)
        put(self, "q", q)
        put(self, "s", s)
        put(self, "alpha", alpha)
        try:
            gpu, qs, ss, block, n = q.get_device(), q.shape, s.shape, _FP4_BLOCK[fmt], q.dim()
            half, rows = qs[-1], qs[0]
            ok = (gpu >= 0 and q.dtype is torch.uint8 and s.dtype is torch.uint8 and s.get_device() == gpu
                  and q.is_contiguous() and s.is_contiguous() and (n == 2 or n == 3) and s.dim() == n and half > 0
                  and half % 16 == 0 and ss[0] == rows and ss[-2] == qs[-2] and ss[-1] == (2 * half // block + 15) // 16 * 16)
            if ok and alpha is not None:
                ok = (block == 16 and alpha.dtype is torch.float32 and alpha.get_device() == gpu and alpha.is_contiguous()
                      and alpha.dim() == 1 and alpha.shape[0] == (rows if n == 3 else 1))
            elif ok:
                ok = block == 32
        except (AttributeError, IndexError, KeyError, TypeError):
            ok = False
        if not ok:
            self._need()

    def __setattr__(self, name, value):
        raise AttributeError("an Fp4's fields are fixed; make a new one")

    def __delattr__(self, name):
        raise AttributeError("an Fp4's fields are fixed; make a new one")

    def __reduce__(self):                                             # copies are made, and checked, anew
        return Fp4, (self.fmt, self.q, self.s, self.alpha)

    def _need(self):
        """What the constructor asks, with the reason why not."""
        dim = 3 if isinstance(self.q, torch.Tensor) and self.q.dim() == 3 else 2
        *lead, half = _arg(self.q, "fp4.q", _U8, dim)
        dev = self.q.device
        Ks = _fp4_shape(half * 2, self.fmt, "fp4")
        *slead, cols = _arg(self.s, "fp4.s", _U8, dim, dev)
        if slead != lead or cols != Ks:
            raise ValueError(f"fp4.s has shape {tuple(self.s.shape)}; expected {(*lead, Ks)}")
        if self.fmt == MOE_FP4_NVFP4:
            n, = _arg(self.alpha, "fp4.alpha", _F32, 1, dev)
            if n != (lead[0] if dim == 3 else 1):
                raise ValueError(f"fp4.alpha holds {n} entries; expected {lead[0] if dim == 3 else 1}")
        elif self.alpha is not None:
            raise ValueError("fp4.alpha is only for NVFP4")


def _fp4_rows(t, name: str, dtypes, per: int, fmt: int, alpha):
    """Check the tensor of values (per = 1) or codes (per = 2 elements a
    byte) and alpha; returns the leading shape, K, Ks, rows and groups."""
    try:
        gpu, shape, block = t.get_device(), t.shape, _FP4_BLOCK[fmt]
        K = shape[-1] * per
        if (gpu >= 0 and t.dtype in dtypes and t.is_contiguous() and 0 < K < 1 << 31 and K % 32 == 0
                and (block == 32 if alpha is None else
                     block == 16 and alpha.dtype is torch.float32 and alpha.get_device() == gpu and alpha.is_contiguous()
                     and alpha.dim() == 1)):
            rows, groups = t.numel() * per // K, 1 if alpha is None else alpha.shape[0]
            if groups and rows % groups == 0:
                return shape[:-1], K, (K // block + 15) // 16 * 16, rows, groups
    except (AttributeError, IndexError, KeyError):
        pass
    *lead, last = _arg(t, name, dtypes, None)                         # the same, with the reason why not
    K = last * per
    Ks = _fp4_shape(K, fmt, name)
    rows = t.numel() * per // K
    return tuple(lead), K, Ks, rows, _fp4_alpha(alpha, fmt, rows, t.device)


def moe_fp4_quantize(v: torch.Tensor, fmt: int, alpha=None, q=None, s=None, stream=None):
    """NVFP4 or MXFP4 codes and scales of v [..., K] (fp32, bf16 or fp16):
    (q uint8 [..., K/2], s uint8 [..., Ks]).  alpha (NVFP4): float32 [groups],
    each for an equal run of rows."""
    lead, K, Ks, rows, groups = _fp4_rows(v, "v", _DT, 1, fmt, alpha)
    gpu, dev = v.get_device(), v.device
    q = _result(q, "q", (*lead, K // 2), torch.uint8, _U8, dev, stream)
    s = _result(s, "s", (*lead, Ks), torch.uint8, _U8, dev, stream)
    _launch(gpu, "moe_fp4_quantize", v.data_ptr(), _DT[v.dtype], rows, K, fmt, _ptr(alpha), groups, q.data_ptr(),
            s.data_ptr(), _on(stream, gpu, dev))
    return q, s


def moe_fp4_dequantize(q: torch.Tensor, s: torch.Tensor, fmt: int, alpha=None, out_dtype=torch.float32, v=None,
                       stream=None):
    """The values v [..., K] that codes and scales stand for."""
    lead, K, Ks, rows, groups = _fp4_rows(q, "q", _U8, 2, fmt, alpha)
    gpu, dev = q.get_device(), q.device
    if _arg(s, "s", _U8, None, dev) != (*lead, Ks):
        raise ValueError(f"s has shape {tuple(s.shape)}; expected {(*lead, Ks)}")
    v = _result(v, "v", (*lead, K), out_dtype, _DT, dev, stream)
    _launch(gpu, "moe_fp4_dequantize", q.data_ptr(), s.data_ptr(), rows, K, fmt, _ptr(alpha), groups, v.data_ptr(),
            _DT[v.dtype], _on(stream, gpu, dev))
    return v


def moe_grouped_mm_fp4(x: Fp4, w: Fp4, offsets: torch.Tensor, out_dtype=torch.bfloat16, y=None, dev_status=None,
                       stream=None):
    """y [R, N]: moe_grouped_mm on 4-bit operands, x [R, K] and w [E, N, K] of
    the same format (offsets [0, R] with E = 1: the dense product)."""
    if not (isinstance(x, Fp4) and isinstance(w, Fp4)):
        raise ValueError("x and w must be Fp4")
    gpu, dev = x.q.get_device(), x.q.device
    if not (isinstance(offsets, torch.Tensor) and offsets.dtype is torch.int32 and offsets.get_device() == gpu >= 0 and offsets.dim() == 1
            and offsets.is_contiguous()):
        _arg(offsets, "offsets", _IDS, 1, dev)
    E = _experts(offsets)
    if x.q.dim() != 2 or w.q.dim() != 3 or x.fmt != w.fmt:
        raise ValueError("x must be [R, K] and w [E, N, K] of one format")
    if w.q.get_device() != gpu:
        raise ValueError(f"w is on {w.q.device}; the call's tensors are on {dev}")
    (R, xh), (e, N, half) = x.q.shape, w.q.shape
    K = half * 2
    if e != E or xh != half:
        raise ValueError(f"w is [{e}, {N}, {K}]; offsets are for {E} experts and x has K = {xh * 2}")
    if (R | E | N | K) >> 31:
        _too_long(R, E, N, K)
    y = _result(y, "y", (R, N), out_dtype, _DT, dev, stream)
    _launch(gpu, "moe_grouped_mm_fp4", x.q.data_ptr(), x.s.data_ptr(), _ptr(x.alpha), w.q.data_ptr(), w.s.data_ptr(),
            _ptr(w.alpha), x.fmt, offsets.data_ptr(), R, E, N, K, y.data_ptr(), _DT[y.dtype], _status(dev_status, dev),
            _on(stream, gpu, dev))
    return y

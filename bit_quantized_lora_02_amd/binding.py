"""Thin ctypes binding over ``libqlora.so`` (the C ABI of ``include/qlora.h``).

This module only marshals arguments: torch tensors supply device memory
(``data_ptr()``) and the current HIP stream; every step of the computation runs
in the library's gfx950 kernels.  There is no CPU or PyTorch fallback: if the
library is missing or the device is not gfx950, calls raise.

Names follow the C ABI: ``quantize_nf4``, ``dequant``, ``linear_fwd``,
``linear_bwd``, ``linear_fwd_dropout``, ``linear_bwd_dropout``, ``linear_fwd_multi``, ``adamw_step``,
``adamw8_step``, ``merge``, ``head_ce``, ``head_distill``, plus ``QLoRALinearFn`` (a torch.autograd.Function whose backward
returns gradients for X, A and B and none for the frozen NF4 weight), ``HeadCEFn`` and ``HeadDistillFn``
(the output layer's losses with their gradients).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlora.so")

QLORA_OK = 0
QLORA_EINVAL = -1
QLORA_EWORKSPACE = -2
QLORA_ENODEV = -3
QLORA_EHIP = -4
OP_FWD = 0
OP_BWD = 1
OP_FWD_DROPOUT = 2
OP_FWD_MULTI = 3
MAX_RANK = 128
MAX_TARGETS = 256

EXPORTED = (
    "qlora_nf4_storage",
    "qlora_nf4_codebook",
    "qlora_workspace_bytes",
    "qlora_quantize_nf4",
    "qlora_dequant",
    "qlora_linear_fwd",
    "qlora_linear_fwd_noalloc",
    "qlora_linear_bwd",
    "qlora_linear_fwd_dropout",
    "qlora_linear_bwd_dropout",
    "qlora_linear_fwd_multi",
    "qlora_adamw_step",
    "qlora_adamw8_step",
    "qlora_merge",
    "qlora_head_ce",
    "qlora_head_distill",
    "qlora_head_workspace_bytes",
    "qlora_strerror",
    "qlora_last_error",
    "qlora_timing_enable",
    "qlora_timing_read",
    "qlora_timing_read_each",
)


class QLoRAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{msg} (code {code})")
        self.code = code


class _NF4(ctypes.Structure):
    _fields_ = [
        ("n_out", ctypes.c_int64),
        ("n_in", ctypes.c_int64),
        ("codes", ctypes.c_void_p),
        ("absmax_q", ctypes.c_void_p),
        ("absmax_step", ctypes.c_void_p),
    ]


class _AdamTensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("master", ctypes.c_void_p),
        ("n", ctypes.c_int64),
    ]


class _Adam8Tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg_code", ctypes.c_void_p),
        ("exp_avg_absmax", ctypes.c_void_p),
        ("exp_avg_sq_code", ctypes.c_void_p),
        ("exp_avg_sq_absmax", ctypes.c_void_p),
        ("master", ctypes.c_void_p),
        ("n", ctypes.c_int64),
    ]


_lib = None


def load_library() -> ctypes.CDLL:
    """Load libqlora.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -m bit_quantized_lora_02_amd.build)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pnf4 = ctypes.POINTER(_NF4)
    sig = {
        "qlora_nf4_storage": ([i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)], ctypes.c_int),
        "qlora_nf4_codebook": ([P], ctypes.c_int),
        "qlora_workspace_bytes": ([ctypes.c_int, i64, i64, i64, i32, ctypes.POINTER(sz)], ctypes.c_int),
        "qlora_quantize_nf4": ([P, pnf4, P], ctypes.c_int),
        "qlora_dequant": ([pnf4, P, P], ctypes.c_int),
        "qlora_linear_fwd": ([P, i64, pnf4, P, P, i32, ctypes.c_float, P, P, P, sz, P], ctypes.c_int),
        "qlora_linear_fwd_noalloc": ([P, i64, pnf4, P, P, i32, ctypes.c_float, P, P, P], ctypes.c_int),
        "qlora_linear_bwd": ([P, P, i64, pnf4, P, P, i32, ctypes.c_float, P, P, P, P, P, sz, P], ctypes.c_int),
        "qlora_linear_fwd_dropout": ([P, i64, pnf4, P, P, i32, ctypes.c_float, ctypes.c_float, ctypes.c_uint64,
                                      ctypes.c_uint64, P, P, P, P, sz, P], ctypes.c_int),
        "qlora_linear_bwd_dropout": ([P, P, i64, pnf4, P, P, i32, ctypes.c_float, ctypes.c_float, P, P, P, P, P, P,
                                      sz, P], ctypes.c_int),
        "qlora_adamw_step": ([ctypes.POINTER(_AdamTensor), i32, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                              ctypes.c_double, ctypes.c_double, i64, P], ctypes.c_int),
        "qlora_merge": ([pnf4, P, i64, i64, P, P, i32, ctypes.c_float, P, P, P], ctypes.c_int),
        "qlora_linear_fwd_multi": ([P, i64, pnf4, P, P, i32, i32, ctypes.c_float, P, P, i32, P, P, sz, P],
                                   ctypes.c_int),
        "qlora_adamw8_step": ([ctypes.POINTER(_Adam8Tensor), i32, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                               ctypes.c_double, ctypes.c_double, i64, P], ctypes.c_int),
        "qlora_head_ce": ([P, i64, P, i64, i64, P, P, P, P, P, P, sz, P], ctypes.c_int),
        "qlora_head_distill": ([P, i64, P, i64, i64, P, P, i32, ctypes.c_float, P, P, P, P, P, sz, P], ctypes.c_int),
        "qlora_head_workspace_bytes": ([i64, i64, i64, i32, ctypes.c_int, ctypes.c_int, ctypes.POINTER(sz)],
                                       ctypes.c_int),
        "qlora_strerror": ([ctypes.c_int], ctypes.c_char_p),
        "qlora_last_error": ([], ctypes.c_char_p),
        "qlora_timing_enable": ([ctypes.c_char_p, ctypes.c_int], ctypes.c_int),
        "qlora_timing_read": ([ctypes.c_char_p, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)], ctypes.c_int),
        "qlora_timing_read_each": ([ctypes.c_char_p, ctypes.POINTER(ctypes.c_double), i64, ctypes.POINTER(i64)],
                                   ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != QLORA_OK:
        lib = load_library()
        raise QLoRAError(rc, f"{what}: {lib.qlora_strerror(rc).decode()}: {lib.qlora_last_error().decode()}")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device):
    """The current HIP stream of `device` (the raw handle; building a torch Stream object costs ~2 us)."""
    if _raw_stream is not None and device.index is not None:
        return ctypes.c_void_p(_raw_stream(device.index))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _bits(t: torch.Tensor) -> torch.Tensor:
    """bf16 tensor -> contiguous view used for the uint16 ABI arguments."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"expected a bfloat16 tensor, got {t.dtype}")
    return t.contiguous()


def _on_gpu(t: torch.Tensor) -> None:
    """Operands live on a GPU (checked after their shapes, so shape errors name themselves first)."""
    if not t.is_cuda:
        raise TypeError("expected GPU tensors")


def _want(t: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device, name: str) -> torch.Tensor:
    """A caller-supplied buffer the library writes (or reads) by address: it must have exactly this shape
    and dtype, be contiguous and sit on `device` (the C ABI sees only the pointer)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _inputs(X: torch.Tensor, *others: torch.Tensor) -> None:
    """X is a 2-D bf16 GPU tensor and every other operand sits on its device."""
    if X.dim() != 2:
        raise ValueError(f"X must be 2-D [T, n_in], got {tuple(X.shape)}")
    for t in others:
        if t is not None and t.device != X.device:
            raise ValueError(f"operands on different devices: {t.device} and {X.device}")


def _ws_bytes(ws: torch.Tensor, device: torch.device) -> int:
    """Size in bytes of a caller-supplied workspace (a contiguous GPU tensor on `device`)."""
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous() or ws.device != device:
        raise ValueError("the workspace must be a contiguous tensor on the operands' device")
    return ws.numel() * ws.element_size()


def _check_weight(w: "NF4Weight", device: torch.device) -> None:
    cb, qb, sb = storage_bytes(w.n_out, w.n_in)
    for t, n, dt, name in ((w.codes, cb, torch.uint8, "codes"), (w.absmax_q, qb, torch.uint8, "absmax_q"),
                           (w.absmax_step, sb // 4, torch.float32, "absmax_step")):
        _want(t, (n,), dt, device, f"NF4 weight {name}")


@functools.lru_cache(maxsize=256)
def storage_bytes(n_out: int, n_in: int) -> tuple[int, int, int]:
    c, q, s = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().qlora_nf4_storage(n_out, n_in, ctypes.byref(c), ctypes.byref(q), ctypes.byref(s)),
           "qlora_nf4_storage")
    return c.value, q.value, s.value


def codebook() -> list[float]:
    arr = (ctypes.c_float * 16)()
    _check(load_library().qlora_nf4_codebook(arr), "qlora_nf4_codebook")
    return list(arr)


def workspace_bytes(op: int, T: int, n_out: int, n_in: int, r: int) -> int:
    b = ctypes.c_size_t()
    _check(load_library().qlora_workspace_bytes(op, T, n_out, n_in, r, ctypes.byref(b)), "qlora_workspace_bytes")
    return b.value


@dataclass
class NF4Weight:
    """A frozen NF4 weight: the three device arrays of the layout plus its shape."""
    n_out: int
    n_in: int
    codes: torch.Tensor  # uint8 [n_out*n_in/2]
    absmax_q: torch.Tensor  # uint8 [n_out*n_in/64]
    absmax_step: torch.Tensor  # float32 [ceil(n_out*n_in/16384)]

    def struct(self) -> _NF4:
        return _NF4(self.n_out, self.n_in, self.codes.data_ptr(), self.absmax_q.data_ptr(), self.absmax_step.data_ptr())

    @property
    def device(self):
        return self.codes.device

    @staticmethod
    def empty(n_out: int, n_in: int, device) -> "NF4Weight":
        cb, qb, sb = storage_bytes(n_out, n_in)
        return NF4Weight(n_out, n_in, torch.empty(cb, dtype=torch.uint8, device=device),
                         torch.empty(qb, dtype=torch.uint8, device=device),
                         torch.empty(sb // 4, dtype=torch.float32, device=device))


def quantize_nf4(W: torch.Tensor) -> NF4Weight:
    """Quantize a float32 [n_out, n_in] GPU tensor to NF4 with double-quantized constants."""
    if W.dtype != torch.float32 or not W.is_cuda or W.dim() != 2:
        raise TypeError("W must be a 2-D float32 GPU tensor")
    W = W.contiguous()
    w = NF4Weight.empty(W.shape[0], W.shape[1], W.device)
    st = w.struct()
    _check(load_library().qlora_quantize_nf4(_ptr(W), ctypes.byref(st), _stream(W.device)), "qlora_quantize_nf4")
    return w


def dequant(w: NF4Weight) -> torch.Tensor:
    """bf16 [n_out, n_in] expansion of an NF4 weight (tests and export only)."""
    _check_weight(w, w.device)
    out = torch.empty((w.n_out, w.n_in), dtype=torch.bfloat16, device=w.device)
    st = w.struct()
    _check(load_library().qlora_dequant(ctypes.byref(st), _ptr(out), _stream(w.device)), "qlora_dequant")
    return out


def _workspace(op, T, w: NF4Weight, r) -> tuple[torch.Tensor | None, int]:
    nb = workspace_bytes(op, T, w.n_out, w.n_in, r)
    if nb == 0:
        return None, 0
    return torch.empty(nb, dtype=torch.uint8, device=w.device), nb


def linear_fwd(X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
               save_u: bool = True, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
               u_out: torch.Tensor | None = None):
    """Y = X . deq(W)^T + (alpha/r) (X A^T) B^T; returns (Y, U or None).

    ``out``/``u_out`` are optional preallocated [T, n_out] / [T, r] bf16 buffers."""
    X, A, B = _bits(X), _bits(A), _bits(B)
    _inputs(X, A, B)
    _check_weight(w, X.device)
    T, r = X.shape[0], A.shape[0]
    if X.shape[1] != w.n_in or A.shape != (r, w.n_in) or B.shape != (w.n_out, r):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, A {tuple(A.shape)}, B {tuple(B.shape)}, "
                         f"W [{w.n_out}, {w.n_in}]")
    bf = torch.bfloat16
    Y = _want(out, (T, w.n_out), bf, X.device, "out") if out is not None else torch.empty((T, w.n_out), dtype=bf,
                                                                                            device=X.device)
    U = (_want(u_out, (T, r), bf, X.device, "u_out") if u_out is not None
         else (torch.empty((T, r), dtype=bf, device=X.device) if save_u else None))
    if ws is None:
        ws, nb = _workspace(OP_FWD, T, w, r)
    else:
        nb = _ws_bytes(ws, X.device)
    _on_gpu(X)
    st = w.struct()
    _check(load_library().qlora_linear_fwd(_ptr(X), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha), _ptr(Y),
                                           _ptr(U), _ptr(ws), nb, _stream(X.device)), "qlora_linear_fwd")
    return Y, U


def _grad_outs(outs, X, A, B, need_dx):
    """(dX or None, dA, dB): the caller's buffers, checked against X, A and B, or new ones."""
    if outs is None:
        return (torch.empty_like(X) if need_dx else None), torch.empty_like(A), torch.empty_like(B)
    dX, dA, dB = outs
    bf = torch.bfloat16
    if dX is not None:
        _want(dX, tuple(X.shape), bf, X.device, "dX")
    return dX, _want(dA, tuple(A.shape), bf, X.device, "dA"), _want(dB, tuple(B.shape), bf, X.device, "dB")


def linear_bwd(X: torch.Tensor, dY: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
               U: torch.Tensor | None = None, need_dx: bool = True, ws: torch.Tensor | None = None,
               outs: tuple | None = None):
    """Gradients (dX or None, dA, dB) of the forward above; W gets none."""
    X, dY, A, B = _bits(X), _bits(dY), _bits(A), _bits(B)
    if U is not None:
        U = _bits(U)
    _inputs(X, dY, A, B, U)
    _check_weight(w, X.device)
    T, r = X.shape[0], A.shape[0]
    if (X.shape[1] != w.n_in or dY.shape != (T, w.n_out) or A.shape != (r, w.n_in) or B.shape != (w.n_out, r)
            or (U is not None and U.shape != (T, r))):
        raise ValueError(f"shape mismatch in linear_bwd: X {tuple(X.shape)}, dY {tuple(dY.shape)}, "
                         f"A {tuple(A.shape)}, B {tuple(B.shape)}, U {None if U is None else tuple(U.shape)}, "
                         f"W [{w.n_out}, {w.n_in}]")
    dX, dA, dB = _grad_outs(outs, X, A, B, need_dx)
    if ws is None:
        ws, nb = _workspace(OP_BWD, T, w, r)
    else:
        nb = _ws_bytes(ws, X.device)
    _on_gpu(X)
    st = w.struct()
    _check(load_library().qlora_linear_bwd(_ptr(X), _ptr(dY), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha),
                                           _ptr(U), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), nb, _stream(X.device)),
           "qlora_linear_bwd")
    return dX, dA, dB


def linear_fwd_dropout(X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float, p: float,
                       seed: int, offset: int = 0, save_u: bool = True, ws: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, u_out: torch.Tensor | None = None,
                       mask_out: torch.Tensor | None = None):
    """Forward with LoRA dropout on the adapter input; returns (Y, U or None, keep-bit mask uint8 [T, n_in/8])."""
    X, A, B = _bits(X), _bits(A), _bits(B)
    _inputs(X, A, B)
    _check_weight(w, X.device)
    T, r = X.shape[0], A.shape[0]
    if X.shape[1] != w.n_in or A.shape != (r, w.n_in) or B.shape != (w.n_out, r):
        raise ValueError("shape mismatch in linear_fwd_dropout")
    bf, dev = torch.bfloat16, X.device
    Y = _want(out, (T, w.n_out), bf, dev, "out") if out is not None else torch.empty((T, w.n_out), dtype=bf,
                                                                                       device=dev)
    U = (_want(u_out, (T, r), bf, dev, "u_out") if u_out is not None
         else (torch.empty((T, r), dtype=bf, device=dev) if save_u else None))
    mask = (_want(mask_out, (T, w.n_in // 8), torch.uint8, dev, "mask_out") if mask_out is not None
            else torch.empty((T, w.n_in // 8), dtype=torch.uint8, device=dev))
    if ws is None:
        ws, nb = _workspace(OP_FWD_DROPOUT, T, w, r)
    else:
        nb = _ws_bytes(ws, dev)
    _on_gpu(X)
    st = w.struct()
    _check(load_library().qlora_linear_fwd_dropout(_ptr(X), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha),
                                                   float(p), int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                                                   _ptr(mask), _ptr(Y), _ptr(U), _ptr(ws), nb, _stream(X.device)),
           "qlora_linear_fwd_dropout")
    return Y, U, mask


def linear_bwd_dropout(X: torch.Tensor, dY: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor,
                       alpha: float, p: float, mask: torch.Tensor, U: torch.Tensor | None = None,
                       need_dx: bool = True, ws: torch.Tensor | None = None, outs: tuple | None = None):
    """Gradients (dX or None, dA, dB) of ``linear_fwd_dropout`` given its keep-bit mask."""
    X, dY, A, B = _bits(X), _bits(dY), _bits(A), _bits(B)
    if U is not None:
        U = _bits(U)
    _inputs(X, dY, A, B, U, mask)
    _check_weight(w, X.device)
    T, r = X.shape[0], A.shape[0]
    if (X.shape[1] != w.n_in or dY.shape != (T, w.n_out) or A.shape != (r, w.n_in) or B.shape != (w.n_out, r)
            or (U is not None and U.shape != (T, r))):
        raise ValueError("shape mismatch in linear_bwd_dropout")
    if mask.dtype != torch.uint8 or not mask.is_cuda or mask.numel() != T * w.n_in // 8:
        raise ValueError("mask must be a uint8 GPU tensor of T * n_in / 8 bytes")
    mask = mask.contiguous()
    dX, dA, dB = _grad_outs(outs, X, A, B, need_dx)
    if ws is None:
        ws, nb = _workspace(OP_BWD, T, w, r)
    else:
        nb = _ws_bytes(ws, X.device)
    _on_gpu(X)
    st = w.struct()
    _check(load_library().qlora_linear_bwd_dropout(_ptr(X), _ptr(dY), T, ctypes.byref(st), _ptr(A), _ptr(B), r,
                                                   float(alpha), float(p), _ptr(mask), _ptr(U), _ptr(dX), _ptr(dA),
                                                   _ptr(dB), _ptr(ws), nb, _stream(X.device)),
           "qlora_linear_bwd_dropout")
    return dX, dA, dB


def linear_fwd_multi(X: torch.Tensor, w: NF4Weight, A_pool: torch.Tensor, B_pool: torch.Tensor, alpha: float,
                     seg_offsets: torch.Tensor, seg_adapter: torch.Tensor, ws: torch.Tensor | None = None,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Y for a batch whose token segments use different adapters of a pool (A_pool [n, r, n_in],
    B_pool [n, n_out, r]); seg_offsets int32 [n_seg + 1], seg_adapter int32 [n_seg] on the GPU."""
    X, A_pool, B_pool = _bits(X), _bits(A_pool), _bits(B_pool)
    _inputs(X, A_pool, B_pool, seg_offsets, seg_adapter)
    _check_weight(w, X.device)
    T = X.shape[0]
    n_pool, r = A_pool.shape[0], A_pool.shape[1]
    if A_pool.shape != (n_pool, r, w.n_in) or B_pool.shape != (n_pool, w.n_out, r) or X.shape[1] != w.n_in:
        raise ValueError("shape mismatch in linear_fwd_multi")
    for t in (seg_offsets, seg_adapter):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise TypeError("segment tables must be contiguous int32 GPU tensors")
    n_seg = seg_adapter.numel()
    if seg_offsets.numel() != n_seg + 1:
        raise ValueError("seg_offsets needs n_seg + 1 entries")
    Y = (_want(out, (T, w.n_out), torch.bfloat16, X.device, "out") if out is not None
         else torch.empty((T, w.n_out), dtype=torch.bfloat16, device=X.device))
    if ws is None:
        ws, nb = _workspace(OP_FWD_MULTI, T, w, r)
    else:
        nb = _ws_bytes(ws, X.device)
    _on_gpu(X)
    st = w.struct()
    _check(load_library().qlora_linear_fwd_multi(_ptr(X), T, ctypes.byref(st), _ptr(A_pool), _ptr(B_pool), n_pool, r,
                                                 float(alpha), _ptr(seg_offsets), _ptr(seg_adapter), n_seg, _ptr(Y),
                                                 _ptr(ws), nb, _stream(X.device)), "qlora_linear_fwd_multi")
    return Y


def merge(A: torch.Tensor, B: torch.Tensor, alpha: float, w: NF4Weight | None = None,
          W_base: torch.Tensor | None = None, bf16_out: bool = True, f32_out: bool = False):
    """Merged weight W + (alpha/r) B A for export, W = deq(w) or the bf16 base W_base (exactly one).

    Returns (bf16 [n_out, n_in] or None, float32 [n_out, n_in] or None); the float32 output is what
    ``quantize_nf4`` takes to quantize the merged weight again."""
    if (w is None) == (W_base is None):
        raise ValueError("give exactly one of w and W_base")
    A, B = _bits(A), _bits(B)
    r = A.shape[0]
    if w is not None:
        _check_weight(w, A.device)
    elif W_base.dim() != 2 or W_base.device != A.device:
        raise ValueError("W_base must be a 2-D tensor on the adapters' device")
    if B.device != A.device:
        raise ValueError("A and B on different devices")
    n_out, n_in = (w.n_out, w.n_in) if w is not None else tuple(W_base.shape)
    if A.shape != (r, n_in) or B.shape != (n_out, r):
        raise ValueError("shape mismatch in merge")
    dev = A.device
    out = torch.empty((n_out, n_in), dtype=torch.bfloat16, device=dev) if bf16_out else None
    out32 = torch.empty((n_out, n_in), dtype=torch.float32, device=dev) if f32_out else None
    _on_gpu(A)
    Wb = _bits(W_base) if W_base is not None else None
    st = w.struct() if w is not None else None
    _check(load_library().qlora_merge(ctypes.byref(st) if st is not None else None, _ptr(Wb), n_out, n_in, _ptr(A),
                                      _ptr(B), r, float(alpha), _ptr(out), _ptr(out32), _stream(dev)), "qlora_merge")
    return out, out32


@dataclass
class AdamState:
    """AdamW state of one bf16 parameter: binary32 moments and an optional binary32 master copy."""
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    master: torch.Tensor | None = None

    @staticmethod
    def zeros_like(param: torch.Tensor, master: bool = False) -> "AdamState":
        z = lambda: torch.zeros(param.shape, dtype=torch.float32, device=param.device)
        return AdamState(z(), z(), param.float().clone() if master else None)


def adamw_step(params, grads, states, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
               eps: float = 1e-8, weight_decay: float = 0.0):
    """One fused AdamW step, in place, over lists of bf16 params, bf16 grads and AdamState."""
    descs = []
    keep = []
    for p, g, st in zip(params, grads, states, strict=True):
        if p.dtype != torch.bfloat16 or g.dtype != torch.bfloat16 or not p.is_contiguous() or not p.is_cuda:
            raise TypeError("params and grads must be contiguous bf16 GPU tensors")
        g = g.contiguous()
        keep.append(g)
        if g.shape != p.shape or st.exp_avg.shape != p.shape or st.exp_avg_sq.shape != p.shape:
            raise ValueError("shape mismatch in adamw_step")
        for t in (st.exp_avg, st.exp_avg_sq) + ((st.master,) if st.master is not None else ()):
            if t.dtype != torch.float32 or not t.is_contiguous():
                raise TypeError("AdamW state must be contiguous float32")
        descs.append(_AdamTensor(p.data_ptr(), g.data_ptr(), st.exp_avg.data_ptr(), st.exp_avg_sq.data_ptr(),
                                 st.master.data_ptr() if st.master is not None else None, p.numel()))
    if not descs:
        return
    arr = (_AdamTensor * len(descs))(*descs)
    _check(load_library().qlora_adamw_step(arr, len(descs), float(lr), float(beta1), float(beta2), float(eps),
                                           float(weight_decay), int(step), _stream(params[0].device)),
           "qlora_adamw_step")


@dataclass
class Adam8State:
    """8-bit AdamW state of one bf16 parameter: codes and per-2048-block absmax of each moment."""
    exp_avg_code: torch.Tensor
    exp_avg_absmax: torch.Tensor
    exp_avg_sq_code: torch.Tensor
    exp_avg_sq_absmax: torch.Tensor
    master: torch.Tensor | None = None

    @staticmethod
    def zeros_like(param: torch.Tensor, master: bool = False) -> "Adam8State":
        n = param.numel()
        nb = (n + 2047) // 2048
        dev = param.device
        return Adam8State(torch.zeros(n, dtype=torch.uint8, device=dev), torch.zeros(nb, dtype=torch.float32, device=dev),
                          torch.zeros(n, dtype=torch.uint8, device=dev), torch.zeros(nb, dtype=torch.float32, device=dev),
                          param.float().clone() if master else None)


def adamw8_step(params, grads, states, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
                eps: float = 1e-8, weight_decay: float = 0.0):
    """One fused AdamW step with block-wise 8-bit moments, in place, over lists of params, grads and Adam8State."""
    descs, keep = [], []
    for p, g, st in zip(params, grads, states, strict=True):
        if p.dtype != torch.bfloat16 or g.dtype != torch.bfloat16 or not p.is_contiguous() or not p.is_cuda:
            raise TypeError("params and grads must be contiguous bf16 GPU tensors")
        g = g.contiguous()
        keep.append(g)
        n, nb = p.numel(), (p.numel() + 2047) // 2048
        if g.numel() != n or st.exp_avg_code.numel() != n or st.exp_avg_sq_code.numel() != n or \
                st.exp_avg_absmax.numel() != nb or st.exp_avg_sq_absmax.numel() != nb:
            raise ValueError("shape mismatch in adamw8_step")
        descs.append(_Adam8Tensor(p.data_ptr(), g.data_ptr(), st.exp_avg_code.data_ptr(), st.exp_avg_absmax.data_ptr(),
                                  st.exp_avg_sq_code.data_ptr(), st.exp_avg_sq_absmax.data_ptr(),
                                  st.master.data_ptr() if st.master is not None else None, n))
    if not descs:
        return
    arr = (_Adam8Tensor * len(descs))(*descs)
    _check(load_library().qlora_adamw8_step(arr, len(descs), float(lr), float(beta1), float(beta2), float(eps),
                                            float(weight_decay), int(step), _stream(params[0].device)),
           "qlora_adamw8_step")


@functools.lru_cache(maxsize=256)
def head_workspace_bytes(T: int, n_vocab: int, n_in: int, k: int = 0, need_dx: bool = True,
                         need_dw: bool = False) -> int:
    """Workspace bytes of ``head_ce`` (k = 0) and ``head_distill`` (k teacher logits per row)."""
    b = ctypes.c_size_t()
    _check(load_library().qlora_head_workspace_bytes(T, n_vocab, n_in, k, int(need_dx), int(need_dw), ctypes.byref(b)),
           "qlora_head_workspace_bytes")
    return b.value


def _head_args(X, W, weight, k, need_dx, need_dw, ws, outs):
    """Checked operands and outputs of the two losses: (X, W, loss, dX or None, dW or None, ws, ws bytes)."""
    X, W = _bits(X), _bits(W)
    _inputs(X, W, weight)
    if W.dim() != 2 or W.shape[1] != X.shape[1]:
        raise ValueError(f"W must be [n_vocab, {X.shape[1]}], got {tuple(W.shape)}")
    T, dev, bf = X.shape[0], X.device, torch.bfloat16
    if weight is not None:
        _want(weight, (T,), torch.float32, dev, "weight")
    if outs is None:
        loss = torch.empty((T,), dtype=torch.float32, device=dev)
        dX = torch.empty_like(X) if need_dx else None
        dW = torch.empty_like(W) if need_dw else None
    else:
        loss, dX, dW = outs
        _want(loss, (T,), torch.float32, dev, "loss")
        if dX is not None:
            _want(dX, tuple(X.shape), bf, dev, "dX")
        if dW is not None:
            _want(dW, tuple(W.shape), bf, dev, "dW")
    if ws is None:
        nb = head_workspace_bytes(T, W.shape[0], W.shape[1], k, dX is not None, dW is not None)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    else:
        nb = _ws_bytes(ws, dev)
    _on_gpu(X)
    return X, W, loss, dX, dW, ws, nb


def head_ce(X: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, weight: torch.Tensor | None = None,
            need_dx: bool = True, need_dw: bool = False, ws: torch.Tensor | None = None, outs: tuple | None = None):
    """Softmax cross entropy of z = X W^T (output layer W, bf16 [n_vocab, n_in]) without storing the logits.

    labels int64 [T]; a label outside the vocabulary ignores its row. Returns (loss float32 [T], dX or None, dW or
    None), the gradients of sum(weight * loss) (weight float32 [T], default 1). ``outs`` are optional preallocated
    (loss, dX or None, dW or None), which then say which gradients are formed."""
    if not isinstance(labels, torch.Tensor) or labels.dtype != torch.int64:
        raise TypeError("labels must be an int64 tensor")
    X, W, loss, dX, dW, ws, nb = _head_args(X, W, weight, 0, need_dx, need_dw, ws, outs)
    _want(labels, (X.shape[0],), torch.int64, X.device, "labels")
    _check(load_library().qlora_head_ce(_ptr(X), X.shape[0], _ptr(W), W.shape[0], W.shape[1], _ptr(labels),
                                        _ptr(weight), _ptr(loss), _ptr(dX), _ptr(dW), _ptr(ws), nb,
                                        _stream(X.device)), "qlora_head_ce")
    return loss, dX, dW


def head_distill(X: torch.Tensor, W: torch.Tensor, index: torch.Tensor, logit: torch.Tensor, tau: float = 1.0,
                 weight: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = False,
                 ws: torch.Tensor | None = None, outs: tuple | None = None):
    """tau^2 KL(teacher's softmax over its top logits || softmax(X W^T / tau)) without storing the logits.

    index int32 [T, k] and logit float32 [T, k] are the teacher's; entries outside the vocabulary (-1) or at -inf have
    no part. Returns (loss, dX or None, dW or None) as ``head_ce`` does."""
    for t, dt, name in ((index, torch.int32, "index"), (logit, torch.float32, "logit")):
        if not isinstance(t, torch.Tensor) or t.dtype != dt or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D {dt} tensor")
    k = index.shape[1]
    if not 1 <= k <= MAX_TARGETS:
        raise ValueError(f"1 to {MAX_TARGETS} teacher logits per row, got {k}")
    X, W, loss, dX, dW, ws, nb = _head_args(X, W, weight, k, need_dx, need_dw, ws, outs)
    _want(index, (X.shape[0], k), torch.int32, X.device, "index")
    _want(logit, (X.shape[0], k), torch.float32, X.device, "logit")
    _check(load_library().qlora_head_distill(_ptr(X), X.shape[0], _ptr(W), W.shape[0], W.shape[1], _ptr(index),
                                             _ptr(logit), k, float(tau), _ptr(weight), _ptr(loss), _ptr(dX), _ptr(dW),
                                             _ptr(ws), nb, _stream(X.device)), "qlora_head_distill")
    return loss, dX, dW


class QLoRALinearFn(torch.autograd.Function):
    """Autograd wrapper: forward(X, w, A, B, alpha) -> Y; gradients for X, A, B only."""

    @staticmethod
    def forward(ctx, X, w: NF4Weight, A, B, alpha: float):
        Y, U = linear_fwd(X, w, A, B, alpha, save_u=True)
        ctx.save_for_backward(X, A, B, U)
        ctx.w, ctx.alpha = w, alpha
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, A, B, U = ctx.saved_tensors
        dX, dA, dB = linear_bwd(X, dY.contiguous(), ctx.w, A, B, ctx.alpha, U=U, need_dx=ctx.needs_input_grad[0])
        return dX, None, dA, dB, None


def _sum(x):
    # In pieces that one workgroup adds each: torch's sum over several workgroups clears its counters with a memset, which
    # does not replay reliably from a captured graph.
    while x.numel() > 4096:
        x = torch.nn.functional.pad(x, (0, -x.numel() % 1024)).view(-1, 1024).sum(1)
    return x.sum()


def _head_total(ctx, loss, weight, dX, dW, weight_at, recorded):
    ctx.have = (dX is not None, dW is not None)
    ctx.weight_at = weight_at if recorded and weight is not None and ctx.needs_input_grad[weight_at] else None
    ctx.save_for_backward(*(t for t in (dX, dW, loss if ctx.weight_at else None) if t is not None))
    ctx.mark_non_differentiable(loss)
    # (an ignored row's weight may be anything)
    return _sum(loss if weight is None else torch.where(loss == 0, loss, loss * weight)), loss


def _head_grads(ctx, g):
    saved = list(ctx.saved_tensors)
    grads = [None] * len(ctx.needs_input_grad)
    for at in (0, 1):
        if ctx.have[at]:
            grads[at] = saved.pop(0) * g
    if ctx.weight_at:
        grads[ctx.weight_at] = saved.pop(0) * g
    return tuple(grads)


class HeadCEFn(torch.autograd.Function):
    """Autograd wrapper of ``head_ce``: forward(X, W, labels, weight) -> (sum(weight * loss), loss [T]).

    The gradients are formed with the losses, in one call, for those of X and W that need them (for neither where
    gradients are off, as under ``torch.no_grad``); the backward multiplies them by the incoming scalar (and the losses,
    for a weight that needs a gradient). They are bf16, so a scalar that is no power of two rounds them once more: a mean's
    1 / n belongs into ``weight``. The per-token losses carry no gradient. Forward and backward can be captured into a HIP
    graph, as any autograd function, where no eager graph of the same leaves is alive."""

    @classmethod
    def apply(cls, X, W, labels, weight=None):
        # (inside forward gradients are always off, and needs_input_grad does not know whether they were before)
        return super().apply(X, W, labels, weight, torch.is_grad_enabled())

    @staticmethod
    def forward(ctx, X, W, labels, weight, recorded):
        loss, dX, dW = head_ce(X, W, labels, weight, need_dx=recorded and ctx.needs_input_grad[0],
                               need_dw=recorded and ctx.needs_input_grad[1])
        return _head_total(ctx, loss, weight, dX, dW, 3, recorded)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g, _):
        return _head_grads(ctx, g)


class HeadDistillFn(torch.autograd.Function):
    """Autograd wrapper of ``head_distill``: forward(X, W, index, logit, tau, weight) -> (sum(weight * loss), loss [T]).

    As ``HeadCEFn``; the teacher's logits get no gradient, so ones that ask for it are refused."""

    @classmethod
    def apply(cls, X, W, index, logit, tau=1.0, weight=None):
        return super().apply(X, W, index, logit, tau, weight, torch.is_grad_enabled())

    @staticmethod
    def forward(ctx, X, W, index, logit, tau, weight, recorded):
        if recorded and ctx.needs_input_grad[3]:
            raise ValueError("the teacher's logits get no gradient: detach them")
        loss, dX, dW = head_distill(X, W, index, logit, tau, weight, need_dx=recorded and ctx.needs_input_grad[0],
                                    need_dw=recorded and ctx.needs_input_grad[1])
        return _head_total(ctx, loss, weight, dX, dW, 5, recorded)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g, _):
        return _head_grads(ctx, g)


def timing_enable(kernel: str, enable: bool = True):
    _check(load_library().qlora_timing_enable(kernel.encode(), 1 if enable else 0), "qlora_timing_enable")


def timing_read(kernel: str) -> tuple[int, float]:
    n, ms = ctypes.c_int64(), ctypes.c_double()
    _check(load_library().qlora_timing_read(kernel.encode(), ctypes.byref(n), ctypes.byref(ms)), "qlora_timing_read")
    return n.value, ms.value


def timing_read_each(kernel: str, cap: int = 1 << 16) -> list:
    """Milliseconds of each recorded launch of `kernel`, in launch order (clears the record)."""
    buf = (ctypes.c_double * cap)()
    n = ctypes.c_int64()
    _check(load_library().qlora_timing_read_each(kernel.encode(), buf, cap, ctypes.byref(n)),
           "qlora_timing_read_each")
    return list(buf[:min(cap, n.value)])

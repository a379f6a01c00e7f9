"""8-bit floating point (e4m3) linear layer with one scale per block of 128.

For projections that do not stand 4 bits, or whose weights come from a
checkpoint in this format: activations have one float32 scale per token and
128 columns, weights one per 128 x 128 tile, and an e4m3 code c of a block with
scale s stands for c * s.

    w = pack_weight(W)                    # or Fp8Weight(q, scale) from a checkpoint
    ws = torch.empty(workspace_size(T, w), dtype=torch.uint8, device="cuda")
    linear(X, w, ws, Y)                   # quant_act, then gemm

quant_act and pack_weight choose the smallest power of two s with
max|x| <= 448 s; the product takes any float32 scales.  Every call checks its
tensors and the status the library returns, runs on the tensors' device and on
the given stream (default: that device's current stream), and allocates
nothing unless it says so.  Calls that may overlap on the GPU need workspaces
of their own.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass, field

import torch

from . import (ERR_INVALID_ARG, OK, W4A4Error, _check, _i64, _rows_bf16, _sig, _st, _vp)

BLOCK = 128
_BF16, _F32 = torch.bfloat16, torch.float32

# the handle of a device's current stream and the current device, without the
# objects and checks around them where torch offers that (2 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class Fp8WeightC(ctypes.Structure):
    _fields_ = [("d_in", _i64), ("d_out", _i64), ("experts", _i64), ("q", _vp), ("scale", _vp)]


_PW = ctypes.POINTER(Fp8WeightC)
_quant_act = _sig("w4a4_fp8_quant_act", _st, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp)
_pack_weight = _sig("w4a4_fp8_pack_weight", _st, _vp, _i64, _PW, _vp)
_gemm = _sig("w4a4_fp8_gemm", _st, _vp, _vp, _i64, _i64, _PW, _vp, _i64, ctypes.c_int, _vp)
_workspace_size = _sig("w4a4_fp8_workspace_size", _st, _i64, _i64, ctypes.POINTER(ctypes.c_size_t))
_linear = _sig("w4a4_fp8_linear", _st, _vp, _i64, _i64, _PW, _vp, ctypes.c_size_t, _vp, _i64,
               ctypes.c_int, _vp)


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _run(device: torch.device, stream, what: str, fn, *args):
    """fn(*args, stream) with `device` current; raises on a non-OK status."""
    index = device.index
    if stream is None:
        s = _raw_stream(index)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == _device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(device):
            st = fn(*args, s)
    if st != OK:
        _check(st, what)


def _allocating(device: torch.device, stream):
    """Context in which new tensors are `stream`'s: memory freed on the current
    stream, whose work there may not have run yet, must not be written by another."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(s, device=device) if s else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _dense(t: torch.Tensor, dtypes, shape, device, what: str):
    """A dense tensor of one of `dtypes`, `shape` and `device`."""
    if t.dtype not in dtypes or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or \
            not t.is_cuda or (device is not None and t.device != device):
        raise W4A4Error(ERR_INVALID_ARG,
                        f"{what}: needs a dense {'/'.join(str(d) for d in dtypes)} CUDA tensor of "
                        f"shape {tuple(shape)}{' on ' + str(device) if device is not None else ''} "
                        f"(got {t.dtype}, {tuple(t.shape)}, strides {tuple(t.stride())}, {t.device})")


def _bytes(t: torch.Tensor, device, what: str):
    """A workspace: any dense CUDA tensor on `device`."""
    if t.device != device or not t.is_contiguous():
        raise W4A4Error(ERR_INVALID_ARG, f"{what}: the workspace must be a dense tensor on {device} "
                                         f"(got strides {tuple(t.stride())}, {t.device})")


def _rows_in(X: torch.Tensor, cols: int, device, what: str):
    """bf16 rows [T, cols] on `device`; T and the row stride."""
    if X.dtype is _BF16 and X.is_cuda and X.device == device and X.dim() == 2:
        (T, n), (ld, one) = X.shape, X.stride()
        if n == cols and one == 1:
            return T, ld if T > 1 else cols + 7 & ~7
    _rows_bf16(X, what, device)
    if X.shape[1] != cols:
        raise W4A4Error(ERR_INVALID_ARG, f"{what}: X has {X.shape[1]} columns, not {cols}")
    return X.shape[0], _ld(X)


def _rows_out(Y: torch.Tensor, rows: int, cols: int, device, what: str):
    """An output [rows, cols], bf16 or float32, unit column stride; its row stride and y_f32."""
    f32 = Y.dtype is _F32
    if (f32 or Y.dtype is _BF16) and Y.device == device and Y.shape == (rows, cols) and \
            (cols <= 1 or Y.stride(1) == 1):
        return _ld(Y), f32
    raise W4A4Error(ERR_INVALID_ARG,
                    f"{what}: Y must be bfloat16 or float32 [{rows}, {cols}] on {device} with unit "
                    f"column stride (got {Y.dtype}, {tuple(Y.shape)}, strides {tuple(Y.stride())}, "
                    f"{Y.device})")


def _ld(t: torch.Tensor) -> int:
    """Row stride of a 2-D tensor; of one with at most one row, its dense row stride."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1] + 7 & ~7, 8)


_F8 = (torch.uint8, torch.float8_e4m3fn)


# The records below are frozen: what the library gets of one (sizes, pointers) is
# taken from its fields when it is made, and none can be assigned after that.  A
# tensor's own memory can still be exchanged (t.data = ...; t.set_(...); t.resize_(...)),
# so each call first looks whether the tensors are where they were (0.2 us) and, if
# one is not, checks and takes everything anew.
def _put(record, **values):
    for name, value in values.items():
        object.__setattr__(record, name, value)


@dataclass(frozen=True)
class Fp8Weight:
    """e4m3 codes [d_out, d_in] with float32 scales [ceil(d_out/128),
    ceil(d_in/128)], or a stack of them with a leading dimension."""
    q: torch.Tensor
    scale: torch.Tensor
    device: torch.device = field(init=False, repr=False, compare=False)
    d_in: int = field(init=False, repr=False, compare=False)
    d_out: int = field(init=False, repr=False, compare=False)
    experts: int = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if self.q.dim() not in (2, 3):
            raise W4A4Error(ERR_INVALID_ARG, f"Fp8Weight: q has {self.q.dim()} dimensions, not 2 or 3")
        lead, (d_out, d_in) = tuple(self.q.shape[:-2]), self.q.shape[-2:]
        _dense(self.q, _F8, self.q.shape, None, "Fp8Weight q")
        _dense(self.scale, (torch.float32,), lead + (blocks(d_out), blocks(d_in)), self.q.device,
               "Fp8Weight scale")
        at = self.q.data_ptr(), self.scale.data_ptr()
        experts = int(lead[0]) if lead else 1
        c = Fp8WeightC(int(d_in), int(d_out), experts, *at)
        _put(self, device=self.q.device, d_in=int(d_in), d_out=int(d_out), experts=experts, _at=at,
             _by=ctypes.byref(c))

    @property
    def _ref(self):
        if (self.q.data_ptr(), self.scale.data_ptr()) != self._at:
            self.__post_init__()
        return self._by

    @property
    def c(self) -> Fp8WeightC:
        """The C record, a copy."""
        return Fp8WeightC.from_buffer_copy(self._ref._obj)


@dataclass(frozen=True)
class Fp8Act:
    """Quantised activations: q uint8 [T, d], scale float32 [ceil(d/128), ld]
    (token t and block b at [b, t]; ld is T rounded up to 4, or more)."""
    q: torch.Tensor
    scale: torch.Tensor
    device: torch.device = field(init=False, repr=False, compare=False)
    T: int = field(init=False, repr=False, compare=False)
    d: int = field(init=False, repr=False, compare=False)
    ld: int = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if self.q.dim() != 2 or self.scale.dim() != 2:
            raise W4A4Error(ERR_INVALID_ARG, "Fp8Act: q and scale are 2-D")
        (T, d), ld, device = (int(n) for n in self.q.shape), int(self.scale.shape[1]), self.q.device
        if ld < (T + 3) // 4 * 4:
            raise W4A4Error(ERR_INVALID_ARG, f"Fp8Act: no room for {T} scales in rows of {ld}")
        if device.type == "cuda":
            _dense(self.q, _F8, (T, d), device, "Fp8Act q")
            _dense(self.scale, (_F32,), (blocks(d), ld), device, "Fp8Act scale")
        at = self.q.data_ptr(), self.scale.data_ptr()
        _put(self, device=device, T=T, d=d, ld=ld, _at=at, _arg=(*at, ld))

    @property
    def _args(self):
        if (self.q.data_ptr(), self.scale.data_ptr()) != self._at:
            self.__post_init__()
        return self._arg


def alloc_act(T: int, d: int, device="cuda") -> Fp8Act:
    return Fp8Act(torch.empty((T, d), dtype=torch.uint8, device=device),
                  torch.empty((blocks(d), max(4, (T + 3) // 4 * 4)), dtype=torch.float32, device=device))


def quant_act(X: torch.Tensor, out: Fp8Act, stream=None) -> Fp8Act:
    args = out._args
    T, ld = _rows_in(X, out.d, out.device, "fp8.quant_act")
    if T != out.T:
        raise W4A4Error(ERR_INVALID_ARG, f"fp8.quant_act: X has {T} rows, out {out.T}")
    _run(out.device, stream, "fp8.quant_act", _quant_act, X.data_ptr(), T, out.d, ld, *args)
    return out


def pack_weight(W: torch.Tensor, stream=None) -> Fp8Weight:
    """Quantises W, bf16 [d_out, d_in] or dense [experts, d_out, d_in]; allocates the
    result, on `stream` where one is given."""
    if W.dim() == 3:
        _dense(W, (torch.bfloat16,), W.shape, None, "fp8.pack_weight")
        ldw = W.shape[2]
    else:
        _rows_bf16(W, "fp8.pack_weight")
        ldw = _ld(W)
    d_out, d_in = W.shape[-2:]
    with _allocating(W.device, stream):
        w = Fp8Weight(torch.empty(W.shape, dtype=torch.uint8, device=W.device),
                      torch.empty(tuple(W.shape[:-2]) + (blocks(d_out), blocks(d_in)), dtype=torch.float32,
                                  device=W.device))
    _run(W.device, stream, "fp8.pack_weight", _pack_weight, W.data_ptr(), ldw, w._ref)
    return w


def gemm(act: Fp8Act, w: Fp8Weight, Y: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = act @ w^T, bf16 or float32 by Y's type."""
    args, ref = act._args, w._ref
    if act.d != w.d_in or act.device != w.device:
        raise W4A4Error(ERR_INVALID_ARG, f"fp8.gemm: activations of {act.d} columns on {act.device}, weight "
                                         f"of {w.d_in} on {w.device}")
    ld, f32 = _rows_out(Y, act.T, w.d_out, w.device, "fp8.gemm")
    _run(w.device, stream, "fp8.gemm", _gemm, *args, act.T, ref, Y.data_ptr(), ld, f32)
    return Y


def workspace_size(T: int, w: Fp8Weight) -> int:
    n = ctypes.c_size_t()
    _check(_workspace_size(T, w.d_in, ctypes.byref(n)), "fp8.workspace_size")
    return n.value


def linear(X: torch.Tensor, w: Fp8Weight, workspace: torch.Tensor, Y: torch.Tensor,
           stream=None) -> torch.Tensor:
    """Y = quant_act(X) @ w^T, bf16 or float32 by Y's type."""
    ref, dev = w._ref, w.device
    T, ldx = _rows_in(X, w.d_in, dev, "fp8.linear")
    ldy, f32 = _rows_out(Y, T, w.d_out, dev, "fp8.linear")
    _bytes(workspace, dev, "fp8.linear")
    _run(dev, stream, "fp8.linear", _linear, X.data_ptr(), T, ldx, ref, workspace.data_ptr(),
         workspace.nbytes, Y.data_ptr(), ldy, f32)
    return Y

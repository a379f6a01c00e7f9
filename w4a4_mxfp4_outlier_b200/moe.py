"""Mixture-of-experts layer for a few tokens on e4m3 expert weights.

The expert form of the FFN: a router picks top_k experts for each token, each
expert is an up projection (with a gate, or GELU alone) and a down projection
in the 8-bit format of w4a4_mxfp4_outlier_b200.fp8, and the chosen experts'
outputs are summed with the router's softmax weights.  The whole layer is two
kernels that read each chosen expert's weights once; up to 64 tokens.

    m = MoE(router, gate, up, down, top_k=8)      # gate=None with act=GELU
    ws = torch.empty(workspace_size(T, m), dtype=torch.uint8, device="cuda")
    forward(X, m, ws, Y)

Calls that may overlap on the GPU need workspaces of their own.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import ERR_INVALID_ARG, W4A4Error, _check, _i64, _sig, _st, _vp
from .fp8 import Fp8Weight, Fp8WeightC, _bytes, _dense, _put, _rows_in, _rows_out, _run

GELU, SILU_GATED = 0, 1          # W4A4_MOE_GELU, W4A4_MOE_SILU_GATED
MAX_TOKENS = 64


class ExpertsC(ctypes.Structure):
    _fields_ = [("top_k", _i64), ("act", ctypes.c_int32), ("renorm", ctypes.c_int32), ("router", _vp),
                ("gate", Fp8WeightC), ("up", Fp8WeightC), ("down", Fp8WeightC)]


_PE = ctypes.POINTER(ExpertsC)
_moe_workspace_size = _sig("w4a4_fp8_moe_workspace_size", _st, _PE, _i64,
                           ctypes.POINTER(ctypes.c_size_t))
_moe = _sig("w4a4_fp8_moe", _st, _vp, _i64, _i64, _PE, _vp, ctypes.c_size_t, _vp, _i64, ctypes.c_int,
            _vp, _vp, _vp)


@dataclass(frozen=True)
class MoE:
    """router bf16 [E, d]; gate and up [E, d_ff, d], down [E, d, d_ff] (Fp8Weight).
    Another layer is another MoE: no field can be assigned (see fp8)."""
    router: torch.Tensor
    gate: Fp8Weight | None
    up: Fp8Weight
    down: Fp8Weight
    top_k: int
    act: int = SILU_GATED
    renorm: bool = True

    def __post_init__(self):
        records = [w.c if w is not None else Fp8WeightC() for w in (self.gate, self.up, self.down)]
        up, dev = self.up, self.up.device
        _dense(self.router, (torch.bfloat16,), (up.experts, up.d_in), dev, "MoE router")
        if (self.gate is None) != (self.act == GELU):
            raise W4A4Error(ERR_INVALID_ARG, "MoE: a gate goes with SILU_GATED, none with GELU")
        for w, shape, what in ((self.gate, (up.d_out, up.d_in), "gate"),
                               (self.down, (up.d_in, up.d_out), "down")):
            if w is not None and ((w.d_out, w.d_in) != shape or w.experts != up.experts or w.device != dev):
                raise W4A4Error(ERR_INVALID_ARG, f"MoE: {what} is {w.experts} x [{w.d_out}, {w.d_in}] on "
                                f"{w.device}, not {up.experts} x {list(shape)} on {dev}")
        c = ExpertsC(self.top_k, self.act, int(self.renorm), self.router.data_ptr(), *records)
        _put(self, _at=self._where(), _by=ctypes.byref(c))

    def _where(self):
        g, u, d = self.gate, self.up, self.down
        at = (self.router.data_ptr(), u.q.data_ptr(), u.scale.data_ptr(), d.q.data_ptr(), d.scale.data_ptr())
        return at if g is None else (*at, g.q.data_ptr(), g.scale.data_ptr())

    @property
    def _ref(self):
        if self._where() != self._at:
            self.__post_init__()
        return self._by

    @property
    def c(self) -> ExpertsC:
        """The C record, a copy."""
        return ExpertsC.from_buffer_copy(self._ref._obj)


def workspace_size(T: int, m: MoE) -> int:
    n = ctypes.c_size_t()
    _check(_moe_workspace_size(m._ref, T, ctypes.byref(n)), "moe.workspace_size")
    return n.value


def forward(X: torch.Tensor, m: MoE, workspace: torch.Tensor, Y: torch.Tensor,
            ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Y = the layer of X, bf16 or float32 by Y's type; ids int32 and weights
    float32, both [T, top_k], receive the selection where given."""
    ref, d, dev = m._ref, m.up.d_in, m.up.device
    T, ldx = _rows_in(X, d, dev, "moe.forward")
    ldy, f32 = _rows_out(Y, T, d, dev, "moe.forward")
    _bytes(workspace, dev, "moe.forward")
    if ids is not None:
        _dense(ids, (torch.int32,), (T, m.top_k), dev, "moe.forward ids")
    if weights is not None:
        _dense(weights, (torch.float32,), (T, m.top_k), dev, "moe.forward weights")
    _run(dev, stream, "moe.forward", _moe, X.data_ptr(), T, ldx, ref, workspace.data_ptr(),
         workspace.nbytes, Y.data_ptr(), ldy, f32, None if ids is None else ids.data_ptr(),
         None if weights is None else weights.data_ptr())
    return Y

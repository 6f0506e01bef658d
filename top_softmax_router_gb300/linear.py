"""Python binding of the products grouped by expert (include/moe_linear.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _args, _lib
from ._lib import LinearConfig as _C
from ._lib import check
from .blocks8 import CODES, SCALES, blocks

__all__ = ["ExpertLinearConfig", "ExpertLinear", "linear_workspace_bytes"]


@dataclasses.dataclass(frozen=True)
class ExpertLinearConfig:
    N: int                   # rows (the most a call may have)
    K: int                   # columns of x (multiple of 16)
    O: int                   # columns of y (multiple of 16)
    E: int = 1               # experts, up to 1024
    blocks8: bool = False    # room for the backward pass of operands in 8 bits

    def c_struct(self, n=None):
        return _C(self.N if n is None else n, self.K, self.O, self.E, int(self.blocks8))


def linear_workspace_bytes(cfg: ExpertLinearConfig) -> tuple[int, int]:
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    check(_lib.load().moe_linear_workspace_bytes(ctypes.byref(cfg.c_struct()), ctypes.byref(f), ctypes.byref(b)),
          "moe_linear_workspace_bytes")
    return f.value, b.value


class ExpertLinear:
    """Owns the workspace for up to N rows; calls on one object run on one stream at a time."""

    def __init__(self, cfg: ExpertLinearConfig, device="cuda"):
        self.cfg = cfg
        self._c = _args.Structs(cfg)
        self._shared, most = linear_workspace_bytes(cfg)   # what both passes use comes first
        self.ws = _args.workspace(most, device)

    def _x(self, x, scales):
        c = self.cfg
        n = _args.count(x, "x", c.N)
        xp, ldx = _args.rows(x, "x", torch.bfloat16 if scales is None else CODES, (n, c.K))
        if xp % 16 or ldx * x.element_size() % 16:
            raise ValueError("x: expected rows that lie on 16 bytes")
        return n, xp, ldx, _args.ptr(scales, "x_scales", SCALES, (n, blocks(c.K)))

    def _w(self, w, scales):
        c = self.cfg
        wp = _args.ptr(w, "w", torch.bfloat16 if scales is None else CODES, (c.E, c.O, c.K))
        if wp is None:
            raise TypeError("w: expected a torch.Tensor")
        return wp, _args.ptr(scales, "w_scales", SCALES, (c.E, blocks(c.O), blocks(c.K)))

    def _offsets(self, offsets):
        if offsets is None and self.cfg.E != 1:
            raise ValueError("offsets: needed for more than one expert")
        return _args.ptr(offsets, "offsets", torch.int32, (self.cfg.E + 1,))

    def forward(self, x, w, offsets=None, x_scales=None, w_scales=None, stream=None):
        """x [n <= N, K] (rows may be strided), w [E, O, K]: bf16, or float8_e4m3fn codes with their scales
        (Checkpoint8.pack or RMSNorm; pack_weight8).  offsets [E + 1] int32: rows offsets[e] .. offsets[e + 1] are
        expert e's (None: all rows are the one expert's).  -> y [n, O] bf16, 0 in rows of no expert."""
        c = self.cfg
        if (x_scales is None) != (w_scales is None):
            raise ValueError("x_scales and w_scales: expected both or neither")
        n, xp, ldx, xs = self._x(x, x_scales)
        wp, wsp = self._w(w, w_scales)
        op = self._offsets(offsets)
        _args.here(self.ws.device, x, w, offsets, x_scales, w_scales)
        on = _args.On(stream, x.device)
        y = on.empty((n, c.O), torch.bfloat16, x.device)
        check(_lib.load().moe_linear_forward(self._c(n), xp, ldx, xs, wp, wsp, op, y.data_ptr(), self.ws.data_ptr(),
                                             self.ws.numel(), on.handle), "moe_linear_forward")
        on.uses(x, w, offsets, x_scales, w_scales, self.ws)
        return y

    def backward(self, x, w, dy, offsets=None, x_scales=None, w_scales=None, want_dx=True, want_dw=True,
                 dw_dtype=torch.float32, stream=None):
        """dy [n, O] bf16 -> dx [n, K] bf16, dw [E, O, K] in dw_dtype (float32 or bfloat16); None for what is not
        wanted.  x and w as in the forward, or x alone in 8 bits: a checkpoint.  With w in 8 bits dx is the product of
        dy packed in 8 bits, too; dw takes dy as it is.  x may be None without dw, w without dx."""
        c = self.cfg
        n = _args.count(dy, "dy", c.N)
        gp = _args.ptr(dy, "dy", torch.bfloat16, (n, c.O))
        xp, ldx, xs, wp, wsp = None, c.K, None, None, None
        if want_dw:
            nx, xp, ldx, xs = self._x(x, x_scales)
            if nx != n:
                raise ValueError(f"dy: expected shape {(nx, c.O)}, got {(n, c.O)}")
            if xs is not None and ldx != c.K:
                raise ValueError("x: expected a contiguous tensor")
        if want_dx:
            wp, wsp = self._w(w, w_scales)
        if (xs is not None or wsp is not None) and not c.blocks8:
            raise ValueError("operands in 8 bits: the unit was made without blocks8")
        if want_dw and dw_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dw_dtype: expected torch.bfloat16 or torch.float32")
        op = self._offsets(offsets)
        _args.here(self.ws.device, dy, offsets, *((x, x_scales) if want_dw else ()), *((w, w_scales) if want_dx else ()))
        on = _args.On(stream, dy.device)
        dx = on.empty((n, c.K), torch.bfloat16, dy.device) if want_dx else None
        dw = on.empty((c.E, c.O, c.K), dw_dtype, dy.device) if want_dw else None
        check(_lib.load().moe_linear_backward(
            self._c(n), xp, ldx, xs, wp, wsp, op, gp, dx.data_ptr() if want_dx else None,
            dw.data_ptr() if want_dw else None, _args.TYPES[dw_dtype] if want_dw else 0, self.ws.data_ptr(), self.ws.numel(), on.handle),
            "moe_linear_backward")
        on.uses(x, w, dy, offsets, x_scales, w_scales, self.ws)
        return dx, dw

    def check(self, stream=None) -> None:
        """Raises if a call since the last check met offsets that are none, or a wait ran out; the workspace is then as
        new for calls on `stream`, the one the unit's calls ran on."""
        from .api import check_status
        on = _args.On(stream, self.ws.device)
        code = check_status(self.ws, on.handle)
        if code:
            with torch.cuda.stream(on.stream):     # before the next call there, whatever the current stream
                self.ws[:self._shared].zero_()     # the shares and their counters; nothing else has to be zero
        check(code, "device status")

"""Python binding of the root-mean-square norm (include/moe_rmsnorm.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _args, _lib
from ._lib import RmsNormConfig as _C
from ._lib import check
from .blocks8 import CODES, SCALES, blocks

__all__ = ["RMSNormConfig", "RMSNorm", "rmsnorm_workspace_bytes"]


@dataclasses.dataclass(frozen=True)
class RMSNormConfig:
    N: int               # rows (the most a call may have)
    H: int               # row width, up to 16384
    eps: float = 1e-6

    def c_struct(self, n=None):
        return _C(self.N if n is None else n, self.H, self.eps)


def rmsnorm_workspace_bytes(cfg: RMSNormConfig) -> int:
    b = ctypes.c_size_t()
    check(_lib.load().moe_rmsnorm_workspace_bytes(ctypes.byref(cfg.c_struct()), ctypes.byref(b)),
          "moe_rmsnorm_workspace_bytes")
    return b.value


class RMSNorm:
    """Owns the backward's workspace for up to N rows; calls on one object run on one stream at a time."""

    def __init__(self, cfg: RMSNormConfig, device="cuda"):
        self.cfg = cfg
        self._c = _args.Structs(cfg)
        self.ws = _args.workspace(rmsnorm_workspace_bytes(cfg), device)

    def _weight(self, x, weight):
        p = _args.ptr(weight, "weight", _args.TYPES, (self.cfg.H,))
        if weight is not None and weight.dtype != torch.float32 and weight.dtype != x.dtype:
            raise TypeError(f"weight: expected float32 or {x.dtype}")
        return p, _args.TYPES[x.dtype if weight is None else weight.dtype]

    def forward(self, x, weight=None, residual=None, want_y=True, want_codes=False, stream=None):
        """x, residual [n <= N, H] (rows may be strided; residual None: none); weight [H] or None -> y, h, rstd, codes,
        scales: the norm of h = x + residual (x itself without one) in x's type, and in 8 bits as Checkpoint8.pack makes
        them; None for what is not wanted."""
        c = self.cfg
        n = _args.count(x, "x", c.N)
        xp, ldx = _args.rows(x, "x", _args.TYPES, (n, c.H))
        rp, ldr = (None, c.H) if residual is None else _args.rows(residual, "residual", x.dtype, (n, c.H))
        wp, pt = self._weight(x, weight)
        _args.here(self.ws.device, x, weight, residual)
        on = _args.On(stream, x.device)
        h = x if residual is None else on.empty((n, c.H), x.dtype, x.device)
        y = on.empty((n, c.H), x.dtype, x.device) if want_y else None
        rstd = on.empty((n,), torch.float32, x.device)
        codes = on.empty((n, c.H), CODES, x.device) if want_codes else None
        scales = on.empty((n, blocks(c.H)), SCALES, x.device) if want_codes else None
        check(_lib.load().moe_rmsnorm_forward(
            self._c(n), xp, ldx, rp, ldr, wp, None if residual is None else h.data_ptr(),
            y.data_ptr() if want_y else None, codes.data_ptr() if want_codes else None,
            scales.data_ptr() if want_codes else None, rstd.data_ptr(), _args.TYPES[x.dtype], pt, on.handle),
            "moe_rmsnorm_forward")
        on.uses(x, weight, residual)
        return y, h, rstd, codes, scales

    def backward(self, h, weight, rstd, dy, dh=None, want_dx=True, want_dweight=True, stream=None):
        """h, rstd from the forward; dy the output's gradient, dh that of h from elsewhere (None: 0), in h's type, rows
        may be strided -> dx [n, H], the gradient of x and of the residual alike, dweight [H] fp32 (None for what is not
        wanted)."""
        c = self.cfg
        n = _args.count(h, "h", c.N)
        hp, ldh = _args.rows(h, "h", _args.TYPES, (n, c.H))
        gp, ldg = _args.rows(dy, "dy", h.dtype, (n, c.H))
        dp, ldd = (None, c.H) if dh is None else _args.rows(dh, "dh", h.dtype, (n, c.H))
        wp, pt = self._weight(h, weight)
        sp = _args.ptr(rstd, "rstd", torch.float32, (n,))
        if sp is None:
            raise TypeError("rstd: expected a torch.Tensor")
        _args.here(self.ws.device, h, weight, rstd, dy, dh)
        on = _args.On(stream, h.device)
        dx = on.empty((n, c.H), h.dtype, h.device) if want_dx else None
        dw = on.empty((c.H,), torch.float32, h.device) if want_dweight else None
        check(_lib.load().moe_rmsnorm_backward(
            self._c(n), hp, ldh, wp, sp, gp, ldg, dp, ldd, dx.data_ptr() if want_dx else None,
            dw.data_ptr() if want_dweight else None, _args.TYPES[h.dtype], pt, self.ws.data_ptr(), self.ws.numel(),
            on.handle), "moe_rmsnorm_backward")
        on.uses(h, weight, rstd, dy, dh, self.ws)
        return dx, dw

"""Python binding of layer normalisation (include/moe_norm.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _args, _lib
from ._lib import LayerNormConfig as _C
from ._lib import check

__all__ = ["LayerNormConfig", "LayerNorm", "layernorm_workspace_bytes"]


@dataclasses.dataclass(frozen=True)
class LayerNormConfig:
    N: int               # rows (the most a call may have)
    H: int               # row width, up to 16384
    eps: float = 1e-5

    def c_struct(self, n=None):
        return _C(self.N if n is None else n, self.H, self.eps)


def layernorm_workspace_bytes(cfg: LayerNormConfig) -> int:
    b = ctypes.c_size_t()
    check(_lib.load().moe_layernorm_workspace_bytes(ctypes.byref(cfg.c_struct()), ctypes.byref(b)),
          "moe_layernorm_workspace_bytes")
    return b.value


class LayerNorm:
    """Owns the backward's workspace for up to N rows; calls on one object run on one stream at a time."""

    def __init__(self, cfg: LayerNormConfig, device="cuda"):
        self.cfg = cfg
        self._c = _args.Structs(cfg)
        self.ws = _args.workspace(layernorm_workspace_bytes(cfg), device)

    def _params(self, x, weight, bias):
        if weight is not None and bias is not None and weight.dtype != bias.dtype:
            raise TypeError("weight and bias: expected one type")
        p = weight if weight is not None else bias
        if p is None:
            return _args.TYPES[x.dtype]
        if p.dtype != torch.float32 and p.dtype != x.dtype:
            raise TypeError(f"weight and bias: expected float32 or {x.dtype}")
        return _args.TYPES[p.dtype]

    def forward(self, x, weight=None, bias=None, stream=None):
        """x [n <= N, H] (rows may be strided); weight, bias [H] or None -> y [n, H], mean [n], rstd [n]."""
        c = self.cfg
        n = _args.count(x, "x", c.N)
        xp, ldx = _args.rows(x, "x", _args.TYPES, (n, c.H))
        wp, bp = _args.ptr(weight, "weight", _args.TYPES, (c.H,)), _args.ptr(bias, "bias", _args.TYPES, (c.H,))
        pt = self._params(x, weight, bias)
        on = _args.On(stream, x.device)
        y = on.empty((n, c.H), x.dtype, x.device)
        mean, rstd = on.empty((n,), torch.float32, x.device), on.empty((n,), torch.float32, x.device)
        check(_lib.load().moe_layernorm_forward(self._c(n), xp, ldx, wp, bp, y.data_ptr(),
                                                mean.data_ptr(), rstd.data_ptr(), _args.TYPES[x.dtype], pt,
                                                on.handle), "moe_layernorm_forward")
        on.uses(x, weight, bias)
        return y, mean, rstd

    def backward(self, x, weight, mean, rstd, dy, want_dx=True, want_dweight=True, want_dbias=True, stream=None):
        """mean, rstd from the forward; dy [n, H] in x's type -> dx [n, H], dweight [H] fp32, dbias [H] fp32 (None
        for what is not wanted)."""
        c = self.cfg
        n = _args.count(x, "x", c.N)
        xp, ldx = _args.rows(x, "x", _args.TYPES, (n, c.H))
        gp, ldg = _args.rows(dy, "dy", x.dtype, (n, c.H))
        wp = _args.ptr(weight, "weight", _args.TYPES, (c.H,))
        pt = self._params(x, weight, None)
        mp, rp = _args.ptr(mean, "mean", torch.float32, (n,)), _args.ptr(rstd, "rstd", torch.float32, (n,))
        on = _args.On(stream, x.device)
        dx = on.empty((n, c.H), x.dtype, x.device) if want_dx else None
        dw = on.empty((c.H,), torch.float32, x.device) if want_dweight else None
        db = on.empty((c.H,), torch.float32, x.device) if want_dbias else None
        check(_lib.load().moe_layernorm_backward(
            self._c(n), xp, ldx, wp, mp, rp, gp, ldg, dx.data_ptr() if want_dx else None,
            dw.data_ptr() if want_dweight else None, db.data_ptr() if want_dbias else None, _args.TYPES[x.dtype], pt,
            self.ws.data_ptr(), self.ws.numel(), on.handle), "moe_layernorm_backward")
        on.uses(x, weight, mean, rstd, dy, self.ws)
        return dx, dw, db

    def check(self, stream=None) -> None:
        """Raises if a wait of a backward since the last check ran out: its gradients are then of no use."""
        from .api import check_status
        check(check_status(self.ws, stream), "device status")

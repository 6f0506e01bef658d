"""Python binding of the distillation head (include/moe_distill.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _args, _lib
from ._lib import DistillConfig as _C
from ._lib import check

__all__ = ["DistillConfig", "VocabDistill", "distill_workspace_bytes"]


@dataclasses.dataclass(frozen=True)
class DistillConfig:
    N: int                     # tokens (the most a call may have)
    H: int                     # hidden size (multiple of 64)
    V: int                     # classes
    K: int                     # teacher entries a token, up to 256
    P: int = 1                 # vocabulary strips of the backward pass
    temperature: float = 1.0

    def c_struct(self, n=None):
        return _C(self.N if n is None else n, self.H, self.V, self.K, self.P, self.temperature)


def distill_workspace_bytes(cfg: DistillConfig) -> tuple[int, int]:
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    check(_lib.load().moe_distill_workspace_bytes(ctypes.byref(cfg.c_struct()), ctypes.byref(f), ctypes.byref(b)),
          "moe_distill_workspace_bytes")
    return f.value, b.value


class VocabDistill:
    """Owns the workspace for up to N tokens; calls on one object run on one stream at a time."""

    def __init__(self, cfg: DistillConfig, device="cuda"):
        self.cfg = cfg
        self._c = _args.Structs(cfg)
        self.ws = _args.workspace(max(distill_workspace_bytes(cfg)), device)

    def _inputs(self, X, W, ids, teacher):
        c = self.cfg
        n = _args.count(X, "X", c.N)
        return (n, _args.ptr(X, "X", torch.bfloat16, (n, c.H)), _args.ptr(W, "W", torch.bfloat16, (c.V, c.H)),
                _args.ptr(ids, "ids", torch.int32, (n, c.K)), _args.ptr(teacher, "teacher", torch.float32, (n, c.K)))

    def forward(self, X, W, ids, teacher, stream=None):
        """X [n <= N, H], W [V, H] bf16; ids [n, K] int32 (-1: no entry), teacher [n, K] fp32 logits -> loss [n],
        lse [n], mean [1], fp32."""
        c = self.cfg
        n, xp, wp, ip, tp = self._inputs(X, W, ids, teacher)
        on = _args.On(stream, X.device)
        loss = on.empty((n,), torch.float32, X.device)
        lse = on.empty((n,), torch.float32, X.device)
        mean = on.empty((1,), torch.float32, X.device)
        check(_lib.load().moe_distill_forward(self._c(n), xp, wp, ip, tp, loss.data_ptr(),
                                              lse.data_ptr(), mean.data_ptr(), self.ws.data_ptr(), self.ws.numel(),
                                              on.handle), "moe_distill_forward")
        on.uses(X, W, ids, teacher, self.ws)
        return loss, lse, mean

    def backward(self, X, W, ids, teacher, lse, dloss, dW_dtype=torch.bfloat16, stream=None):
        """lse from the forward; dloss [n] fp32 -> dX [n, H] bf16, dW [V, H] in dW_dtype (bfloat16 or float32)."""
        c = self.cfg
        n, xp, wp, ip, tp = self._inputs(X, W, ids, teacher)
        lp, gp = _args.ptr(lse, "lse", torch.float32, (n,)), _args.ptr(dloss, "dloss", torch.float32, (n,))
        if dW_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dW_dtype: expected torch.bfloat16 or torch.float32")
        on = _args.On(stream, X.device)
        dX = on.empty((n, c.H), torch.bfloat16, X.device)
        dW = on.empty((c.V, c.H), dW_dtype, X.device)
        check(_lib.load().moe_distill_backward(self._c(n), xp, wp, ip, tp, lp, gp, dX.data_ptr(),
                                               dW.data_ptr(), _args.TYPES[dW_dtype], self.ws.data_ptr(),
                                               self.ws.numel(), on.handle), "moe_distill_backward")
        on.uses(X, W, ids, teacher, lse, dloss, self.ws)
        return dX, dW

    def check(self, stream=None) -> None:
        """Raises if a call since the last check met a class outside the vocabulary, or a wait ran out."""
        from .api import check_status
        check(check_status(self.ws, stream), "device status")

"""Python binding of routing to experts from given logits (include/moe_scores.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _args, _lib
from ._lib import ScoresConfig as _C
from ._lib import check

__all__ = ["ScoreRouterConfig", "ScoreRouter"]

_SCORES = {"softmax": 0, "sigmoid": 1}


@dataclasses.dataclass(frozen=True)
class ScoreRouterConfig:
    N: int                   # tokens (the most a call may have)
    E: int                   # experts, up to 1024
    k: int                   # experts a token
    groups: int = 1          # equal runs of experts
    topk_groups: int = 1     # groups open to a token
    score: str = "softmax"   # or "sigmoid"
    renormalize: bool = True
    scale: float = 1.0
    group_top: int = 2       # how many of a group's values make its score: 1 or 2

    def c_struct(self, n=None):
        if self.score not in _SCORES:
            raise ValueError(f"score: expected one of {sorted(_SCORES)}, got {self.score!r}")
        return _C(self.N if n is None else n, self.E, self.k, self.groups, self.topk_groups, self.group_top,
                  _SCORES[self.score], int(self.renormalize), self.scale)


class ScoreRouter:
    """Chooses the experts of up to N tokens and weighs them; its outputs are MoEBlock.forward's idx and gates."""

    def __init__(self, cfg: ScoreRouterConfig, device="cuda"):
        self.cfg = cfg
        self._c = _args.Structs(cfg)
        b = ctypes.c_size_t()
        check(_lib.load().moe_scores_workspace_bytes(ctypes.byref(cfg.c_struct()), ctypes.byref(b)),
              "moe_scores_workspace_bytes")
        self.ws = _args.workspace(b.value, device)

    def forward(self, logits, bias=None, stream=None):
        """logits [n <= N, E] (rows may be strided); bias [E] fp32 or None, for the choice only -> idx [n, k] int32,
        weights [n, k] fp32, counts [E] int32 (tokens of each expert)."""
        c = self.cfg
        n = _args.count(logits, "logits", c.N)
        lp, ld = _args.rows(logits, "logits", _args.TYPES, (n, c.E))
        bp = _args.ptr(bias, "bias", torch.float32, (c.E,))
        dev = logits.device
        on = _args.On(stream, dev)
        idx = on.empty((n, c.k), torch.int32, dev)
        w = on.empty((n, c.k), torch.float32, dev)
        counts = on.empty((c.E,), torch.int32, dev)
        check(_lib.load().moe_scores_forward(self._c(n), lp, ld, _args.TYPES[logits.dtype], bp,
                                             idx.data_ptr(), w.data_ptr(), counts.data_ptr(), self.ws.data_ptr(),
                                             self.ws.numel(), on.handle), "moe_scores_forward")
        on.uses(logits, bias, self.ws)
        return idx, w, counts

    def backward(self, logits, idx, dweights, stream=None):
        """idx from the forward; dweights [n, k] fp32 -> the logits' gradient [n, E], in their type."""
        c = self.cfg
        n = _args.count(logits, "logits", c.N)
        lp, ld = _args.rows(logits, "logits", _args.TYPES, (n, c.E))
        ip = _args.ptr(idx, "idx", torch.int32, (n, c.k))
        gp = _args.ptr(dweights, "dweights", torch.float32, (n, c.k))
        on = _args.On(stream, logits.device)
        d = on.empty((n, c.E), logits.dtype, logits.device)
        check(_lib.load().moe_scores_backward(self._c(n), lp, ld, _args.TYPES[logits.dtype], ip, gp,
                                              d.data_ptr(), self.ws.data_ptr(), self.ws.numel(), on.handle),
              "moe_scores_backward")
        on.uses(logits, idx, dweights, self.ws)
        return d

    def check(self, stream=None) -> None:
        """Raises if a backward since the last check met an expert outside [0, E)."""
        from .api import check_status
        check(check_status(self.ws, stream), "device status")

"""Python binding of token embedding and its gradient (include/moe_embed.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _args, _lib
from ._lib import EmbedConfig as _C
from ._lib import check

__all__ = ["EmbeddingConfig", "TokenEmbedding", "embed_workspace_bytes"]


@dataclasses.dataclass(frozen=True)
class EmbeddingConfig:
    N: int               # tokens (the most a call may have)
    V: int               # table rows
    H: int               # row width
    scale: float = 1.0
    padding_idx: int = -1    # id whose row gets no gradient; -1: none

    def c_struct(self, n=None):
        return _C(self.N if n is None else n, self.V, self.H, self.padding_idx, self.scale)


def embed_workspace_bytes(cfg: EmbeddingConfig) -> tuple[int, int]:
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    check(_lib.load().moe_embed_workspace_bytes(ctypes.byref(cfg.c_struct()), ctypes.byref(f), ctypes.byref(b)),
          "moe_embed_workspace_bytes")
    return f.value, b.value


class TokenEmbedding:
    """Owns the workspace for up to N tokens; calls on one object run on one stream at a time."""

    def __init__(self, cfg: EmbeddingConfig, device="cuda"):
        self.cfg = cfg
        self._c = _args.Structs(cfg)
        self.ws = _args.workspace(max(embed_workspace_bytes(cfg)), device)

    def forward(self, ids, table, stream=None):
        """ids [n <= N] int32 or int64; table [V, H] -> scale * table[ids] [n, H], in the table's type."""
        c = self.cfg
        n = _args.count(ids, "ids", c.N)
        ip = _args.ptr(ids, "ids", _args.INDEX_TYPES, (n,))
        tp = _args.ptr(table, "table", _args.TYPES, (c.V, c.H))
        on = _args.On(stream, table.device)
        y = on.empty((n, c.H), table.dtype, table.device)
        check(_lib.load().moe_embed_forward(self._c(n), ip, _args.INDEX_TYPES[ids.dtype], tp,
                                            y.data_ptr(), _args.TYPES[table.dtype], self.ws.data_ptr(),
                                            self.ws.numel(), on.handle), "moe_embed_forward")
        on.uses(ids, table, self.ws)
        return y

    def backward(self, ids, dy, into=None, stream=None):
        """dy [n, H] (rows may be strided) -> the table's gradient [V, H] fp32; `into`: a gradient so far, which is
        added to (only the rows of tokens that occur are touched) and returned."""
        c = self.cfg
        n = _args.count(ids, "ids", c.N)
        ip = _args.ptr(ids, "ids", _args.INDEX_TYPES, (n,))
        gp, ldg = _args.rows(dy, "dy", _args.TYPES, (n, c.H))
        on = _args.On(stream, dy.device)
        dW = on.empty((c.V, c.H), torch.float32, dy.device) if into is None else into
        wp = _args.ptr(dW, "into", torch.float32, (c.V, c.H))
        check(_lib.load().moe_embed_backward(self._c(n), ip, _args.INDEX_TYPES[ids.dtype], gp, ldg,
                                             _args.TYPES[dy.dtype], wp, 0 if into is None else 1, self.ws.data_ptr(),
                                             self.ws.numel(), on.handle), "moe_embed_backward")
        on.uses(ids, dy, into, self.ws)
        return dW

    def check(self, stream=None) -> None:
        """Raises if a call since the last check met an id outside [0, V)."""
        from .api import check_status
        check(check_status(self.ws, stream), "device status")

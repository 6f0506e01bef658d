"""Python binding of matrices in 8 bits with a scale for each block of 128 (include/moe_blocks8.h), for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import dataclasses

import torch

from . import _args, _lib
from ._lib import check

__all__ = ["Checkpoint8Config", "Checkpoint8", "pack_weight8", "BLOCK8"]

BLOCK8 = 128
CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu


def blocks(n: int) -> int:
    return -(-n // BLOCK8)


@dataclasses.dataclass(frozen=True)
class Checkpoint8Config:
    N: int               # rows (the most a call may have)
    H: int               # row width, up to 2^20


class Checkpoint8:
    """Activations kept in 8 bits: e4m3 codes, and a power-of-two scale for each 128 columns of a row.  It holds no
    workspace: calls may run on any streams at once."""

    def __init__(self, cfg: Checkpoint8Config, device="cuda"):
        if cfg.N < 0 or not 1 <= cfg.H <= 1 << 20:
            raise ValueError("N or H out of range")
        self.cfg = cfg

    def pack(self, x, stream=None):
        """x [n <= N, H] bf16, fp16 or fp32 (rows may be strided) -> codes [n, H] float8_e4m3fn, scales
        [n, ceil(H / 128)] float8_e8m0fnu."""
        c = self.cfg
        n = _args.count(x, "x", c.N)
        xp, ldx = _args.rows(x, "x", _args.TYPES, (n, c.H))
        _args.here(x.device)
        on = _args.On(stream, x.device)
        codes = on.empty((n, c.H), CODES, x.device)
        scales = on.empty((n, blocks(c.H)), SCALES, x.device)
        check(_lib.load().moe_blocks8_pack(xp, ldx, _args.TYPES[x.dtype], n, c.H, codes.data_ptr(), scales.data_ptr(),
                                           on.handle), "moe_blocks8_pack")
        on.uses(x)
        return codes, scales

    def unpack(self, codes, scales, dtype=torch.bfloat16, stream=None):
        """The values [n, H] that the codes stand for; exact in bfloat16 and float32."""
        c = self.cfg
        n = _args.count(codes, "codes", c.N)
        cp = _args.ptr(codes, "codes", CODES, (n, c.H))
        sp = _args.ptr(scales, "scales", SCALES, (n, blocks(c.H)))
        if dtype not in _args.TYPES:
            raise TypeError("dtype: expected float32, bfloat16 or float16")
        _args.here(codes.device, scales)
        on = _args.On(stream, codes.device)
        y = on.empty((n, c.H), dtype, codes.device)
        check(_lib.load().moe_blocks8_unpack(cp, sp, n, c.H, y.data_ptr(), _args.TYPES[dtype], on.handle),
              "moe_blocks8_unpack")
        on.uses(codes, scales)
        return y


def pack_weight8(w, stream=None):
    """Weights [E, O, K] in bf16, fp16 or fp32 -> codes [E, O, K] float8_e4m3fn, scales [E, ceil(O / 128),
    ceil(K / 128)] float8_e8m0fnu: one for each 128 x 128 values, as ExpertLinear takes them."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise TypeError("w: expected a torch.Tensor of three dimensions")
    E, O, K = w.shape
    if max(E, O, K) >= 2 ** 31:
        raise ValueError(f"w: shape {tuple(w.shape)} is out of range")
    wp = _args.ptr(w, "w", _args.TYPES, (E, O, K))
    _args.here(w.device)
    on = _args.On(stream, w.device)
    codes = on.empty((E, O, K), CODES, w.device)
    scales = on.empty((E, blocks(O), blocks(K)), SCALES, w.device)
    check(_lib.load().moe_blocks8_pack_weight(wp, _args.TYPES[w.dtype], E, O, K, codes.data_ptr(), scales.data_ptr(),
                                              on.handle), "moe_blocks8_pack_weight")
    on.uses(w)
    return codes, scales

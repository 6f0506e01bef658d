"""Argument marshalling shared by the layer operators' bindings (norm.py, embed.py, scores.py, distill.py, rmsnorm.py,
blocks8.py, linear.py)."""
from __future__ import annotations

import ctypes

import torch

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}      # MOE_TYPE_* of moe_types.h
_raw_stream = torch._C._cuda_getCurrentRawStream   # current_stream(device).cuda_stream without the Stream object
INDEX_TYPES = {torch.int32: 0, torch.int64: 1}                       # MOE_INDEX_*


def _is(dtype, wanted) -> bool:
    return dtype in wanted if type(wanted) is dict else dtype is wanted


def ptr(t, name: str, dtype, shape) -> int | None:
    """Device pointer of a dense CUDA tensor of `shape` and of type `dtype` (or one of a dict's); None stays None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not _is(t.dtype, dtype):
        raise TypeError(f"{name}: unexpected type {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def rows(t, name: str, dtype, shape) -> tuple[int, int]:
    """(device pointer, row stride) of a CUDA matrix whose rows are dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not _is(t.dtype, dtype):
        raise TypeError(f"{name}: unexpected type {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    n, h = shape
    if t.is_contiguous():
        return t.data_ptr(), h
    s = t.stride()
    if (h > 1 and s[1] != 1) or (n > 1 and s[0] < h):
        raise ValueError(f"{name}: expected rows of consecutive elements, at least a row apart")
    return t.data_ptr(), s[0] if n > 1 else h


def count(t, name: str, most: int) -> int:
    """Rows of this call: at most the `most` its unit was made for."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise TypeError(f"{name}: expected a torch.Tensor with rows")
    n = t.shape[0]
    if n > most:
        raise ValueError(f"{name}: {n} rows, made for at most {most}")
    return n


def here(device, *tensors):
    """The tensors of a call lie on the unit's device, and that is the current one: the library launches there."""
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"expected tensors on {device}, got one on {t.device}")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"expected {device} to be the current device")


class On:
    """The stream a call's kernels run on.  Where it is not the current one, the outputs made inside `with` belong
    to it, and the tensors named to `uses` are kept from reuse until its work so far is done."""

    __slots__ = ("stream", "handle")

    def __init__(self, stream, device):
        if stream is None:
            self.stream = None
            self.handle = _raw_stream(device.index)
        else:
            self.stream = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))
            self.handle = self.stream.cuda_stream

    def empty(self, shape, dtype, device):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=device)

    def uses(self, *tensors):
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)


def workspace(nbytes: int, device) -> torch.Tensor:
    """Zeroed, so that the status word starts clear."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class Structs:
    """A unit's C configuration by the number of rows of a call, as the pointer that the library takes."""

    def __init__(self, cfg):
        self._cfg, self._made = cfg, {}

    def __call__(self, n: int):
        got = self._made.get(n)
        if got is None:
            if len(self._made) >= 64:
                self._made.clear()
            got = self._made[n] = ctypes.pointer(self._cfg.c_struct(n))
        return got

"""Checks of tensor arguments shared by the tensor-level functions of the 8-bit linear and
the attention entry points, and the call on the tensors' own device."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from ._binding import _check, load_library

_SAME = contextlib.nullcontext()


def expect(t: torch.Tensor, what: str, dtypes, shape) -> torch.Size:
    """The shape of `t`, a contiguous tensor of one of `dtypes` and of `shape` (None entries
    are free)."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_contiguous():
        got = t.shape
        if got == shape:
            return got
        if len(got) == len(shape):
            for n, w in zip(got, shape):
                if w is not None and w != n:
                    break
            else:
                return got
    _refuse(t, what, dtypes, shape)


def _refuse(t, what, dtypes, shape):
    """The error of a tensor that `expect` does not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a tensor, got %s" % (what, type(t).__name__))
    if t.dtype not in dtypes:
        raise TypeError("%s: expected %s, got %s" % (what, " or ".join(map(str, dtypes)), t.dtype))
    if len(t.shape) != len(shape) or any(w is not None and w != n for n, w in zip(t.shape, shape)):
        raise ValueError("%s: expected shape %s, got %s"
                         % (what, tuple("*" if w is None else w for w in shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % what)


def expect_rows(t: torch.Tensor, what: str, dtypes, shape):
    """(shape, elements from one row to the next) of `t`, a tensor of one of `dtypes` and of
    `shape` (None entries are free) whose rows are contiguous but may lie apart (a part of a
    projection's columns)."""
    if isinstance(t, torch.Tensor) and t.dim() == 3 and not t.is_contiguous():
        _, n, m = t.shape
        s = t.stride()
        if (m <= 1 or s[2] == 1) and (n <= 1 or s[1] == m) and s[0] >= n * m:
            rows, n_want, m_want = shape
            if (t.dtype not in dtypes or rows not in (None, t.shape[0]) or n_want not in (None, n)
                    or m_want not in (None, m)):
                _refuse(t, what, dtypes, shape)
            return t.shape, s[0]
    got = expect(t, what, dtypes, shape)
    return got, got[1] * got[2]


BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # bf16 or its bit patterns
F32 = (torch.float32,)
I8 = (torch.int8,)
U8 = (torch.uint8,)
I32 = (torch.int32,)


def one_device(**tensors: Optional[torch.Tensor]) -> torch.device:
    """The GPU that holds every given tensor (None entries are passed over)."""
    first, index = None, -1
    for what, t in tensors.items():
        if t is None:
            continue
        i = t.get_device()
        if i < 0:
            raise ValueError("%s must be on a GPU, is on %s" % (what, t.device))
        if first is None:
            first, index = t, i
        elif i != index:
            raise ValueError("%s is on %s, the other tensors on %s" % (what, t.device, first.device))
    return first.device


def on(dev: torch.device):
    """Context in which `dev` is the current device (the library launches on the current one)."""
    return _SAME if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def at(t: Optional[torch.Tensor]):
    """The address of a tensor that `expect` has seen, or None."""
    return None if t is None else t.data_ptr()


def ptr(t: Optional[torch.Tensor]):
    """The address of a tensor, which has to be contiguous, or None."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libsvdq must be contiguous")
    return t.data_ptr()


# The current stream's handle alone; torch.cuda.current_stream makes an object of it, which
# takes as long as half a launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_ptr(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if not torch.cuda.is_initialized() and not torch.cuda.is_available():
        return None
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def stream_of(dev: torch.device):
    """The handle of the current stream of `dev`."""
    if _raw_stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(dev.index)


def scratch(workspace: Optional[torch.Tensor], need: int, dev: torch.device):
    """`workspace` if it holds `need` bytes on `dev`, otherwise a new one (None when need == 0)."""
    if need == 0:
        return None
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % (dev,))
        if workspace.numel() * workspace.element_size() >= need:
            return workspace
    return torch.empty(need, dtype=torch.uint8, device=dev)


class Entries:
    """The entry points of one header: argument types are set on first use."""

    def __init__(self, signatures: dict):
        self._signatures = signatures
        self._fns = None

    def names(self):
        return tuple(self._signatures)

    def __getitem__(self, name):
        if self._fns is None:
            lib, fns = load_library(), {}
            for n, (args, res) in self._signatures.items():
                fns[n] = getattr(lib, n)
                fns[n].argtypes, fns[n].restype = args, res
            self._fns = fns
        return self._fns[name]

    def call(self, name, *args):
        _check(self[name](*args), name)


P, I64, I32T, SZ, F32T = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                          ctypes.c_float)

"""Operators of causal sequence layers: argument marshalling for the ``bilstm_causal_conv``,
``bilstm_scan``, ``bilstm_add_rms_norm`` and ``bilstm_token_logprobs`` entry points of bilstm.h,
which gives the formulas and the conventions of packed sequences and state caches.

Tensors are CUDA (HIP) tensors of one device; float32, bfloat16 and float16 are taken unless a
tensor is said to be of another type. Rows may have a stride; what lies within a row must be
contiguous. Work is enqueued on ``stream`` (the device's current stream if None), and outputs and
scratch memory that a call allocates belong to that stream. Serving only: a tensor that requires a
gradient is refused while gradients are enabled.
"""

from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import NamedTuple

_VIEW = "3Q"
_BUFFER = "2Q"
_CONV = struct.Struct("<iiQIIIIii" + _VIEW + _BUFFER * 6 + _VIEW)

NO_BUFFER = (0, 0)
NO_ROWS = (0, 0, 0)


def signatures() -> dict:
    P = ctypes.c_void_p
    args = [ctypes.c_char_p, P]
    return {name: (args, ctypes.c_int) for name in ("bilstm_causal_conv", "bilstm_causal_conv_step")}


def _kinds():
    import torch
    return {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


_TYPES: dict = {}


def _type_of(t, name: str) -> int:
    if not _TYPES:
        _TYPES.update(_kinds())
    kind = _TYPES.get(getattr(t, "dtype", None))
    if kind is None:
        raise TypeError(f"{name} must be a float32, bfloat16 or float16 tensor")
    return kind


class _Call:
    """What the tensors of one call have in common: the device, and the element type of most."""

    __slots__ = ("device", "dtype", "kind", "grad", "stream")

    def __init__(self, first, name: str, stream):
        import torch
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        self.kind = _type_of(first, name)
        self.dtype = first.dtype
        self.device = first.get_device()
        self.grad = torch.is_grad_enabled()
        if stream is not None and stream.device_index != self.device:
            raise ValueError(f"stream belongs to device {stream.device_index}, {name} to device {self.device}")
        self.stream = stream

    def _check(self, t, name: str, dtype, shape) -> None:
        import torch
        if not isinstance(t, torch.Tensor) or t.get_device() != self.device:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor on device {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be a {dtype} tensor, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if self.grad and t.requires_grad:
            raise TypeError(f"{name} requires a gradient; these operators have none (use torch.no_grad())")

    def rows(self, t, name: str, shape: tuple, dtype=None) -> tuple:
        """(pointer, elements, row stride) of a tensor of rows: [rows, width] or [rows, parts, width]."""
        self._check(t, name, self.dtype if dtype is None else dtype, shape)
        strides = t.stride()
        width = shape[-1]
        if (width > 1 and strides[-1] != 1) or (len(shape) == 3 and shape[1] > 1 and strides[1] != width):
            raise ValueError(f"{name} must be contiguous within a row, got strides {strides}")
        if len(shape) == 3:
            width *= shape[1]
        count = shape[0]
        if count == 0 or width == 0:
            return NO_ROWS
        stride = strides[0] if count > 1 else width
        return t.data_ptr(), (count - 1) * stride + width, stride

    def buffer(self, t, name: str, shape: tuple, dtype=None) -> tuple:
        """(pointer, elements) of a contiguous tensor; None is no buffer."""
        if t is None:
            return NO_BUFFER
        self._check(t, name, self.dtype if dtype is None else dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous, got strides {t.stride()}")
        return t.data_ptr(), t.numel()

    def empty(self, shape, dtype=None):
        """A new tensor that belongs to the call's stream."""
        import torch
        with contextlib.nullcontext() if self.stream is None else torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=self.dtype if dtype is None else dtype, device=f"cuda:{self.device}")

    def run(self, name: str, packed: bytes) -> None:
        import torch
        from . import _check, library
        stream = self.stream if self.stream is not None else torch.cuda.current_stream(self.device)
        _check(getattr(library(), name)(packed, stream.cuda_stream))


def _dims(t, name: str, count: int) -> tuple:
    shape = getattr(t, "shape", None)
    if shape is None or len(shape) != count:
        raise ValueError(f"{name} must have {count} dimensions, got {None if shape is None else len(shape)}")
    return tuple(shape)


def _sequences(call: _Call, seq_starts, state, slots, fresh) -> tuple:
    """(sequences, starts, slots, fresh) of a packed batch, the last three as buffers."""
    import torch
    count = _dims(seq_starts, "seq_starts", 1)[0] - 1
    if count < 0:
        raise ValueError("seq_starts must hold one row number more than there are sequences")
    if state is None and (slots is not None or fresh is not None):
        raise ValueError("slots and fresh need a state")
    if fresh is not None and fresh.dtype == torch.bool:
        fresh = fresh.view(torch.uint8)
    return (count, call.buffer(seq_starts, "seq_starts", (count + 1,), torch.int32),
            call.buffer(slots, "slots", (count,), torch.int32), call.buffer(fresh, "fresh", (count,), torch.uint8))


def causal_conv(x, weight, seq_starts, bias=None, state=None, slots=None, fresh=None, silu: bool = True, out=None,
                stream=None):
    """Short causal convolution per channel over packed sequences; returns y like ``x``.

    ``x`` [rows, channels]; ``weight`` [channels, taps] with 2, 3 or 4 taps, the last one for the
    current row; ``seq_starts`` int32 [sequences + 1]: sequence j is rows seq_starts[j] ..
    seq_starts[j + 1] - 1; ``state`` [places, taps - 1, channels] holds the rows before each
    sequence and is updated in place; ``slots`` int32 [sequences] names each sequence's place (j if
    None, one outside the cache skips the sequence); ``fresh`` bool [sequences]: start from zeros.
    Rows of no sequence are not written: pass ``out`` to keep what they hold.
    """
    call = _Call(x, "x", stream)
    rows, channels = _dims(x, "x", 2)
    taps = _dims(weight, "weight", 2)[1]
    count, starts, places, begin = _sequences(call, seq_starts, state, slots, fresh)
    cache = _dims(state, "state", 3)[0] if state is not None else 0
    if out is None:
        out = call.empty((rows, channels))
    xv, yv = call.rows(x, "x", (rows, channels)), call.rows(out, "out", (rows, channels))
    call.run("bilstm_causal_conv", _CONV.pack(
        call.device, call.kind, rows, channels, taps, count, cache, 1 if silu else 0, 0, *xv,
        *call.buffer(weight, "weight", (channels, taps)), *call.buffer(bias, "bias", (channels,)), *starts,
        *call.buffer(state, "state", (cache, taps - 1, channels)), *places, *begin, *yv))
    return out


def causal_conv_step(x, weight, state, bias=None, slots=None, silu: bool = True, out=None, stream=None):
    """One new row per sequence of ``causal_conv``: row i of ``x`` [rows, channels] continues the
    sequence at place ``slots[i]`` (i if None) of ``state``, which is updated in place."""
    import torch
    call = _Call(x, "x", stream)
    rows, channels = _dims(x, "x", 2)
    taps = _dims(weight, "weight", 2)[1]
    cache = _dims(state, "state", 3)[0]
    if out is None:
        out = call.empty((rows, channels))
    xv, yv = call.rows(x, "x", (rows, channels)), call.rows(out, "out", (rows, channels))
    call.run("bilstm_causal_conv_step", _CONV.pack(
        call.device, call.kind, rows, channels, taps, 0, cache, 1 if silu else 0, 0, *xv,
        *call.buffer(weight, "weight", (channels, taps)), *call.buffer(bias, "bias", (channels,)), *NO_BUFFER,
        *call.buffer(state, "state", (cache, taps - 1, channels)), *call.buffer(slots, "slots", (rows,), torch.int32),
        *NO_BUFFER, *yv))
    return out

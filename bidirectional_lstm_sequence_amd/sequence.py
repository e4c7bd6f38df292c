"""Operators of causal sequence layers: argument marshalling for the ``bilstm_causal_conv``,
``bilstm_scan``, ``bilstm_add_rms_norm`` and ``bilstm_token_logprobs`` entry points of bilstm.h,
which gives the formulas and the conventions of packed sequences and state caches.

Tensors are CUDA (HIP) tensors of one device; float32, bfloat16 and float16 are taken unless a
tensor is said to be of another type. Rows may have a stride; what lies within a row must be
contiguous. Work is enqueued on ``stream`` (the device's current stream if None), and outputs and
scratch memory that a call allocates belong to that stream. Serving only: a tensor that requires a
gradient is refused while gradients are enabled, one with a forward-mode tangent always.
"""

from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple

_VIEW = "3Q"
_BUFFER = "2Q"
_CONV = struct.Struct("<iiQIIIIii" + _VIEW + _BUFFER * 6 + _VIEW)

_SCAN = struct.Struct("<iiQIIIIIIii" + _VIEW * 5 + _BUFFER * 7 + _VIEW + _BUFFER)
_NORM = struct.Struct("<iiQIifi" + _VIEW * 2 + _BUFFER + _VIEW * 3 + _BUFFER)
_LOGPROBS = struct.Struct("<iiQIIIi" + _VIEW + _BUFFER * 6)

_nothing = (ctypes.c_float * 8)()
_NO_PLACES = (ctypes.addressof(_nothing) + 15) // 16 * 16

NO_BUFFER = (0, 0)
NO_ROWS = (0, 0, 0)


def signatures() -> dict:
    P = ctypes.c_void_p
    args = [ctypes.c_char_p, P]
    sizes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_uint64)]
    sig = {name: (args, ctypes.c_int) for name in ("bilstm_causal_conv", "bilstm_causal_conv_step", "bilstm_scan",
                                                   "bilstm_scan_step", "bilstm_add_rms_norm", "bilstm_token_logprobs")}
    for name in ("bilstm_scan_scratch", "bilstm_token_logprobs_scratch"):
        sig[name] = (sizes, ctypes.c_int)
    return sig


class _Torch:
    """What the calls need of torch and the library, looked up at the first call."""

    def __init__(self):
        import torch
        from . import _check, library
        self.Tensor, self.empty = torch.Tensor, torch.empty
        self.kinds = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        self.float32, self.int32, self.int64 = torch.float32, torch.int32, torch.int64
        self.uint8, self.bool = torch.uint8, torch.bool
        self.eight = {None: (0, None), "e4m3": (1, torch.float8_e4m3fn), "int8": (2, torch.int8)}
        self.grad = torch.is_grad_enabled
        self.forward = torch.autograd.forward_ad
        self.on_stream = torch.cuda.stream
        # the handle alone, without a Stream object around it
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        self.check, self.library = _check, library()


_torch = None


def _get_torch() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


class _Call:
    """What the tensors of one call have in common: the device, and the element type of most."""

    __slots__ = ("torch", "like", "device", "dtype", "kind", "grad", "dual", "stream")

    def __init__(self, first, name: str, stream):
        self.torch = t = _torch or _get_torch()
        if not isinstance(first, t.Tensor) or not first.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        self.like = first
        self.dtype = first.dtype
        self.kind = t.kinds.get(self.dtype)
        if self.kind is None:
            raise TypeError(f"{name} must be a float32, bfloat16 or float16 tensor, got {self.dtype}")
        self.device = first.get_device()
        self.grad = t.grad()
        # outside of every level no tensor has a tangent
        self.dual = getattr(t.forward, "_current_level", 0) >= 0
        if stream is not None and stream.device_index != self.device:
            raise ValueError(f"stream belongs to device {stream.device_index}, {name} to device {self.device}")
        self.stream = stream

    def _check(self, t, name: str, dtype, shape) -> None:
        try:
            if (t.get_device() == self.device and t.dtype == dtype and t.shape == shape
                    and not (self.grad and t.requires_grad) and not self.dual):
                return
        except AttributeError:
            pass
        if not isinstance(t, self.torch.Tensor) or t.get_device() != self.device:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor on device {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be a {dtype} tensor, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if self.dual and self.torch.forward.unpack_dual(t).tangent is not None:
            raise TypeError(f"{name} has a forward-mode tangent; these operators have no derivatives")
        if self.grad and t.requires_grad:
            raise TypeError(f"{name} requires a gradient; these operators have none (use torch.no_grad())")

    def rows(self, t, name: str, shape: tuple, dtype=None) -> tuple:
        """(pointer, elements, row stride) of a tensor of rows: [rows, width] or [rows, parts, width]."""
        self._check(t, name, dtype or self.dtype, shape)
        count, width = shape[0], shape[-1]
        if t.is_contiguous():
            if len(shape) == 3:
                width *= shape[1]
            return (t.data_ptr(), count * width, width) if count and width else NO_ROWS
        strides = t.stride()
        if (width > 1 and strides[-1] != 1) or (len(shape) == 3 and shape[1] > 1 and strides[1] != width):
            raise ValueError(f"{name} must be contiguous within a row, got strides {strides}")
        if len(shape) == 3:
            width *= shape[1]
        stride = strides[0] if count > 1 else width
        return t.data_ptr(), (count - 1) * stride + width, stride

    def buffer(self, t, name: str, shape: tuple, dtype=None) -> tuple:
        """(pointer, elements) of a contiguous tensor; None is no buffer."""
        if t is None:
            return NO_BUFFER
        self._check(t, name, dtype or self.dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous, got strides {t.stride()}")
        return t.data_ptr(), t.numel()

    def cache(self, t, shape: tuple, dtype=None) -> tuple:
        """``buffer`` of a state. One of no places or elements, which has no memory, is still not the lack of one:
        the library, which tells them apart by the pointer, gets the address of a float that it never reads."""
        pointer, count = self.buffer(t, "state", shape, dtype)
        return (pointer, count) if pointer or t is None else (_NO_PLACES, count)

    def empty(self, shape, dtype=None):
        """A new tensor that belongs to the call's stream."""
        if self.stream is None:
            return self.like.new_empty(shape, dtype=dtype)
        with self.torch.on_stream(self.stream):
            return self.like.new_empty(shape, dtype=dtype)

    def scratch(self, bytes_needed: int):
        """(tensor, buffer) of the call's scratch memory."""
        if bytes_needed == 0:
            return None, NO_BUFFER
        t = self.empty((bytes_needed,), self.torch.uint8)
        return t, (t.data_ptr(), bytes_needed)

    def run(self, name: str, packed: bytes) -> None:
        t = self.torch
        stream = t.stream(self.device) if self.stream is None else self.stream.cuda_stream
        status = getattr(t.library, name)(packed, stream)
        if status != 0:
            t.check(status)


@functools.lru_cache(maxsize=256)
def _scratch_bytes(name: str, packed: bytes) -> int:
    """Bytes of scratch memory by the library's own count: a function of the sizes in ``packed``."""
    t = _get_torch()
    need = ctypes.c_uint64()
    t.check(getattr(t.library, name)(packed, ctypes.byref(need)))
    return need.value


def _dims(t, name: str, count: int) -> tuple:
    shape = getattr(t, "shape", None)
    if shape is None or len(shape) != count:
        raise ValueError(f"{name} must have {count} dimensions, got {None if shape is None else len(shape)}")
    return tuple(shape)


def _sequences(call: _Call, seq_starts, state, slots, fresh) -> tuple:
    """(sequences, starts, slots, fresh) of a packed batch, the last three as buffers."""
    torch = call.torch
    count = _dims(seq_starts, "seq_starts", 1)[0] - 1
    if count < 0:
        raise ValueError("seq_starts must hold one row number more than there are sequences")
    if state is None and (slots is not None or fresh is not None):
        raise ValueError("slots and fresh need a state")
    flag = torch.bool if getattr(fresh, "dtype", None) == torch.bool else torch.uint8
    return (count, call.buffer(seq_starts, "seq_starts", (count + 1,), torch.int32),
            call.buffer(slots, "slots", (count,), torch.int32), call.buffer(fresh, "fresh", (count,), flag))


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
        *call.cache(state, (cache, taps - 1, channels)), *places, *begin, *yv))
    return out


def causal_conv_step(x, weight, state, bias=None, slots=None, silu: bool = True, out=None, stream=None):
    """One new row per sequence of ``causal_conv``: row i of ``x`` [rows, channels] continues the
    sequence at place ``slots[i]`` (i if None) of ``state``, which is updated in place."""
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
        *call.cache(state, (cache, taps - 1, channels)), *call.buffer(slots, "slots", (rows,), call.torch.int32),
        *NO_BUFFER, *yv))
    return out


def _scan(name: str, x, dt, a, b, c, seq_starts, d, z, dt_bias, softplus, state, slots, fresh, out, stream):
    call = _Call(x, "x", stream)
    torch = call.torch
    rows, heads, width = shape = _dims(x, "x", 3)
    _, groups, states = _dims(b, "b", 3)
    if seq_starts is None:
        count, starts, begin = 0, NO_BUFFER, NO_BUFFER
        places = call.buffer(slots, "slots", (rows,), torch.int32)
    else:
        count, starts, places, begin = _sequences(call, seq_starts, state, slots, fresh)
    cache = _dims(state, "state", 4)[0] if state is not None else 0
    if out is None:
        out = call.empty(shape)
    sizes = (call.device, call.kind, rows, heads, width, groups, states, count)
    head = (*sizes, cache, 1 if softplus else 0, 0, *call.rows(x, "x", shape), *call.rows(dt, "dt", (rows, heads)),
            *call.rows(b, "b", (rows, groups, states)), *call.rows(c, "c", (rows, groups, states)), *(NO_ROWS if z is None else call.rows(z, "z", shape)),
            *call.buffer(a, "a", (heads,), torch.float32), *call.buffer(d, "d", (heads,), torch.float32),
            *call.buffer(dt_bias, "dt_bias", (heads,), torch.float32), *starts,
            *call.cache(state, (cache, heads, width, states), torch.float32), *places, *begin,
            *call.rows(out, "out", shape))
    hold, scratch = None, NO_BUFFER
    if seq_starts is not None:
        hold, scratch = call.scratch(_scratch_bytes("bilstm_scan_scratch", _SCAN.pack(*sizes, *(0,) * 37)))
    call.run(name, _SCAN.pack(*head, *scratch))
    del hold  # its memory goes back to the call's stream, behind the call's work
    return out


def selective_scan(x, dt, a, b, c, seq_starts, d=None, z=None, dt_bias=None, softplus: bool = True, state=None, slots=None,
                   fresh=None, out=None, stream=None):
    """Selective state space scan over packed sequences; returns y like ``x``.

    ``x`` and the optional gate ``z`` [rows, heads, width] (width 32, 64 or 128); ``dt`` [rows, heads];
    ``b`` and ``c`` [rows, groups, states] (16, 32, 64, 128 or 256 states; head h belongs to group
    h * groups // heads); ``a``, ``d`` (optional) and ``dt_bias`` (optional) float32 [heads]; with
    ``softplus`` the step is log(1 + exp(dt + dt_bias)). ``seq_starts``, ``slots`` and ``fresh`` as in
    ``causal_conv``; ``state`` float32 [places, heads, width, states] holds each sequence's state and is
    updated in place. Rows of no sequence are not written: pass ``out`` to keep what they hold.
    """
    return _scan("bilstm_scan", x, dt, a, b, c, seq_starts, d, z, dt_bias, softplus, state, slots, fresh, out, stream)


def selective_scan_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, softplus: bool = True, slots=None, out=None,
                        stream=None):
    """One new row per sequence of ``selective_scan``: row i continues the state at place ``slots[i]``
    (i if None) of ``state``, which is updated in place."""
    return _scan("bilstm_scan_step", x, dt, a, b, c, None, d, z, dt_bias, softplus, state, slots, None, out, stream)


class NormResult(NamedTuple):
    """``add_rms_norm``'s outputs; what was not asked for is None."""

    y: object
    q: object
    scales: object
    residual: object


def add_rms_norm(x, weight, eps: float = 1e-5, residual=None, eight_bit=None, keep_y=None, out=None, residual_out=None,
                 q=None, scales=None, stream=None) -> NormResult:
    """Root-mean-square norm of the rows of ``x`` [rows, width] (with ``residual`` added first) times
    ``weight`` [width].

    Returns ``NormResult(y, q, scales, residual)``: ``residual`` is x + residual (None without one);
    ``eight_bit`` "e4m3" or "int8" gives the rows in 8 bits, ``q``, and their ``scales`` [rows] float32
    with y close to q * scales[:, None]; ``y`` itself comes with them if ``keep_y`` is true, without
    ``eight_bit`` always. ``out`` and ``residual_out`` may be ``x`` or ``residual`` themselves.
    """
    call = _Call(x, "x", stream)
    torch = call.torch
    shape = _dims(x, "x", 2)
    if eight_bit not in torch.eight:
        raise ValueError(f"eight_bit must be None, 'e4m3' or 'int8', got {eight_bit!r}")
    kind, code = torch.eight[eight_bit]
    if kind == 0 and (q is not None or scales is not None or keep_y is False):
        raise ValueError("without eight_bit the norm gives y only")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is None and (kind == 0 or keep_y):
        out = call.empty(shape)
    if residual is not None and residual_out is None:
        residual_out = call.empty(shape)
    if kind:
        q = call.empty(shape, code) if q is None else q
        scales = call.empty(shape[:1], torch.float32) if scales is None else scales
    rows = lambda t, name, dtype=None: NO_ROWS if t is None else call.rows(t, name, shape, dtype)  # noqa: E731
    call.run("bilstm_add_rms_norm", _NORM.pack(
        call.device, call.kind, shape[0], shape[1], kind, eps, 0, *rows(x, "x"), *rows(residual, "residual"),
        *call.buffer(weight, "weight", shape[1:]), *rows(residual_out, "residual_out"), *rows(out, "out"),
        *rows(q, "q", code), *call.buffer(scales, "scales", shape[:1], torch.float32)))
    return NormResult(out, q, scales, residual_out)


class TokenLogprobs(NamedTuple):
    """``token_logprobs``' outputs; ``top_tokens`` and ``top_logprobs`` are None without ``top``."""

    logprobs: object
    entropy: object
    top_tokens: object
    top_logprobs: object


def token_logprobs(logits, tokens, top: int = 0, stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens under the softmax of each row of ``logits`` [rows, vocabulary]
    (a vocabulary of at most 2^20; class scores or log probabilities, as ``Heads.forward`` gives, are taken too).

    ``tokens`` int64 [rows] or [rows, given]; ``logprobs`` has its shape, float32, with NaN for a token
    outside the vocabulary. ``entropy`` [rows] is in nats. ``top`` (at most 32) asks for that many of
    each row's most likely tokens, int64, in falling order, of equally likely ones the lowest first,
    and their log probabilities.
    """
    call = _Call(logits, "logits", stream)
    torch = call.torch
    rows, vocabulary = _dims(logits, "logits", 2)
    shape = tuple(getattr(tokens, "shape", ()))
    if len(shape) not in (1, 2) or shape[0] != rows:
        raise ValueError(f"tokens must be [{rows}] or [{rows}, given], got {list(shape)}")
    given = shape[1] if len(shape) == 2 else 1
    if top < 0:
        raise ValueError(f"top must be 0 or more, got {top}")
    view = call.rows(logits, "logits", (rows, vocabulary))
    ids = call.buffer(tokens, "tokens", shape, torch.int64)
    sizes = (call.device, call.kind, rows, vocabulary, given, top)
    hold, scratch = call.scratch(_scratch_bytes("bilstm_token_logprobs_scratch", _LOGPROBS.pack(*sizes, *(0,) * 16)))
    logprobs, entropy = call.empty(shape, torch.float32), call.empty((rows,), torch.float32)
    top_tokens = call.empty((rows, top), torch.int64) if top else None
    top_logprobs = call.empty((rows, top), torch.float32) if top else None
    place = lambda t: NO_BUFFER if t is None else (t.data_ptr(), t.numel())  # noqa: E731
    call.run("bilstm_token_logprobs", _LOGPROBS.pack(
        *sizes, 0, *view, *ids, *place(logprobs), *place(entropy), *place(top_tokens), *place(top_logprobs), *scratch))
    del hold  # its memory goes back to the call's stream, behind the call's work
    return TokenLogprobs(logprobs, entropy, top_tokens, top_logprobs)

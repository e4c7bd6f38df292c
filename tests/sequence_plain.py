"""64-bit definitions of the causal sequence operators and the bounds their tests use.

Plain torch double precision on the CPU, written from the formulas in include/bilstm.h, row by row
and step by step. Bounds count roundings: one to nearest is off by at most half a step,
``torch.finfo(t).eps / 2`` relative to the value.
"""

import torch

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U32 = 2.0 ** -24  # half a step of float32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def rounded(value, error, dtype):
    """Bound after rounding a value known to within ``error``: the error and half a step; below the
    type's normal range the step is the smallest one."""
    info = torch.finfo(dtype)
    return error + half_step(dtype) * (value.abs() + error) + info.smallest_normal * info.eps / 2


def sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def spans(starts, rows):
    out = []
    for j in range(len(starts) - 1):
        first, end = min(max(starts[j], 0), rows), min(max(starts[j + 1], 0), rows)
        out.append((first, max(0, end - first)))
    return out


def conv(x, weight, starts, bias, state, slots, fresh, silu, y):
    """Returns y, state and the bound of y; ``state`` may be None. All CPU tensors; y holds what
    rows of no sequence keep."""
    dtype = x.dtype
    x, w = x.double(), weight.double()
    taps, channels = w.shape[1], w.shape[0]
    y = y.double().clone()
    bound = torch.zeros_like(y)
    state = None if state is None else state.double().clone()
    for j, (first, length) in enumerate(spans(starts, x.shape[0])):
        place = (slots[j] if slots is not None else j) if state is not None else 0
        if length == 0 or place < 0 or (state is not None and place >= state.shape[0]):
            continue
        kept = torch.zeros(taps - 1, channels, dtype=torch.float64)
        if state is not None and not (fresh is not None and fresh[j]):
            kept = state[place].clone()
        line = torch.cat([kept, x[first: first + length]])
        v = torch.zeros(length, channels, dtype=torch.float64)
        size = torch.zeros_like(v)
        if bias is not None:
            v += bias.double()
            size += bias.double().abs()
        for k in range(taps):
            v += w[:, k] * line[k: k + length]
            size += (w[:, k] * line[k: k + length]).abs()
        # a chain of `taps` fused multiply-adds, one rounding each, of sums no larger than `size`
        error = taps * U32 * size
        out = v
        if silu:
            out = v * sigmoid(v)
            # |d silu / dv| < 1.1; the exponential's argument (rounded: |v| half steps), the exponential and the
            # reciprocal (1 ulp = 2 half steps each), the sum and the product
            error = 1.1 * error + (6 + v.abs()) * U32 * (out.abs() + 1.1 * error)
        y[first: first + length] = out
        bound[first: first + length] = rounded(out, error, dtype)
        if state is not None:
            state[place] = line[length:]
    return y, state, bound

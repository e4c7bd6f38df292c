"""64-bit definitions of cross attention and of the matrix product with its epilogue, and the bounds
their tests use: roundings counted as in sequence_plain.py."""

import torch

from tests.sequence_plain import U32, half_step, rounded, sigmoid, spans

EIGHT = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def attention(q, k, v, starts, memory_starts, lengths, slots, mask, scale, y):
    """Returns y and its bound; all CPU tensors. ``starts`` None: row i is sequence i. ``y`` holds what rows of
    no sequence keep."""
    dtype, (rows, heads, width) = q.dtype, q.shape
    groups = k.shape[1]
    per = heads // groups
    places = len(memory_starts) - 1
    memories = spans(memory_starts, k.shape[0])
    out, bound = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    steps = torch.finfo(dtype).eps / 2
    weights_off = 0.0 if dtype == torch.float32 else steps  # weights enter their product in the tensors' type
    for j, (first, length) in enumerate([(i, 1) for i in range(rows)] if starts is None else spans(starts, rows)):
        place = slots[j] if slots is not None else j
        if length == 0 or place < 0 or place >= places:
            continue
        begin, held = memories[place]
        if lengths is not None:
            held = max(0, min(held, lengths[place]))
        chosen = torch.arange(begin, begin + held)
        if mask is not None:
            chosen = chosen[mask[chosen]]
        here = slice(first, first + length)
        if chosen.numel() == 0:
            out[here], bound[here] = 0, 0
            continue
        qs = q[here].double().transpose(0, 1)  # [heads, rows, width]
        ks = k[chosen].double().transpose(0, 1).repeat_interleave(per, 0)
        vs = v[chosen].double().transpose(0, 1).repeat_interleave(per, 0)
        s = torch.matmul(qs, ks.transpose(1, 2)) * scale
        size = torch.matmul(qs.abs(), ks.abs().transpose(1, 2)) * scale
        w = torch.softmax(s, 2)
        w = torch.where(torch.isneginf(s.amax(2, keepdim=True)), 0.0, w)
        # A score is a sum of `width` products, a whole step of float32 each. Its exponent takes the factor's two
        # roundings, the shift's and its own; shifts change from tile to tile (at least 32 frames each), and with
        # each change the sums take an exponential (1 ulp) and a product.
        most = torch.nan_to_num(s, neginf=0.0).abs().amax(2, keepdim=True)
        tiles = (held + 31) // 32
        off = 2 * U32 * (width + 2) * size + U32 * (6 * most + 8 + 6 * tiles)
        value = torch.matmul(w, vs)
        weight = torch.matmul(w, vs.abs())
        off = torch.where(w > 0, off, 0.0) + weights_off
        # Weights w (1 + e) in the values' sum and in their own: y' - y = sum w e (v - y) / (1 + sum w e), where the last
        # factor is below 1.01. Then additions: 40 in a row within a tile for the sum, one a frame for the values.
        error = torch.zeros_like(value)
        for column in range(0, width, 8):  # a few columns at a time, for the memory
            at = slice(column, column + 8)
            away = (vs[:, None, :, at] - value[:, :, None, at]).abs()
            error[:, :, at] = 1.01 * ((w * off)[..., None] * away).sum(2)
        error = error + U32 * (40 + tiles) * weight + U32 * (held + 8) * weight
        if dtype == torch.float16:  # weights below 2^-24 of the largest lose bits: half of 2^-24 * 2^-10 each
            error = error + 2.0 ** -35 / w.amax(2, keepdim=True).reciprocal() * vs.abs().sum(1)[:, None]
        out[here] = value.transpose(0, 1)
        bound[here] = rounded(value, error, dtype).transpose(0, 1)
    return out, bound


def activation(v, kind, slope):
    if kind == "relu":
        return v.clamp(min=0)
    if kind == "leaky_relu":
        return torch.where(v > 0, v, v * slope)
    if kind == "gelu":
        return 0.5 * v * torch.erfc(-v * 0.5 ** 0.5)
    if kind == "silu":
        return v * sigmoid(v)
    return v


def linear(x, weight, bias, kind, residual, x_scales, weight_scales, slope, dtype):
    """y and its bound; CPU tensors."""
    a, b = x.double(), weight.double()
    n = a.shape[1]
    v, size = a @ b.t(), a.abs() @ b.abs().t()
    # a sum of n terms in any order, a whole step of float32 each; codes of int8 are summed exactly
    error = U32 * v.abs() if x.dtype == torch.int8 else 2 * U32 * (n + 20) * size
    if x.dtype == torch.float8_e4m3fn and dtype != torch.float32:
        # the matrix cores drop what lies below 2^-13 of the largest of eight neighbouring products
        pad = torch.nn.functional.pad
        groups = [pad(t.abs(), (0, -n % 8)).view(t.shape[0], -1, 8) for t in (a, b)]
        for i in range(groups[0].shape[1]):
            most = (groups[0][:, None, i] * groups[1][None, :, i]).amax(2)
            error = error + 2.0 ** -10 * most
    if x_scales is not None:
        scale = x_scales.double()[:, None] * weight_scales.double()
        v, error = v * scale, (error + 3 * U32 * (v.abs() + error)) * scale.abs()
    if bias is not None:
        v = v + bias.double()
        error = error + U32 * (v.abs() + error)
    y = activation(v, kind, slope)
    if kind in ("gelu", "silu"):
        # slopes are below 1.13; the exponent's rounding (v^2 / 2 or |v| half steps), exponential, quotient and
        # products, erfc to 16 ulp
        error = 1.13 * error + (40 + v.abs() + (v * v if kind == "gelu" else 0)) * U32 * y.abs() + 2.0 ** -126 * v.abs()
    elif kind == "leaky_relu":
        error = max(1.0, abs(slope)) * error + U32 * y.abs()
    if residual is not None:
        y = y + residual.double()
        error = error + U32 * (y.abs() + error)
    return y, rounded(y, error, dtype)

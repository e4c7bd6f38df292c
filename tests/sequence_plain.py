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


def norm(x, weight, eps, residual):
    """y, s = x + residual, and the bound of y before its rounding."""
    s = x.double() + (0 if residual is None else residual.double())
    n = s.shape[1]
    mean = s.pow(2).sum(1, keepdim=True) / n
    y = s / torch.sqrt(mean + eps) * weight.double()
    # s is rounded once (and enters the mean twice), the sum of squares has at most n / 64 + 16 roundings
    # in a row (a lane's own terms, then lanes and waves), then division, sum, square root, reciprocal and
    # the two products; half the relative error of the mean reaches the root
    steps = 1 + (2 + n / 64 + 16) / 2 + 6
    return y, s, steps * U32 * y.abs()


def logprobs(logits, tokens, top):
    """Per row: log probabilities of `tokens`, entropy, top tokens and their log probabilities, and the
    bounds of the first two and the last. Masked tokens are minus infinity."""
    z = logits.double()
    rows, v = z.shape
    masked = torch.isinf(z) & (z < 0)
    empty = masked.all(1)
    m = torch.where(empty, 0.0, z.amax(1))[:, None]
    d = torch.where(masked, 0.0, z - m)
    e = torch.where(masked, 0.0, torch.exp(d))
    s = e.sum(1, keepdim=True)
    safe = torch.where(s > 0, s, 1.0)
    log_s = torch.log(safe)
    lp = torch.where(masked | empty[:, None], -float("inf"), d - log_s)
    entropy = (log_s - (e * d).sum(1, keepdim=True) / safe)[:, 0]
    inside = (tokens >= 0) & (tokens < v)
    given = torch.where(inside, torch.gather(lp, 1, tokens.clamp(0, v - 1)), float("nan"))
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    # Relative error of the sum: each term's exponential takes a rounded difference and a rounded product
    # (|d| half steps each; the moves to larger maxima add up to at most |d| once more each) and up to 20
    # exponentials and products of 3 half steps, and at most 32 + 8 + 20 additions in a row.
    spread = (e * d.abs()).sum(1) / safe[:, 0]
    square = (e * d * d).sum(1) / safe[:, 0]
    rel = U32 * (6 * spread + 150)
    big = torch.nan_to_num(given.abs(), nan=0.0, posinf=0.0)
    given_bound = rel[:, None] + 4 * U32 * (2 * log_s.abs() + 2 * big)
    top_lp = torch.gather(lp, 1, order)
    size = torch.nan_to_num(top_lp.abs(), posinf=0.0)
    top_bound = rel[:, None] + 4 * U32 * (2 * log_s.abs() + 2 * size)
    entropy_bound = rel * (1 + spread) + U32 * (6 * square + 150 * spread + 4 * (log_s[:, 0].abs() + spread))
    return (given, entropy, order, top_lp), (given_bound, entropy_bound, top_bound)


def scan(x, dt, a, b, c, starts, d, z, dt_bias, softplus, state, slots, fresh, y, whole_parts=False):
    """The recurrence step by step. Returns y, state, and the bounds of both (y's after its rounding).

    ``state`` may be None; all tensors on the CPU, y holds what rows of no sequence keep.
    """
    dtype = x.dtype
    rows, heads, width = x.shape
    groups, n = b.shape[1], b.shape[2]
    per = heads // groups
    xs, bs, cs, a = x.double(), b.double(), c.double(), a.double()
    v = dt.double() + (0 if dt_bias is None else dt_bias.double())
    # dt + bias is rounded; softplus' slope over its value is at most 1, so |v| half steps carry over;
    # its exponential, logarithm and sum take 8 more
    step, step_rel = (torch.nn.functional.softplus(v, threshold=1000), U32 * (v.abs() + 8)) if softplus else (v, U32 + 0 * v)
    # Products of 16-bit tensors are taken in bf16 parts of each float32 operand, a part leaving at most bf16's half
    # step, 2^-8, of what it rounds. Two parts in products that only meet an output leave 2^-16; an fp16 input is
    # two parts itself (exactly, 16 bits hold its 11), and the product of the two small ones, 2^-8 * 2^-8, is left
    # out too: 2^-15. Three parts in products that meet the state leave 2^-24, and as much for fp16 inputs.
    parts = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -15}[dtype]
    kept = 0.0 if dtype == torch.float32 else 2.0 ** -23
    if whole_parts:  # three parts in the products that only meet an output too
        parts = kept
    y, bound = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    state = None if state is None else state.double().clone()
    state_bound = None if state is None else torch.zeros_like(state)
    for j, (first, length) in enumerate(spans(starts, rows)):
        place = (slots[j] if slots is not None else j) if state is not None else 0
        if length == 0 or place < 0 or (state is not None and place >= state.shape[0]):
            continue
        s = torch.zeros(heads, width, n, dtype=torch.float64)
        if state is not None and not (fresh is not None and fresh[j]):
            s = state[place].clone()
        size, error = s.abs(), torch.zeros_like(s)
        for t in range(first, first + length):
            arg = step[t] * a
            keep = torch.exp(arg)[:, None, None]
            bt, ct = bs[t].repeat_interleave(per, 0)[:, None], cs[t].repeat_interleave(per, 0)[:, None]
            term = (step[t][:, None] * xs[t])[:, :, None] * bt
            # the decay's exponent carries the step's error, two roundings and the exponential's 1 ulp
            off = (arg.abs() * (step_rel[t] + 3 * U32) + 4 * U32)[:, None, None]
            s = keep * s + term
            error = keep * (error + off * size) + (step_rel[t][:, None, None] + kept + 8 * U32) * term.abs()
            size = keep * size + term.abs()
            error = error + 2 * U32 * size  # one more addition, in sums of any order
            out = (s * ct).sum(2)
            weight = (size * ct.abs()).sum(2)
            off_y = (error * ct.abs()).sum(2) + (parts + 2 * U32 * (n + 80)) * weight
            if d is not None:
                skip = d.double()[:, None] * xs[t]
                out, off_y = out + skip, off_y + 2 * U32 * (skip.abs() + weight)
            if z is not None:
                zt = z[t].double()
                gate = zt * sigmoid(zt)
                off_y = off_y * gate.abs() + (8 + zt.abs()) * U32 * gate.abs() * (out.abs() + off_y)
                out = out * gate
            y[t] = out
            bound[t] = rounded(out, off_y, dtype)
        if state is not None:
            state[place] = s
            state_bound[place] = rounded(s, error, torch.float32)
    return y, state, bound, state_bound

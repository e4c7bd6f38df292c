"""64-bit definition of cross attention of one sequence to frames of one memory, with bounds that count what the
kernels promise: weights keep 16 bits and more in every form, exponents are those of differences of scores."""

import torch

from tests.sequence_plain import U32, rounded


def attention(q, k, v, chosen, scale, exact_scores=False):
    """y [rows, heads, width] of all rows of q over the frames ``chosen`` (row numbers of k and v), and its bound; CPU
    tensors. ``exact_scores``: the products' sums are whole numbers that float32 holds."""
    dtype, (rows, heads, width) = q.dtype, q.shape
    per = heads // k.shape[1]
    chosen = torch.as_tensor(chosen, dtype=torch.long)
    if chosen.numel() == 0:
        return torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    qs = q.double().transpose(0, 1)  # [heads, rows, width]
    ks = k[chosen].double().transpose(0, 1).repeat_interleave(per, 0)
    vs = v[chosen].double().transpose(0, 1).repeat_interleave(per, 0)
    s = torch.matmul(qs, ks.transpose(1, 2)) * scale
    size = torch.matmul(qs.abs(), ks.abs().transpose(1, 2)) * scale
    top = s.amax(2, keepdim=True)
    w = torch.softmax(s, 2)
    tiles = (int(chosen.max()) - int(chosen.min())) // 32 + 2
    # A score is a sum of `width` products, a whole step of float32 each.
    off = torch.zeros_like(s) if exact_scores else 2 * U32 * (width + 2) * size
    # An exponent is a rounded difference to a reference up to 2^8 below the maximum, times a factor: in two parts for
    # float32 tensors, else one rounded factor and a rounded product; the moves of the reference add up to the difference
    # once more. Then an exponential and products, with each move too.
    off = off + U32 * ((2 if dtype == torch.float32 else 6) * (top - s + 6) + 8 + 6 * tiles)
    if dtype != torch.float32:
        # weights in two parts, each rounded by at most half a step of the rest
        off = off + (torch.finfo(dtype).eps / 2) ** 2
    value, weight = torch.matmul(w, vs), torch.matmul(w, vs.abs())
    # weights w (1 + e) in the values' sum and in their own: y' - y = sum w e (v - y) / (1 + sum w e)
    error = torch.zeros_like(value)
    for at in range(width):
        error[:, :, at] = 1.01 * (w * off * (vs[:, None, :, at] - value[:, :, at, None]).abs()).sum(2)
    # additions, one a frame for the values and 40 a tile for the sum; quotients of waves, splits and the row
    error = error + U32 * (chosen.numel() + 64 + tiles) * weight
    if dtype == torch.float16:  # weights below 2^-24 of the largest lose bits: half of 2^-34 each
        error = error + 2.0 ** -35 * w.amax(2, keepdim=True) * vs.abs().sum(1)[:, None]
    return value.transpose(0, 1), rounded(value, error, dtype).transpose(0, 1)

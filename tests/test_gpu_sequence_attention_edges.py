"""Cross attention at the edges of its range, in both of its forms (up to 32 packed rows a sequence, and more): bits of
the weights, values and scores of any size, infinities, masks."""

import pytest
import torch

from tests import decoder_strict as strict
from tests.sequence_plain import TYPES

pytestmark = pytest.mark.gpu

ROWS = [3, 70]  # of two heads: the form of few rows, and that of many


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _whole(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32).cuda()


def _make(dtype, rows, frames, heads, groups, width, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return (r(rows, heads, width) * scale).to(dtype), r(frames, groups, width).to(dtype), r(frames, groups, width).to(dtype)


def _run(bl, q, k, v, scale=None, mask=None, lengths=None, starts=None, memory_starts=None, slots=None):
    """One sequence of all rows over one memory of all frames, unless said."""
    return bl.cross_attention(q.cuda(), k.cuda(), v.cuda(), _whole(starts or [0, q.shape[0]]),
                              _whole(memory_starts or [0, k.shape[0]]), memory_lengths=_whole(lengths), slots=_whole(slots),
                              mask=None if mask is None else mask.cuda(), scale=scale).cpu()


def _within(got, ref):
    value, bound = ref
    off = (got.double() - value).abs()
    assert torch.isfinite(off).all() and (off <= bound).all(), f"{(off - bound).max():.3e} over the bound"


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [1, 4, 40, 300])
@pytest.mark.parametrize("width", [32, 64, 128, 256])
def test_weights_keep_their_bits(bl, dtype, rows, width):
    """Sums of values that nearly cancel show what weights lose, for few rows and for many."""
    for frames in (2, 31, 100, 589):
        q, k, v = _make(dtype, rows, frames, 2, 1, width, frames + rows)
        _within(_run(bl, q, k, v), strict.attention(q, k, v, range(frames), width ** -0.5))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [2, 50])
def test_weights_keep_their_bits_over_splits(bl, dtype, rows):
    q, k, v = _make(dtype, rows, 3001, 2, 2, 64, rows)
    _within(_run(bl, q, k, v), strict.attention(q, k, v, range(3001), 64 ** -0.5))

"""Cross attention at the edges of its range, in both of its forms (up to 32 packed rows a sequence, and more): bits of
the weights, values and scores of any size, infinities, masks."""

import pytest
import torch

from tests import decoder_strict as strict
from tests.sequence_plain import TYPES, U32, rounded

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


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("width", [64, 13, 200])
@pytest.mark.parametrize("frames", [1, 32, 50, 64, 130, 3000])
def test_queries_that_are_no_numbers_read_no_masked_frame(bl, dtype, rows, width, frames):
    """A row with nothing to read gets zeros, whatever its query holds, and so does one whose scores are all minus
    infinity, in whole tiles of frames and in tiles with frames that do not count."""
    q, k, v = _make(dtype, rows, frames, 2, 2, width, frames)
    q[0, 0, 3], q[1, 1, 0], q[2, 0, 5] = float("nan"), float("inf"), float("-inf")
    nothing = torch.zeros(frames, dtype=torch.bool)
    assert (_run(bl, q, k, v, mask=nothing) == 0).all() and (_run(bl, q, k, v, lengths=[0]) == 0).all()
    q, k, v = _make(dtype, rows, frames, 2, 2, width, frames)
    q[1, :, 2], k[:, :, 2] = float("inf"), -1.0
    mask = torch.arange(frames) % 5 != 4
    k[~mask] = 1.0
    clean = q.clone()
    clean[1] = 0
    keep = torch.arange(rows) != 1
    for m, lengths in ((mask, None), (None, [min(frames, 4)]), (mask, [max(1, frames - 3)])):
        got = _run(bl, q, k, v, mask=m, lengths=lengths)
        assert (got[1] == 0).all()
        assert torch.equal(got[keep], _run(bl, clean, k, v, mask=m, lengths=lengths)[keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("frames", [40, 600, 3000])
@pytest.mark.parametrize("scale, size", [(1.0, 1.2e19), (1.6e38, 1.0), (1e-3, 1.2e19)])
def test_scores_at_the_ends_of_the_range(bl, dtype, rows, frames, scale, size):
    """Scores near the largest float32, and a scale near it: only the largest count."""
    q, k, v = _make(dtype, rows, frames, 2, 1, 64, frames)
    q[:], k[:] = 0, 0
    for sign in (1, -1):
        q[:, :, 0], k[:, 0, 0] = sign * size, -2 * size
        k[::7, 0, 0] = -size
        k[3, 0, 0], k[frames - 1, 0, 0] = 2 * size, 2 * size
        chosen = [3, frames - 1] if sign > 0 else [f for f in range(frames) if f % 7 and f not in (3, frames - 1)]
        want = v[chosen, 0].double().mean(0).expand(rows, 2, -1)
        # equal weights and their sum are exact; a sum of n values is rounded n times, at most at n of the largest, of which
        # the quotient takes an n-th; then some products, and the output's rounding
        n = len(chosen)
        bound = rounded(want, U32 * (n + 64) * v[chosen].double().abs().amax() + 0 * want, dtype)
        _within(_run(bl, q, k, v, scale=scale), (want, bound))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("frames", [40, 600, 3000])
@pytest.mark.parametrize("far", [1e3, 1.5e5, 1e7])
def test_scores_far_from_zero(bl, dtype, rows, frames, far):
    """Whole numbers far from zero, as sums exact in float32: weights are those of the differences."""
    q, k, v = _make(dtype, rows, frames, 2, 1, 64, frames)
    g = torch.Generator().manual_seed(3)
    q[:], k[:] = 0, 0
    # far = a b, then differences of 0 .. 7
    a = 2.0 ** round(torch.log2(torch.tensor(far) / 2).item())
    q[:, :, 0], q[:, :, 1], k[:, 0, 0] = a, 1, 2
    k[:, 0, 1] = torch.randint(0, 8, (frames,), generator=g).to(dtype)
    if a > torch.finfo(dtype).max:
        pytest.skip("not a number of this type")
    _within(_run(bl, q, k, v, scale=1.0), strict.attention(q, k, v, range(frames), 1.0, exact_scores=True))


@pytest.mark.parametrize("dtype, size", [(torch.float32, 1e35), (torch.float32, 3e36), (torch.float32, 3e38), (torch.float32, 1e-30),
                                         (torch.float32, 1e-36), (torch.bfloat16, 1e35), (torch.bfloat16, 3e36), (torch.bfloat16, 3e38),
                                         (torch.bfloat16, 1e-30), (torch.bfloat16, 1e-36), (torch.float16, 6e4), (torch.float16, 1e-7)],
                         ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("width", [64, 200])
def test_values_of_any_size(bl, dtype, size, rows, width):
    """Weights are measured from a reference that the maximum may pass, and many add up: the quotient is a value's size."""
    for frames in (64, 300, 3000):
        q, k, v = _make(dtype, rows, frames, 2, 1, width, frames, scale=0.5)
        q[:, :, 0], k[:, 0, 0] = 1.0, (torch.arange(frames) // 32 % 4 * 1.5 * width ** 0.5).to(dtype)  # rises from tile to tile
        v = ((0.5 + torch.rand(frames, 1, width, generator=torch.Generator().manual_seed(1)) / 2) * size).to(dtype)
        v[:, :, 1::2] *= -1
        value, bound = strict.attention(q, k, v, range(frames), width ** -0.5)
        _within(_run(bl, q, k, v), (value, bound + frames * 2.0 ** -149))  # products may be subnormal numbers


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("width", [64, 13])
@pytest.mark.parametrize("frames", [1, 40, 600, 3000])
def test_infinite_values_give_infinities(bl, dtype, rows, width, frames):
    q, k, v = _make(dtype, rows, frames, 2, 1, width, frames, scale=0.3)
    v[:, :, 2], v[:, :, 5], v[:, :, 9] = 0, 0, 0
    clean = _run(bl, q, k, v)
    inf = float("inf")
    v[frames // 2, 0, 2], v[frames - 1, 0, 5] = inf, -inf
    v[0, 0, 9], v[frames - 1, 0, 9] = inf, -inf
    got = _run(bl, q, k, v)
    assert (got[:, :, 2] == inf).all() and (got[:, :, 5] == -inf).all()
    assert torch.isnan(got[:, :, 9]).all() if frames > 1 else (got[:, :, 9] == -inf).all()
    rest = [c for c in range(width) if c not in (2, 5, 9)]
    assert torch.equal(got[:, :, rest], clean[:, :, rest])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("width", [64, 80, 13, 100, 200, 256])
def test_masks_over_many_tiles(bl, dtype, rows, width):
    """Masked frames among others, whole tiles of them, and a memory of them alone; what they hold is nothing."""
    held = 333
    g = torch.Generator().manual_seed(width)
    q, k, v = _make(dtype, 3 * rows, 3 * held, 4, 2, width, 7)
    mask = torch.rand(3 * held, generator=g) < 0.5
    mask[20: 20 + 150], mask[held + 256:], mask[2 * held:] = False, False, False
    lengths, memory_starts, starts = [held - 9, held, held], [3, held, 2 * held, 3 * held], [0, rows, 2 * rows, 3 * rows]
    run = lambda: _run(bl, q, k, v, mask=mask, lengths=lengths, starts=starts, memory_starts=memory_starts)  # noqa: E731
    clean = run()
    for j in range(2):
        chosen = [f for f in range(memory_starts[j], min(memory_starts[j] + lengths[j], memory_starts[j + 1])) if mask[f]]
        value, bound = strict.attention(q[j * rows: (j + 1) * rows], k, v, chosen, width ** -0.5)
        _within(clean[j * rows: (j + 1) * rows], (value, bound))
    assert (clean[2 * rows:] == 0).all()
    reads = torch.zeros(3 * held, dtype=torch.bool)
    for j in range(3):
        reads[memory_starts[j]: min(memory_starts[j] + lengths[j], memory_starts[j + 1])] = True
    for t, bad in ((k, float("nan")), (v, float("inf")), (k, float("-inf")), (v, float("nan")), (k, torch.finfo(dtype).max)):
        t[~(reads & mask)] = bad
        assert torch.equal(run(), clean)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [2, 50])
@pytest.mark.parametrize("width", [64, 100])
def test_masks_over_splits(bl, dtype, rows, width):
    frames = 4099
    q, k, v = _make(dtype, rows, frames, 4, 2, width, rows)
    mask = torch.rand(frames, generator=torch.Generator().manual_seed(2)) < 0.3
    mask[500:1800] = False
    chosen = torch.nonzero(mask[:frames - 40])[:, 0]
    clean = _run(bl, q, k, v, mask=mask, lengths=[frames - 40])
    _within(clean, strict.attention(q, k, v, chosen, width ** -0.5))
    k[~mask], v[~mask] = float("nan"), float("inf")
    k[frames - 40:], v[frames - 40:] = float("inf"), float("nan")
    assert torch.equal(_run(bl, q, k, v, mask=mask, lengths=[frames - 40]), clean)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("width", [65, 96, 127, 128, 129, 200, 255, 256])
@pytest.mark.parametrize("offset", [1, 8])
def test_wide_heads_at_any_element(bl, dtype, rows, width, offset):
    """Keys and values side by side in wider rows, at an element or at 16 bytes; single rows too."""
    held, groups, heads = 150, 2, 4
    q, k, v = _make(dtype, rows, held, heads, groups, width, width)
    n = groups * width
    wide = torch.full((held, 2 * n + 2 * offset), float("nan"), dtype=dtype, device="cuda")
    kd, vd = wide[:, offset: offset + n].view(held, groups, width), wide[:, offset + n: offset + 2 * n].view(held, groups, width)
    kd.copy_(k), vd.copy_(v)
    into = torch.full((rows, heads * width + offset), 3.0, dtype=dtype, device="cuda")
    yd = into[:, offset:].view(rows, heads, width)
    got = bl.cross_attention(q.cuda(), kd, vd, _whole([0, rows]), _whole([20, held - 3]), out=yd)
    ref = strict.attention(q, k, v, range(20, held - 3), width ** -0.5)
    assert got is yd and (into[:, :offset] == 3).all()
    _within(yd.cpu(), ref)
    _within(bl.cross_attention_step(q.cuda(), kd, vd, _whole([20, held - 3]), slots=_whole([0] * rows)).cpu(), ref)


@pytest.mark.parametrize("rows", ROWS)
def test_captured_with_ordinary_values_and_replayed_with_large_ones(bl, rows):
    """Whether the frames are gone over again is found out on the device, by each replay."""
    frames, width = 3000, 64
    q, k, v = (t.cuda() for t in _make(torch.bfloat16, rows, frames, 2, 1, width, 5, scale=0.5))
    large, infinite = (v.abs() + 1) * 2.5e37, v.clone()  # up to 1.4e38
    infinite[frames // 2] = float("inf")
    starts, memory_starts = _whole([0, rows]), _whole([0, frames])
    call = lambda held: bl.cross_attention(q, k, held, starts, memory_starts)  # noqa: E731
    expect = [call(t) for t in (v, large, infinite)]
    held = v.clone()
    call(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(held)
    for i in (0, 1, 2, 0, 1):
        held.copy_((v, large, infinite)[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect[i])
        call(v)
        torch.cuda.synchronize()
    assert torch.isfinite(expect[1]).all() and (expect[2] == float("inf")).all()

"""Cross attention of packed and single rows to memories of frames, against 64 bits."""

import pytest
import torch

from tests import decoder_plain as plain
from tests.sequence_plain import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _whole(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32).cuda()


def _make(dtype, rows, memory_rows, heads, groups, width, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((r(rows, heads, width) * scale).to(dtype), r(memory_rows, groups, width).to(dtype), r(memory_rows, groups, width).to(dtype))


def _run(bl, q, k, v, starts, memory_starts, lengths=None, slots=None, mask=None, scale=None, out=None, **more):
    to = lambda t: None if t is None else t.cuda()  # noqa: E731
    rest = dict(memory_lengths=_whole(lengths), slots=_whole(slots), mask=to(mask), scale=scale, out=out, **more)
    if starts is None:
        return bl.cross_attention_step(to(q), to(k), to(v), _whole(memory_starts), **rest)
    return bl.cross_attention(to(q), to(k), to(v), _whole(starts), _whole(memory_starts), **rest)


def _same(got, value, bound):
    got = got.cpu().double()
    fine = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got), fine)
    assert torch.equal(torch.isnan(got), torch.isnan(value))
    off = (got - value)[fine].abs()
    assert (off <= bound[fine]).all(), f"{(off - bound[fine]).max():.3e} over the bound"


def _check(bl, q, k, v, starts, memory_starts, lengths=None, slots=None, mask=None, scale=None, **more):
    keep = torch.full(q.shape, 7.5).to(q.dtype)
    got = _run(bl, q, k, v, starts, memory_starts, lengths, slots, mask, scale, keep.cuda(), **more)
    width = q.shape[2]
    _same(got, *plain.attention(q, k, v, starts, memory_starts, lengths, slots, mask, scale or width ** -0.5, keep))
    return got


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("width", [1, 7, 8, 32, 40, 64, 80, 96, 128, 200, 256])
@pytest.mark.parametrize("heads, groups", [(2, 2), (6, 2)])
def test_widths(bl, dtype, width, heads, groups):
    q, k, v = _make(dtype, 45, 150, heads, groups, width, width)
    _check(bl, q, k, v, [0, 3, 40, 45], [0, 90, 91, 150])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("frames", [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 589])
@pytest.mark.parametrize("rows", [1, 33])
def test_lengths(bl, dtype, frames, rows):
    q, k, v = _make(dtype, rows, frames + 2, 4, 4, 64, frames)
    _check(bl, q, k, v, [0, rows], [1, frames + 1])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300])
def test_row_counts(bl, dtype, rows):
    q, k, v = _make(dtype, rows + 3, 200, 6, 3, 64, rows)
    _check(bl, q, k, v, [2, rows + 2], [0, 200])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("step", [False, True])
def test_long_memories_are_split_and_joined(bl, dtype, step):
    frames = 4099 if dtype != torch.float32 else 2051
    q, k, v = _make(dtype, 5, 2 * frames, 4, 2, 64, 9)
    mask = torch.rand(2 * frames, generator=torch.Generator().manual_seed(1)) < 0.7
    _check(bl, q, k, v, None if step else [0, 2, 2, 5], [0, frames, frames, 2 * frames],
           lengths=[frames - 70, 0, frames], slots=[2, 0, 1, 2, 9] if step else [2, 1, 0], mask=mask)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("heads, groups, width", [(1, 1, 64), (8, 8, 64), (8, 2, 128), (32, 1, 32), (70, 1, 16), (9, 3, 80), (160, 1, 8)])
def test_single_rows(bl, dtype, heads, groups, width):
    q, k, v = _make(dtype, 7, 500, heads, groups, width, heads)
    _check(bl, q, k, v, None, [0, 100, 101, 350, 350, 420, 500], lengths=[90, 1, 300, 5, 70, 0], slots=[5, 0, 1, 2, 2, 4, 3])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_packed_sequences_read_named_memories(bl, dtype):
    """Empty sequences and memories, one memory read twice, padding, rows of no sequence, lengths outside."""
    q, k, v = _make(dtype, 300, 400, 4, 2, 64, 5)
    starts = [4, 4, 20, 170, 171, 171, 290]
    got = _check(bl, q, k, v, starts, [10, 130, 130, 300, 395], lengths=[500, 3, 64, -1], slots=[0, 2, 0, -1, 1, 4])
    keep = torch.full((1, 4, 64), 7.5).to(dtype)
    assert torch.equal(got[:4].cpu(), keep.expand(4, -1, -1)) and torch.equal(got[290:].cpu(), keep.expand(10, -1, -1))
    assert torch.equal(got[170:171].cpu(), keep)  # slot -1
    got = _check(bl, q, k, v, starts, [10, 130, 130, 300, 395], lengths=[500, 3, 64, -1], slots=[3, 1, 2, 0, 1, 2])
    assert (got[4:20] == 0).all()  # a memory of no rows


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_starts_outside_are_clamped(bl, dtype):
    q, k, v = _make(dtype, 20, 50, 2, 1, 32, 6)
    _check(bl, q, k, v, [-5, 3, 900, 7], [-3, 20, 1000, 5], slots=[0, 1, 2])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("width", [64, 80, 13])
def test_masked_frames_may_hold_anything(bl, dtype, step, width):
    """Not-a-numbers and infinities in masked frames, behind a memory's length and outside of every memory, and
    memories whose mask leaves nothing."""
    rows, held = 6, 130
    q, k, v = _make(dtype, rows, 3 * held, 4, 2, width, 7)
    g = torch.Generator().manual_seed(8)
    mask = torch.rand(3 * held, generator=g) < 0.5
    mask[2 * held:] = False
    starts = None if step else [0, 1, 4, 6]
    memory_starts, lengths = [3, held, 2 * held, 3 * held], [100, 77, held]
    slots = [0, 1, 2, 1, 0, 2] if step else [0, 1, 2]
    clean = _run(bl, q, k, v, starts, memory_starts, lengths, slots, mask)
    dirty = torch.ones(3 * held, dtype=torch.bool)
    for p in range(3):
        at = torch.arange(memory_starts[p], memory_starts[p] + min(lengths[p], memory_starts[p + 1] - memory_starts[p]))
        dirty[at] = ~mask[at]
    for t, bad in ((k, float("nan")), (v, float("inf")), (k, float("-inf")), (v, float("nan")), (k, torch.finfo(dtype).max)):
        t[dirty] = bad
        assert torch.equal(_run(bl, q, k, v, starts, memory_starts, lengths, slots, mask), clean)
    _same(clean, *plain.attention(q, torch.where(dirty[:, None, None], 0, k), torch.where(dirty[:, None, None], 0, v), starts,
                                  memory_starts, lengths, slots, mask, width ** -0.5, torch.zeros(q.shape).to(dtype)))
    assert (clean[2 if step else 4:][:1] == 0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_not_numbers_stay_in_their_rows(bl, dtype):
    q, k, v = _make(dtype, 40, 100, 2, 2, 64, 11)
    clean = _run(bl, q, k, v, [0, 40], [0, 100])
    q[3, 1, 5] = float("nan")
    q[7, 0, 0] = float("inf")
    got = _run(bl, q, k, v, [0, 40], [0, 100])
    assert torch.isnan(got[3, 1]).all() and torch.isnan(got[7, 0]).all()
    other = torch.ones(40, 2, dtype=torch.bool)
    other[3, 1] = other[7, 0] = False
    assert torch.equal(got[other.cuda()], clean[other.cuda()])
    v[50, 0, 9] = float("nan")
    got = _run(bl, q, k, v, [0, 40], [0, 100])
    assert torch.isnan(got[:, 0, 9]).all() and torch.equal(got[:3, 1], clean[:3, 1])
    assert torch.isfinite(got[:3, 0, :9]).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [5, 150])
def test_a_row_does_not_depend_on_its_neighbours(bl, dtype, rows):
    """Neighbours whose maxima rise from tile to tile leave a row's bits as they are."""
    q, k, v = _make(dtype, rows, 400, 2, 1, 64, 18)
    k[:, 0, 0] = (torch.arange(400.0) / 50).to(dtype)
    clean = _run(bl, q, k, v, [0, rows], [0, 400])
    q[1::2, :, 0] = 60.0
    got = _run(bl, q, k, v, [0, rows], [0, 400])
    assert torch.equal(got[::2], clean[::2]) and not torch.equal(got[1::2], clean[1::2])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scores_of_minus_infinity_and_of_any_size(bl, dtype):
    """Frames at minus infinity do not count, rows of them alone get zeros; scores may be far from 0."""
    q, k, v = _make(dtype, 34, 70, 1, 1, 8, 12)
    q[:, 0, 0], k[:, 0, 0] = 1, 0
    k[::2, 0, 0] = float("-inf")
    keep = torch.ones(70, dtype=torch.bool)
    keep[::2] = False
    k_without = torch.where(keep[:, None, None], k, 0)
    got = _run(bl, q, k, v, [0, 34], [0, 70])
    _same(got, *plain.attention(q, k_without, v, [0, 34], [0, 70], None, None, keep, 8 ** -0.5, torch.zeros(q.shape).to(dtype)))
    k[:, 0, 0] = float("-inf")
    assert (_run(bl, q, k, v, [0, 34], [0, 70]) == 0).all()
    q, k, v = _make(dtype, 34, 300, 2, 1, 64, 13, scale=60.0)
    k[:, 0, 3] += torch.arange(300.0).to(dtype) / 8  # maxima move from tile to tile
    _check(bl, q, k, v, [0, 34], [0, 300], scale=1.0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_many_small_weights(bl, dtype):
    """One frame with the largest score and thousands far below, which together matter."""
    frames = 3000
    q, k, v = _make(dtype, 3, frames, 1, 1, 32, 14)
    q[:] = 0
    q[:, 0, 0] = 1
    k[:, 0, 0] = -8.0
    k[17, 0, 0] = 3.0
    v = v.abs()
    _check(bl, q, k, v, [0, 3], [0, frames], scale=1.0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_strides_and_alignments(bl, dtype, offset):
    """Keys and values side by side in one projection's rows, queries and outputs inside wider rows."""
    heads, groups, width, rows, held = 4, 2, 64, 50, 130
    q, k, v = _make(dtype, rows, held, heads, groups, width, 15)
    wide = torch.zeros(held, 2 * groups * width + offset, dtype=dtype, device="cuda")
    into = torch.full((rows, heads * width + 5 + offset), 3.0, dtype=dtype, device="cuda")
    of = torch.zeros(rows, heads * width + 9, dtype=dtype, device="cuda")
    n = groups * width
    kd, vd = wide[:, offset: offset + n].view(held, groups, width), wide[:, offset + n:].view(held, groups, width)
    qd, yd = of[:, offset: offset + heads * width].view(rows, heads, width), into[:, offset: offset + heads * width].view(rows, heads, width)
    kd.copy_(k), vd.copy_(v), qd.copy_(q)
    whole = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    got = bl.cross_attention(qd, kd, vd, whole([0, 20, rows]), whole([0, 50, held]), out=yd)
    assert got is yd
    _same(yd, *plain.attention(q, k, v, [0, 20, rows], [0, 50, held], None, None, None, width ** -0.5, torch.zeros(q.shape)))
    assert (into[:, :offset] == 3).all() and (into[:, offset + heads * width:] == 3).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_forms_agree(bl, dtype):
    """Single rows as sequences of one row, and hypotheses of one memory as one sequence or as several."""
    q, k, v = _make(dtype, 12, 300, 4, 2, 64, 16)
    slots = [0, 0, 0, 1, 1, 1, 2, 2, 2, 0, 1, 2]
    args = (q, k, v, None, [0, 100, 170, 300])
    step = _check(bl, *args, slots=slots)
    _check(bl, q, k, v, list(range(13)), [0, 100, 170, 300], slots=slots)
    got = _check(bl, q[:9], k, v, [0, 3, 6, 9], [0, 100, 170, 300])
    assert (got.float() - step[:9].float()).abs().max() < 0.05


def test_nothing_to_do(bl):
    for dtype in TYPES:
        q, k, v = (t.cuda() for t in _make(dtype, 4, 6, 2, 1, 32, 17))
        whole = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
        assert bl.cross_attention(q[:0], k, v, whole([0, 0]), whole([0, 6])).shape == (0, 2, 32)
        out = torch.full_like(q, 2.0)
        bl.cross_attention(q, k, v, whole([0]), whole([0, 6]), out=out)
        assert (out == 2).all()
        # memories without rows, and no memories at all
        assert (bl.cross_attention(q, k[:0], v[:0], whole([0, 4]), whole([0, 0])) == 0).all()
        out = torch.full_like(q, 2.0)
        bl.cross_attention_step(q, k, v, whole([0]), slots=whole([0, 0, -1, 1]), out=out)
        assert (out == 2).all()
        bl.cross_attention_step(q, k[:0], v[:0], whole([0, 0]), slots=whole([0, 0, -1, 1]), mask=torch.ones(0, dtype=torch.bool).cuda(), out=out)
        assert (out[:2] == 0).all() and (out[2:] == 2).all()


def test_thousands_of_sequences(bl):
    """More sequences than one round of the search looks at, most of one row, some of none, one long."""
    count = 5000
    rows = [j % 3 for j in range(count)]
    rows[777] = 600
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    q, k, v = _make(torch.bfloat16, starts[-1], 90, 2, 1, 32, 19)
    _check(bl, q, k, v, starts, [0, 40, 41, 90], slots=[j % 4 - (j % 11 == 0) * 4 for j in range(count)])


def test_a_mask_of_bytes(bl):
    q, k, v = _make(torch.float16, 9, 80, 2, 2, 64, 20)
    mask = torch.arange(80) % 3 != 1
    want = _run(bl, q, k, v, [0, 9], [0, 80], mask=mask)
    assert torch.equal(_run(bl, q, k, v, [0, 9], [0, 80], mask=mask.to(torch.uint8) * 255), want)
    _check(bl, q, k, v, [0, 9], [0, 80], mask=mask)

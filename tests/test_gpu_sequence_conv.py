"""The causal convolution on the GPU against its 64-bit definition."""

import pytest
import torch

from tests import sequence_plain as plain

pytestmark = pytest.mark.gpu

LENGTHS = {
    "one": [1],
    "short": [1, 0, 2, 3, 0, 4],
    "edges": [15, 16, 17, 31, 33, 0, 48, 64],
    "long": [1000, 7],
    "ones": [1] * 40,
}


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _starts(lengths, before=0):
    out = [before]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _inputs(dtype, rows, channels, taps, sequences, seed, places=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=g).to(dtype)  # noqa: E731
    places = sequences + 2 if places is None else places
    return r(rows, channels), r(channels, taps), r(channels), r(places, taps - 1, channels), \
        torch.randperm(places, generator=g)[:sequences].to(torch.int32), torch.rand(sequences, generator=g) < 0.5


def _compare(y, state, ref, ref_state, bound):
    assert torch.isfinite(y.double()).all()
    off = (y.cpu().double() - ref).abs()
    assert (off <= bound).all(), f"worst {(off - bound).max().item():.3e} over the bound"
    if ref_state is not None:
        assert torch.equal(state.cpu().double(), ref_state)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("channels", [1, 13, 64])
def test_packed_sequences_match_the_definition(bl, dtype, taps, lengths, channels):
    lens = LENGTHS[lengths]
    before, behind = 3, 5
    starts = _starts(lens, before)
    rows = starts[-1] + behind
    x, w, b, state, slots, fresh = _inputs(dtype, rows, channels, taps, len(lens), 100 + taps)
    slots[len(lens) // 2] = -1 if len(lens) > 3 else slots[len(lens) // 2]
    out = torch.full((rows, channels), 7.0, dtype=dtype)
    ref, ref_state, bound = plain.conv(x, w, starts, b, state, slots.tolist(), fresh.tolist(), True, out)
    s = state.cuda()
    y = bl.causal_conv(x.cuda(), w.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), bias=b.cuda(), state=s,
                       slots=slots.cuda(), fresh=fresh.cuda(), out=out.cuda())
    _compare(y, s, ref, ref_state, bound)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_without_state_bias_and_activation(bl, dtype):
    starts = _starts([5, 20, 1])
    x, w, _, _, _, _ = _inputs(dtype, 26, 24, 4, 3, 5)
    ref, _, bound = plain.conv(x, w, starts, None, None, None, None, False, torch.zeros_like(x))
    y = bl.causal_conv(x.cuda(), w.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), silu=False)
    _compare(y, None, ref, None, bound)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("channels", [1, 37, 256])
def test_steps_continue_a_prompt(bl, dtype, taps, channels):
    """A prompt, then single rows: the same rows as one longer prompt, bit for bit."""
    lens, more = [3, 1, 20, 2], 5
    x, w, b, state, slots, fresh = _inputs(dtype, sum(lens) + len(lens) * more, channels, taps, len(lens), 9)
    x, w, b, slots = x.cuda(), w.cuda(), b.cuda(), slots.cuda()
    whole_starts = _starts([n + more for n in lens])
    s_whole, s_parts = state.cuda(), state.cuda()
    whole = bl.causal_conv(x, w, torch.tensor(whole_starts, dtype=torch.int32).cuda(), bias=b, state=s_whole, slots=slots)
    prompt = torch.cat([x[whole_starts[j]: whole_starts[j] + n] for j, n in enumerate(lens)])
    bl.causal_conv(prompt, w, torch.tensor(_starts(lens), dtype=torch.int32).cuda(), bias=b, state=s_parts, slots=slots)
    for k in range(more):
        at = [whole_starts[j] + n + k for j, n in enumerate(lens)]
        y = bl.causal_conv_step(x[at].contiguous(), w, s_parts, bias=b, slots=slots)
        assert torch.equal(y, whole[at])
    assert torch.equal(s_whole, s_parts)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_step_skips_padding_and_takes_strided_rows(bl, dtype):
    wide = torch.randn(4, 96, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    x = wide[:, 16:48]
    _, w, b, state, _, _ = _inputs(dtype, 4, 32, 4, 4, 3)
    slots = torch.tensor([2, -1, 99, 0], dtype=torch.int32)
    out = torch.full((4, 32), 5.0, dtype=dtype)
    s = state.cuda()
    y = bl.causal_conv_step(x, w.cuda(), s, bias=b.cuda(), slots=slots.cuda(), out=out.cuda())
    ref, ref_state, bound = plain.conv(x.cpu(), w, [0, 1, 2, 3, 4], b, state, slots.tolist(), None, True, out)
    _compare(y, s, ref, ref_state, bound)


def test_output_columns_beside_input_columns(bl):
    """x and y as columns of one wide buffer, at an offset that leaves no wide alignment."""
    buffer = torch.randn(40, 103, generator=torch.Generator().manual_seed(4)).cuda()
    x, y = buffer[:, 1:51], buffer[:, 52:102]
    w = torch.randn(50, 3, generator=torch.Generator().manual_seed(5))
    keep = buffer.clone()
    ref, _, bound = plain.conv(x.cpu(), w, [0, 25, 40], None, None, None, None, True, y.cpu())
    bl.causal_conv(x, w.cuda(), torch.tensor([0, 25, 40], dtype=torch.int32).cuda(), out=y)
    _compare(y, None, ref, None, bound)
    assert torch.equal(buffer[:, :52], keep[:, :52]) and torch.equal(buffer[:, 102:], keep[:, 102:])


def test_row_offsets_past_32_bits(bl):
    stride = (1 << 30) + 8
    base = torch.zeros(2 * stride + 64, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((3, 64), (stride, 1))
    x.copy_(torch.randn(3, 64, generator=torch.Generator().manual_seed(6)))
    w = torch.randn(64, 4, generator=torch.Generator().manual_seed(7)).bfloat16()
    ref, _, bound = plain.conv(x.cpu(), w, [0, 3], None, None, None, None, True, torch.zeros(3, 64, dtype=torch.bfloat16))
    y = bl.causal_conv(x, w.cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda())
    _compare(y, None, ref, None, bound)


def test_starts_outside_the_rows_are_clamped(bl):
    """Row numbers that no batch has: every access stays inside the buffers, sound sequences are right."""
    x, w, b, state, _, _ = _inputs(torch.float32, 20, 32, 4, 4, 8)
    starts = [-7, 6, 6, 100, 2 ** 31 - 1]
    out = torch.zeros(20, 32)
    s = state.cuda()
    y = bl.causal_conv(x.cuda(), w.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), bias=b.cuda(), state=s,
                       out=out.cuda())
    ref, ref_state, bound = plain.conv(x, w, starts, b, state, None, None, True, out)
    _compare(y, s, ref, ref_state, bound)


def test_own_stream_and_captured_graph(bl):
    x, w, b, state, slots, _ = _inputs(torch.bfloat16, 50, 128, 4, 3, 11)
    starts = torch.tensor([0, 20, 20, 50], dtype=torch.int32).cuda()
    x, w, b, slots = x.cuda(), w.cuda(), b.cuda(), slots.cuda()
    expect_state = state.cuda()
    expect = [bl.causal_conv(x, w, starts, bias=b, state=expect_state, slots=slots) for _ in range(4)]
    side = torch.cuda.Stream()
    s = state.cuda()
    torch.cuda.synchronize()
    first = bl.causal_conv(x, w, starts, bias=b, state=s, slots=slots, stream=side)
    side.synchronize()
    assert torch.equal(first, expect[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = bl.causal_conv(x, w, starts, bias=b, state=s, slots=slots)
    for k in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect[k])
        x.mul_(1.0)
    assert torch.equal(s, expect_state)


# values where a sigmoid's exponential leaves float32's range on either side, and what is not a number
GATE_VALUES = [0.0, -0.0, 1e-30, -1e-30, 1.0, -1.0, 20.0, -20.0, 60.0, -60.0, 86.0, -86.0, 88.0, -88.0, 90.0, -90.0, -100.0,
               -104.0, 127.0, -127.0, 1e4, -1e4, 6e4, -6e4, 1e30, -1e30, 2.3e38, 2.4e38, -2.4e38, 3e38, -3e38, float("inf"),
               float("-inf"), float("nan")]


def _check_gate(got, v):
    """``got`` is v * sigmoid(v), with a bound of plain.conv's: the exponential's rounded argument, itself and the
    reciprocal, the sum and the product. A sigmoid below float32's normal range may count as zero."""
    got, dtype = got.cpu(), v.dtype
    x = v.double()
    expect = torch.where(x == float("-inf"), float("nan"), x * plain.sigmoid(x))
    fine = torch.isfinite(expect)
    assert torch.equal(torch.isnan(got), torch.isnan(expect)), (got, expect)
    assert torch.equal(got[~fine & ~torch.isnan(expect)].double(), expect[~fine & ~torch.isnan(expect)])
    error = torch.where(fine, (6 + x.abs().clamp(max=1e3)) * plain.U32 * expect.abs() + x.abs().clamp(max=1e3) * 2.0 ** -126, 0.0)
    off = (got.double() - expect).abs()
    assert (off[fine] <= plain.rounded(expect, error, dtype)[fine]).all(), (v[fine], got[fine], expect[fine])


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("step", [False, True])
def test_gate_of_any_value(bl, dtype, step):
    """One tap of 1, so that the gate gets x itself: infinities, values near the type's largest, far negative ones."""
    v = torch.tensor(GATE_VALUES).to(dtype)
    x = v[:, None].repeat(1, 24).contiguous()
    weight = torch.zeros(24, 2, dtype=dtype)
    weight[:, 1] = 1.0
    rows = x.shape[0]
    if step:
        y = bl.causal_conv_step(x.cuda(), weight.cuda(), torch.zeros(rows, 1, 24, dtype=dtype, device="cuda"))
    else:
        y = bl.causal_conv(x.cuda(), weight.cuda(), torch.arange(rows + 1, dtype=torch.int32, device="cuda"))
    _check_gate(y, x)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("channels, taps", [((1 << 29) + 13, 4), ((1 << 31) - 1, 2)])
def test_channels_whose_taps_pass_32_bits(bl, step, channels, taps):
    """A row's number of taps, and of vectors of channels, beyond 31 bits, up to the most channels there are.
    Looked at where they would wrap and at both ends."""
    g = torch.Generator(device="cuda").manual_seed(41)
    make = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    x, weight, state = make(2, channels), make(channels, taps), make(2, taps - 1, channels)
    at = torch.cat([torch.arange(0, 40), torch.arange((1 << 28) - 20, (1 << 28) + 20), torch.arange(channels - 40, channels)])
    on = at.cuda()
    few = (x[:, on].cpu(), weight[on].cpu(), state[:, :, on].cpu())
    if step:
        y = bl.causal_conv_step(x, weight, state)
    else:
        y = bl.causal_conv(x, weight, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), state=state)
    ref, ref_state, bound = plain.conv(few[0], few[1], [0, 1, 2], None, few[2], None, None, True, torch.zeros_like(few[0]))
    _compare(y[:, on], state[:, :, on], ref, ref_state, bound)


def test_a_state_without_places(bl):
    """A cache of no places is not the lack of one: no sequence may take a place in it."""
    x = torch.randn(3, 8).cuda()
    w, none = torch.randn(8, 2).cuda(), torch.zeros(0, 1, 8).cuda()
    starts = torch.tensor([0, 3], dtype=torch.int32).cuda()
    out = torch.full((3, 8), 5.0).cuda()
    with pytest.raises(bl.BilstmError):
        bl.causal_conv(x, w, starts, state=none, out=out)
    with pytest.raises(bl.BilstmError):
        bl.causal_conv_step(x, w, none, out=out)
    heads, dt, a, b = x.new_ones(3, 1, 32), x.new_ones(3, 1), -x.new_ones(1), x.new_ones(3, 1, 16)
    with pytest.raises(bl.BilstmError):
        bl.selective_scan(heads, dt, a, b, b, starts, state=x.new_zeros(0, 1, 32, 16))
    with pytest.raises(bl.BilstmError):
        bl.selective_scan_step(heads, dt, a, b, b, x.new_zeros(0, 1, 32, 16))
    # with slots every sequence is padding: its rows stay as they were
    slots = torch.tensor([0], dtype=torch.int32).cuda()
    bl.causal_conv(x, w, starts, state=none, slots=slots, out=out)
    bl.causal_conv_step(x, w, none, slots=slots.repeat(3), out=out)
    assert (out == 5.0).all()
    kept = x.new_full((3, 1, 32), 5.0)
    bl.selective_scan(heads, dt, a, b, b, starts, state=x.new_zeros(0, 1, 32, 16), slots=slots, out=kept)
    bl.selective_scan_step(heads, dt, a, b, b, x.new_zeros(0, 1, 32, 16), slots=slots.repeat(3), out=kept)
    assert (kept == 5.0).all()

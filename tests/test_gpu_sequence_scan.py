"""The selective state space scan on the GPU against its recurrence in 64 bits."""

import pytest
import torch

from tests import sequence_plain as plain

pytestmark = pytest.mark.gpu

LENGTHS = {
    "one": [1],
    "edges": [31, 32, 33, 0, 1, 63, 64, 65],
    "chunks": [130, 2, 257],
    "ones": [1] * 20,
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


class Case:
    """Inputs on the CPU; x, b and c as columns of one buffer."""

    def __init__(self, dtype, rows, heads, width, groups, states, sequences, seed, pad=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
        self.dtype, self.rows, self.heads, self.width, self.groups, self.states = dtype, rows, heads, width, groups, states
        inner = heads * width
        self.wide = (r(rows, inner + 2 * groups * states + pad) * 0.7).to(dtype)
        self.dt = (r(rows, heads) * 0.5).to(dtype)
        self.dt_bias = r(heads) - 2.0
        self.a = -(torch.rand(heads, generator=g) * 8 + 0.5)
        self.d = r(heads)
        self.z = r(rows, heads, width).to(dtype)
        self.state = r(sequences + 2, heads, width, states)
        self.slots = torch.randperm(sequences + 2, generator=g)[:sequences].to(torch.int32)
        self.fresh = torch.rand(sequences, generator=g) < 0.5

    def views(self, wide):
        inner, gn = self.heads * self.width, self.groups * self.states
        rows = wide.shape[0]
        return (wide[:, :inner].view(rows, self.heads, self.width),
                wide[:, inner: inner + gn].view(rows, self.groups, self.states),
                wide[:, inner + gn: inner + 2 * gn].view(rows, self.groups, self.states))


def _compare(got, ref, bound, what):
    got = got.cpu().double()
    assert torch.isfinite(got).all(), what
    off = (got - ref).abs()
    assert (off <= bound).all(), f"{what}: {(off - bound).max():.3e} over the bound, at most {(off / bound.clamp(min=1e-300)).max():.2f} of it"


def _run_and_check(bl, k, starts, stateful=True, extras=True, softplus=True, slots=None, fresh=None):
    x, b, c = k.views(k.wide)
    gx, gb, gc = k.views(k.wide.cuda())
    d, z, bias = (k.d, k.z, k.dt_bias) if extras else (None, None, None)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    slots = k.slots if slots is None else slots
    fresh = k.fresh if fresh is None else fresh
    out = torch.full((k.rows, k.heads, k.width), 3.0, dtype=k.dtype)
    state = k.state.cuda() if stateful else None
    y = bl.selective_scan(gx, k.dt.cuda(), k.a.cuda(), gb, gc, torch.tensor(starts, dtype=torch.int32).cuda(), d=cu(d),
                          z=cu(z), dt_bias=cu(bias), softplus=softplus, state=state, slots=slots.cuda() if stateful else None,
                          fresh=fresh.cuda() if stateful else None, out=out.cuda())
    ref, ref_state, bound, state_bound = plain.scan(
        x, k.dt, k.a, b, c, starts, d, z, bias, softplus, k.state if stateful else None,
        slots.tolist() if stateful else None, fresh.tolist() if stateful else None, out)
    _compare(y, ref, bound, "y")
    if stateful:
        _compare(state, ref_state, state_bound, "state")


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width", [32, 64, 128])
@pytest.mark.parametrize("states", [16, 32, 64, 128, 256])
def test_every_shape_matches_the_recurrence(bl, dtype, width, states):
    starts = _starts(LENGTHS["edges"], before=2)
    k = Case(dtype, starts[-1] + 3, 2, width, 1, states, 8, width + states)
    _run_and_check(bl, k, starts)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("heads, groups", [(1, 1), (6, 2), (4, 4)])
def test_packed_sequences_and_groups(bl, dtype, lengths, heads, groups):
    lens = LENGTHS[lengths]
    starts = _starts(lens)
    k = Case(dtype, starts[-1], heads, 64, groups, 32, len(lens), 7)
    slots = k.slots.clone()
    if len(lens) > 2:
        slots[1] = -1  # padding: its rows and every place stay as they were
        slots[2] = 1000
    _run_and_check(bl, k, starts, slots=slots)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_one_long_sequence(bl, dtype):
    """Few sequences and heads: the time axis is split and joined."""
    for rows, before in ((700, 0), (1500, 5)):
        k = Case(dtype, rows + before, 1, 64, 1, 64, 1, rows)
        _run_and_check(bl, k, [before, before + rows], fresh=torch.tensor([rows == 700]))


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_without_options(bl, dtype):
    """No state, bias, skip, gate or softplus; steps as they are, all positive."""
    k = Case(dtype, 100, 2, 64, 1, 16, 2, 3)
    k.dt = k.dt.abs() * 0.2
    _run_and_check(bl, k, [0, 37, 100], stateful=False, extras=False, softplus=False)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_rows_without_alignment(bl, dtype):
    """An odd row stride: no row is aligned to more than an element."""
    k = Case(dtype, 150, 2, 32, 2, 16, 2, 4, pad=3)
    _run_and_check(bl, k, [0, 70, 150])


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_far_decays(bl, dtype):
    """Decays from hardly any to a state that is gone within a row, for hundreds of rows."""
    k = Case(dtype, 400, 4, 32, 1, 32, 1, 5)
    k.a = -torch.tensor([1e-4, 0.3, 16.0, 300.0])
    k.dt_bias = torch.tensor([-6.0, 0.0, 1.0, 2.0])
    _run_and_check(bl, k, [0, 400], fresh=torch.tensor([False]))


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_growing_states_and_negative_steps(bl, dtype):
    """Exponents of either sign: states that grow by powers of ten, and steps below zero."""
    k = Case(dtype, 300, 3, 32, 1, 32, 2, 13)
    k.a = torch.tensor([0.3, 2.0, -1.0])
    k.dt_bias = torch.tensor([-2.0, -4.0, -1.0])
    _run_and_check(bl, k, [0, 110, 300])
    k = Case(dtype, 300, 3, 32, 1, 32, 2, 14)
    k.dt = (k.dt.float() * 0.05).to(dtype)
    k.dt_bias = torch.zeros(3)
    _run_and_check(bl, k, [0, 110, 300], softplus=False)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_many_runs_joined(bl, dtype):
    """More runs than the join takes at a time, behind a sequence of one run and before a padded one."""
    k = Case(dtype, 1700, 1, 64, 1, 32, 3, 15)
    k.a = -torch.tensor([0.05])
    slots = k.slots.clone()
    slots[2] = -1
    for fresh in (True, False):
        _run_and_check(bl, k, [0, 40, 1300, 1700], slots=slots, fresh=torch.tensor([fresh] * 3))


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width, states", [(32, 16), (64, 128), (128, 256), (64, 64)])
def test_steps_match_the_recurrence(bl, dtype, width, states):
    rows = 5
    k = Case(dtype, rows, 6, width, 3, states, rows, 6)
    slots = k.slots.clone()
    slots[3] = -5
    x, b, c = k.views(k.wide)
    gx, gb, gc = k.views(k.wide.cuda())
    state, out = k.state.cuda(), torch.full((rows, 6, width), 2.0, dtype=dtype)
    y = bl.selective_scan_step(gx, k.dt.cuda(), k.a.cuda(), gb, gc, state, d=k.d.cuda(), z=k.z.cuda(),
                               dt_bias=k.dt_bias.cuda(), slots=slots.cuda(), out=out.cuda())
    ref, ref_state, bound, state_bound = plain.scan(x, k.dt, k.a, b, c, list(range(rows + 1)), k.d, k.z, k.dt_bias, True,
                                                    k.state, slots.tolist(), None, out)
    _compare(y, ref, bound, "y")
    _compare(state, ref_state, state_bound, "state")


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width,states", [(32, 64), (64, 64), (64, 128), (32, 256), (128, 32), (128, 16)])
def test_many_sequences_of_few_rows(bl, dtype, width, states):
    """Sequences of up to five rows, some of them empty."""
    sequences, heads = 150, 8
    starts = _starts([(7 * j) % 6 for j in range(sequences)], before=2)
    k = Case(dtype, starts[-1] + 3, heads, width, 2, states, sequences, 21)
    _run_and_check(bl, k, starts)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width,states", [(64, 64), (32, 16)])
def test_long_sequences_among_many_short_ones(bl, dtype, width, states):
    """More sequences than scratch has blocks of rows; two of them are split into runs."""
    starts = _starts([1] * 150 + [700] + [0] * 100 + [1, 2] * 20 + [500, 97])
    k = Case(dtype, starts[-1], 4, width, 2, states, len(starts) - 1, 22)
    _run_and_check(bl, k, starts)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_a_step_of_many_sequences(bl, dtype):
    """Enough rows that a workgroup takes several passes over a state's rows."""
    rows, heads, width, states = 70, 8, 64, 128
    k = Case(dtype, rows, heads, width, 2, states, rows, 23)
    x, b, c = k.views(k.wide)
    gx, gb, gc = k.views(k.wide.cuda())
    state = k.state.cuda()
    y = bl.selective_scan_step(gx, k.dt.cuda(), k.a.cuda(), gb, gc, state, d=k.d.cuda(), z=k.z.cuda(),
                               dt_bias=k.dt_bias.cuda(), slots=k.slots.cuda())
    ref, ref_state, bound, state_bound = plain.scan(x, k.dt, k.a, b, c, list(range(rows + 1)), k.d, k.z, k.dt_bias, True,
                                                    k.state, k.slots.tolist(), None, torch.zeros_like(x))
    _compare(y, ref, bound, "y")
    _compare(state, ref_state, state_bound, "state")


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_a_prompt_and_steps_match_one_longer_prompt(bl, dtype):
    rows, more = 90, 6
    k = Case(dtype, rows + more, 4, 64, 1, 128, 1, 8)
    x, b, c = k.views(k.wide)
    gx, gb, gc = k.views(k.wide.cuda())
    ref, ref_state, bound, state_bound = plain.scan(x, k.dt, k.a, b, c, [0, rows + more], k.d, k.z, k.dt_bias, True,
                                                    k.state, [1], [False], torch.zeros_like(x))
    dt, a, d, z, bias, state = (t.cuda() for t in (k.dt, k.a, k.d, k.z, k.dt_bias, k.state))
    one = torch.tensor([1], dtype=torch.int32).cuda()
    y = [bl.selective_scan(gx[:rows], dt[:rows], a, gb[:rows], gc[:rows], torch.tensor([0, rows], dtype=torch.int32).cuda(),
                           d=d, z=z[:rows], dt_bias=bias, state=state, slots=one)]
    for t in range(rows, rows + more):
        s = slice(t, t + 1)
        y.append(bl.selective_scan_step(gx[s], dt[s], a, gb[s], gc[s], state, d=d, z=z[s], dt_bias=bias, slots=one))
    _compare(torch.cat(y), ref, bound, "y")
    _compare(state, ref_state, state_bound, "state")


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_a_number_stays_behind_its_row(bl, dtype, bad):
    """Rows before one that is not a number, other channels and other sequences are as without it."""
    k = Case(dtype, 200, 2, 64, 1, 64, 2, 9)
    x, b, c = k.views(k.wide)
    run = lambda wide: bl.selective_scan(*(k.views(wide)[0], k.dt.cuda(), k.a.cuda()), *k.views(wide)[1:],  # noqa: E731
                                         torch.tensor([0, 120, 200], dtype=torch.int32).cuda(), d=k.d.cuda(), z=k.z.cuda(),
                                         dt_bias=k.dt_bias.cuda())
    sound = run(k.wide.cuda())
    wide = k.wide.cuda()
    wide[75, 64 + 9] = bad  # head 1, channel 9
    got = run(wide)
    ref, _, bound, _ = plain.scan(x, k.dt, k.a, b, c, [0, 120, 200], k.d, k.z, k.dt_bias, True, None, None, None,
                                  torch.zeros_like(x))
    assert not torch.isfinite(got[75:120, 1, 9]).any()
    got[75:120, 1, 9] = sound[75:120, 1, 9]
    _compare(got, ref, bound, "y")


def test_state_offsets_past_32_bits(bl):
    """A cache of more than 2^31 floats, the last place used."""
    heads, width, states = 64, 128, 256
    places = (1 << 31) // (heads * width * states) + 2
    state = torch.zeros(places, heads, width, states, device="cuda")
    k = Case(torch.bfloat16, 3, heads, width, 1, states, 1, 10)
    state[places - 1] = k.state[0].cuda()
    x, b, c = k.views(k.wide)
    gx, gb, gc = k.views(k.wide.cuda())
    place = torch.tensor([places - 1], dtype=torch.int32).cuda()
    y = bl.selective_scan(gx, k.dt.cuda(), k.a.cuda(), gb, gc, torch.tensor([0, 3], dtype=torch.int32).cuda(),
                          dt_bias=k.dt_bias.cuda(), state=state, slots=place)
    ref, ref_state, bound, state_bound = plain.scan(x, k.dt, k.a, b, c, [0, 3], None, None, k.dt_bias, True, k.state[:1],
                                                    None, None, torch.zeros_like(x))
    _compare(y, ref, bound, "y")
    _compare(state[places - 1], ref_state[0], state_bound[0], "state")
    assert not state[: places - 1].any()


def test_starts_outside_the_rows_are_clamped(bl):
    k = Case(torch.float32, 90, 2, 32, 1, 32, 4, 11)
    slots = torch.arange(4, dtype=torch.int32)
    _run_and_check(bl, k, [-9, 40, 40, 1000, 2 ** 31 - 1], slots=slots)


def test_captured_graph_stream_and_repeated_calls(bl):
    """Replays continue the state as eager calls do, bit for bit; so does a call on another stream."""
    k = Case(torch.bfloat16, 600, 2, 64, 1, 128, 1, 12)
    gx, gb, gc = k.views(k.wide.cuda())
    starts = torch.tensor([0, 600], dtype=torch.int32).cuda()
    dt, a, d, z, bias = (t.cuda() for t in (k.dt, k.a, k.d, k.z, k.dt_bias))
    run = lambda state, **kw: bl.selective_scan(gx, dt, a, gb, gc, starts, d=d, z=z, dt_bias=bias, state=state, **kw)  # noqa: E731
    eager = k.state.cuda()
    expect = [run(eager) for _ in range(4)]
    side, state = torch.cuda.Stream(), k.state.cuda()
    torch.cuda.synchronize()
    first = run(state, stream=side)
    side.synchronize()
    assert torch.equal(first, expect[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(state)
    for i in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect[i])
        torch.zeros(1000, device="cuda").sum().item()
    assert torch.equal(state, eager)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("step", [False, True])
def test_gates_of_any_value(bl, dtype, step):
    """y = d x = 1 before the gate: z * sigmoid(z) itself."""
    from tests.test_gpu_sequence_conv import GATE_VALUES, _check_gate
    v = torch.tensor(GATE_VALUES).to(dtype)
    rows = v.shape[0]
    one = lambda *s: torch.ones(*s, dtype=dtype, device="cuda")  # noqa: E731
    z = v[:, None, None].repeat(1, 2, 32).contiguous()
    b, a, d = torch.zeros(rows, 1, 16, dtype=dtype, device="cuda"), -torch.ones(2, device="cuda"), torch.ones(2, device="cuda")
    if step:
        y = bl.selective_scan_step(one(rows, 2, 32), one(rows, 2), a, b, b, torch.zeros(rows, 2, 32, 16, device="cuda"), d=d,
                                   z=z.cuda())
    else:
        y = bl.selective_scan(one(rows, 2, 32), one(rows, 2), a, b, b, torch.tensor([0, rows], dtype=torch.int32).cuda(), d=d,
                              z=z.cuda())
    _check_gate(y, z)


@pytest.mark.parametrize("packed", [False, True])
def test_steps_are_as_exact_as_float32_holds(bl, packed):
    """S = D for x = b = 1 and a zero state: log(1 + e^v) itself. The exponential (1 ulp, 2 half steps, and its carried
    remainder), the quotient and the last two operations round by 6 half steps of it together."""
    heads = 4096
    v = torch.linspace(-24.0, 24.0, heads) + 0.011 * torch.randn(heads, generator=torch.Generator().manual_seed(64))
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    x, b, state = one(1, heads, 32), one(1, 1, 16), torch.zeros(1, heads, 32, 16, device="cuda")
    args = (x, torch.zeros(1, heads, device="cuda"), torch.zeros(heads, device="cuda"), b, b)
    if packed:
        bl.selective_scan(*args, torch.tensor([0, 1], dtype=torch.int32).cuda(), dt_bias=v.cuda(), state=state)
    else:
        bl.selective_scan_step(*args, state, dt_bias=v.cuda())
    got = state.cpu().double()[0, :, 0, 0]
    expect = torch.nn.functional.softplus(v.double(), threshold=1000)
    off = (got - expect).abs() / expect
    assert (off <= 6 * plain.U32).all(), (off.max(), v[off.argmax()])


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_decays_of_many_chunks(bl, dtype):
    """A state that nothing is added to, over 256 chunks of one run: S exp(8192 D a). Each chunk's exponent comes
    from 64 bits; the state is multiplied by a power of two at most three times, of an exponent of at most 20 a
    time: an exponential of 1 ulp, what its argument's rounding left and the product, 5 half steps of float32."""
    heads, states, sequences, length = 64, 16, 32, 8192
    rest = length // 2 * sequences + 32 - length
    starts = _starts([length] + [rest // (sequences - 1)] * (sequences - 1))
    rows = starts[-1]
    g = torch.Generator().manual_seed(63)
    a = -(torch.rand(heads, generator=g) * 0.06 + 0.012)
    zeros = lambda *s: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    bc = zeros(rows, heads, states).fill_(1.0)
    state = torch.randn(sequences, heads, 32, states, generator=g)
    got = state.cuda()
    bl.selective_scan(zeros(rows, heads, 32), zeros(rows, heads).fill_(2.0 ** -5), a.cuda(), bc, bc,
                      torch.tensor(starts, dtype=torch.int32).cuda(), softplus=False, state=got)
    for j in range(sequences):
        expect = state[j].double() * torch.exp((starts[j + 1] - starts[j]) * 2.0 ** -5 * a.double())[:, None, None]
        off = (got[j].cpu().double() - expect).abs() / expect.abs()
        assert (off <= 15 * plain.U32).all(), (j, off.max())


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("states", [16, 32, 64, 128, 256])
def test_states_and_weights_are_read_whole(bl, dtype, states):
    """Outputs that are small beside their two terms, so that what a product leaves out of the state or of a
    chunk's weights shows: two states of a channel that c weighs against each other, and two rows of x of opposite
    sign under nearly equal weights. All other terms are exactly zero. Each term rounds a decay (its exponential of
    1 ulp and a product), a step, a weight and what three parts leave, at most 8 half steps of float32, and the sum
    rounds once for each of a term's up to 5 products: 18 of both terms. What both terms share, sums over all states
    among it, rounds y itself."""
    rows, heads, width = 40, 2, 64
    g = torch.Generator().manual_seed(65)
    a = -torch.tensor([1e-5, 1e-4])
    dt, b = torch.ones(rows, heads).to(dtype), (0.5 + torch.rand(1, 1, states, generator=g)).to(dtype).repeat(rows, 1, 1)
    c = (0.5 + torch.rand(1, 1, states, generator=g)).to(dtype).repeat(rows, 1, 1)
    starts = torch.tensor([0, rows], dtype=torch.int32).cuda()
    decay = torch.exp((torch.arange(rows) + 1.0).double()[:, None] * a.double())  # of the first state, up to each row
    cd, none, nothing = c[0, 0].double(), torch.zeros(1, heads, width, states), torch.zeros(rows, heads, width)

    def check(x, state, expect, weight):
        y = bl.selective_scan(x.to(dtype).cuda(), dt.cuda(), a.cuda(), b.cuda(), c.cuda(), starts, softplus=False, state=state.cuda())
        error = 18 * plain.U32 * weight + (3 * states + 40) * plain.U32 * expect.abs()
        _compare(y, expect, plain.rounded(expect, error, dtype), "y")

    # two states of each channel
    first, second = torch.randint(0, states // 2, (2, heads, width), generator=g)
    second = second + states // 2
    value = torch.randn(heads, width, generator=g)
    other = (-value.double() * cd[first] / cd[second]).float()
    state = none.clone()
    state[0].scatter_(2, first[..., None], value[..., None])
    state[0].scatter_(2, second[..., None], other[..., None])
    pair = value.double() * cd[first], other.double() * cd[second]
    check(nothing, state, decay[:, :, None] * (pair[0] + pair[1]), decay[:, :, None] * (pair[0].abs() + pair[1].abs()))
    # two rows of x, in one chunk or in two
    dot = (b[0, 0].double() * cd).sum()
    for at in ((0, 1), (3, 29), (14, 17), (1, 39)):
        x = nothing.clone()
        x[at[0]] = (0.5 + torch.rand(heads, width, generator=g)).to(dtype).float()
        x[at[1]] = -x[at[0]]
        terms = torch.zeros(2, rows, heads, width, dtype=torch.float64)
        for k in range(2):
            since = torch.arange(rows).double() - at[k]
            reach = torch.where(since[:, None] >= 0, torch.exp(since.clamp(min=0)[:, None] * a.double()), 0.0)
            terms[k] = reach[:, :, None] * x[at[k]].double() * dot
        check(x, none, terms.sum(0), terms.abs().sum(0))


class Long(Case):
    """Many groups of one head each, so that few channels make many workgroups: long runs of rows."""

    def __init__(self, dtype, rows, heads, states, sequences, seed):
        super().__init__(dtype, rows, heads, 32, heads, states, sequences, seed)

    def run(self, bl, starts):
        gx, gb, gc = self.views(self.wide.cuda())
        state = self.state.cuda()
        y = bl.selective_scan(gx, self.dt.cuda(), self.a.cuda(), gb, gc, torch.tensor(starts, dtype=torch.int32).cuda(),
                              d=self.d.cuda(), z=self.z.cuda(), dt_bias=self.dt_bias.cuda(), state=state,
                              slots=self.slots.cuda(), fresh=self.fresh.cuda())
        return y.cpu(), state.cpu()

    def check(self, got, starts, heads, sequences):
        """Some heads of some sequences: they know nothing of each other."""
        y, state = got
        x, b, c = self.views(self.wide)
        for j in sequences:
            at, place = slice(starts[j], starts[j + 1]), int(self.slots[j])
            part = lambda t: t[at][:, heads]  # noqa: E731
            ref, ref_state, bound, state_bound = plain.scan(
                part(x), part(self.dt), self.a[heads], part(b), part(c), [0, starts[j + 1] - starts[j]], self.d[heads],
                part(self.z), self.dt_bias[heads], True, self.state[place: place + 1, heads], None, [bool(self.fresh[j])],
                torch.zeros_like(part(x)), whole_parts=True)
            _compare(part(y), ref, bound, f"y of sequence {j}")
            _compare(state[place: place + 1, heads], ref_state, state_bound, f"state of sequence {j}")


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("states", [16, 128])
def test_long_runs(bl, dtype, states):
    """One sequence in 17 runs of 23 chunks: slow, ordinary and fast decays, settled never, now and then and always."""
    k = Long(dtype, 12300, 32, states, 1, 61)
    k.a[:3] = -torch.tensor([0.02, 0.6, 12.0])
    k.check(k.run(bl, [0, 12300]), [0, 12300], [0, 1, 2, 31], [0])


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("states", [16, 64])
def test_many_long_sequences_stay_whole(bl, dtype, states):
    """Four times as many workgroups as there is room for: sequences of up to twice the mean are not split (29
    chunks in one run), one of more is."""
    lengths = [900, 40, 0, 1, 2100, 33] + [437 + 3 * j for j in range(58)]
    starts = _starts(lengths)
    k = Long(dtype, starts[-1], 32, states, len(lengths), 62)
    assert 900 < 2 * starts[-1] // len(lengths) < 2100 and len(lengths) * 32 >= 2048
    k.a[:3] = -torch.tensor([0.02, 0.6, 12.0])
    k.check(k.run(bl, starts), starts, [0, 1, 2, 31], [0, 1, 3, 4, 5, len(lengths) - 1])


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("name", ["dt", "b", "c", "z"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_other_inputs_that_are_not_numbers_reach(bl, dtype, name, bad):
    """dt: its head from its row on; b: its group from its row on; c: its group's row; z: its element. Everything
    before, beside and behind, in other sequences too, is as without it; split and whole sequences, and states."""
    starts = [0, 30, 230, 260]
    k = Case(dtype, 260, 4, 64, 2, 64, 3, 66)
    k.fresh[:] = False
    row = 75
    x, b, c = k.views(k.wide)
    ref, ref_state, bound, state_bound = plain.scan(x, k.dt, k.a, b, c, starts, k.d, k.z, k.dt_bias, True, k.state,
                                                    k.slots.tolist(), None, torch.zeros_like(x))
    wide, dt, z, state = k.wide.clone(), k.dt.clone(), k.z.clone(), k.state.cuda()
    hit, hit_state = torch.zeros(260, 4, 64, dtype=torch.bool), torch.zeros(4, 64, 64, dtype=torch.bool)
    if name == "dt":
        dt[row, 1] = abs(bad)  # minus infinity would be a step of zero
        hit[row:230, 1], hit_state[1] = True, True
    elif name == "b":
        k.views(wide)[1][row, 1, 5] = bad
        hit[row:230, 2:], hit_state[2:, :, 5] = True, True
    elif name == "c":
        k.views(wide)[2][row, 0, 7] = bad
        hit[row, :2] = True
    else:
        z[row, 3, 11] = bad
        hit[row, 3, 11] = True
    gx, gb, gc = k.views(wide.cuda())
    y = bl.selective_scan(gx, dt.cuda(), k.a.cuda(), gb, gc, torch.tensor(starts, dtype=torch.int32).cuda(), d=k.d.cuda(),
                          z=z.cuda(), dt_bias=k.dt_bias.cuda(), state=state, slots=k.slots.cuda())
    y, state = y.cpu().double(), state.cpu().double()
    assert not torch.isfinite(y[hit]).any()
    off = (y - ref).abs()[~hit]
    assert (off <= bound[~hit]).all(), (off - bound[~hit]).max()
    place = int(k.slots[1])
    assert not torch.isfinite(state[place][hit_state]).any()
    rest = torch.ones(state.shape, dtype=torch.bool)
    rest[place] = ~hit_state
    off = (state - ref_state).abs()[rest]
    assert (off <= state_bound[rest]).all()

"""The causal sequence operators as one layer after the stack: norm, convolution, scan, norm, heads and
log probabilities, for packed windows and then row by row. Every operator is checked against its 64-bit
definition on the inputs it got."""

import pytest
import torch

import workloads
from tests import sequence_plain as plain

pytestmark = pytest.mark.gpu

HEADS, WIDTH, STATES, TAPS = 4, 64, 32, 4
INNER, CHANNELS = HEADS * WIDTH, HEADS * WIDTH + 2 * STATES


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _within(got, ref, bound, what):
    off = (got.cpu().double() - ref).abs()
    assert torch.isfinite(off).all() and (off <= bound).all(), f"{what}: {(off - bound).max():.3e} over the bound"


class Layer:
    """Weights of one layer and, per cache place, its convolution rows and states."""

    def __init__(self, seed, places):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).cuda()  # noqa: E731
        self.norm_in, self.norm_out = r(256).abs() + 0.5, r(INNER).abs() + 0.5
        self.into = r(256, INNER + CHANNELS + HEADS, scale=1 / 16)
        self.out = r(INNER, 256, scale=1 / 16)
        self.conv, self.conv_bias = r(CHANNELS, TAPS, scale=0.5), r(CHANNELS, scale=0.1)
        self.a, self.d, self.dt_bias = -r(HEADS).abs() - 0.5, r(HEADS), r(HEADS) - 3
        self.rows = torch.zeros(places, TAPS - 1, CHANNELS, device="cuda")
        self.states = torch.zeros(places, HEADS, WIDTH, STATES, device="cuda")

    def __call__(self, bl, x, residual, starts, slots, fresh=None):
        """Returns the outputs of every operator; `starts` None: one row a sequence."""
        first = bl.add_rms_norm(x, self.norm_in, residual=residual)
        mixed = first.y @ self.into
        z, xbc, dt = mixed[:, :INNER], mixed[:, INNER: INNER + CHANNELS], mixed[:, INNER + CHANNELS:]
        if starts is None:
            conv = bl.causal_conv_step(xbc, self.conv, self.rows, bias=self.conv_bias, slots=slots)
        else:
            conv = bl.causal_conv(xbc, self.conv, starts, bias=self.conv_bias, state=self.rows, slots=slots, fresh=fresh)
        n = conv.shape[0]
        xs = conv[:, :INNER].view(n, HEADS, WIDTH)
        b, c = conv[:, INNER: INNER + STATES].view(n, 1, STATES), conv[:, INNER + STATES:].view(n, 1, STATES)
        gate = z.view(n, HEADS, WIDTH)
        if starts is None:
            y = bl.selective_scan_step(xs, dt, self.a, b, c, self.states, d=self.d, z=gate, dt_bias=self.dt_bias, slots=slots)
        else:
            y = bl.selective_scan(xs, dt, self.a, b, c, starts, d=self.d, z=gate, dt_bias=self.dt_bias, state=self.states,
                                  slots=slots, fresh=fresh)
        last = bl.add_rms_norm(y.reshape(n, INNER) @ self.out, self.norm_out, residual=first.residual, eight_bit="e4m3", keep_y=True)
        return {"first": first, "xbc": xbc, "dt": dt, "conv": conv, "x": xs, "b": b, "c": c, "gate": gate, "y": y, "last": last}


def _check(layer, x, residual, starts, slots, fresh, rows_before, states_before, got):
    cpu = lambda t: t.cpu()  # noqa: E731
    y, s, error = plain.norm(cpu(x), cpu(layer.norm_in), 1e-5, cpu(residual))
    _within(got["first"].y, y, plain.rounded(y, error, torch.float32), "first norm")
    slots, fresh = slots.tolist(), None if fresh is None else fresh.tolist()
    ref, state, bound = plain.conv(cpu(got["xbc"]), cpu(layer.conv), starts, cpu(layer.conv_bias), rows_before, slots, fresh,
                                   True, torch.zeros(got["conv"].shape))
    _within(got["conv"], ref, bound, "convolution")
    assert torch.equal(layer.rows.cpu().double(), state)
    ref, state, bound, state_bound = plain.scan(
        cpu(got["x"]), cpu(got["dt"]), cpu(layer.a), cpu(got["b"]), cpu(got["c"]), starts, cpu(layer.d), cpu(got["gate"]),
        cpu(layer.dt_bias), True, states_before, slots, fresh, torch.zeros(got["y"].shape))
    _within(got["y"], ref, bound, "scan")
    _within(layer.states, state, state_bound, "states")


def test_packed_windows_then_single_rows(bl):
    windows, steps, more = 3, 47, 4
    plan = bl.Plan(workloads.make_layers(31), windows, steps)
    stack = plan.forward(torch.from_numpy(workloads.make_input(32, windows, steps)).cuda()).view(-1, 256)
    plan.check()
    heads = bl.Heads(workloads.make_heads(33))
    layer = Layer(34, places=5)
    g = torch.Generator().manual_seed(35)
    residual = torch.randn(windows * steps, 256, generator=g).cuda()
    starts = [j * steps for j in range(windows + 1)]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32)
    fresh = torch.tensor([True, True, False])
    rows, states = layer.rows.cpu(), layer.states.cpu()
    got = layer(bl, stack, residual, torch.tensor(starts, dtype=torch.int32).cuda(), slots.cuda(), fresh.cuda())
    _check(layer, stack, residual, starts, slots, fresh, rows, states, got)
    scores = heads.forward(got["last"].y)
    labels = torch.randint(0, 7, (windows * steps, 1), generator=g)
    answer = bl.token_logprobs(scores, labels.cuda(), top=3)
    (given, entropy, order, top_lp), (gb, eb, tb) = plain.logprobs(scores.cpu(), labels, 3)
    _within(answer.logprobs, given, gb, "log probabilities")
    _within(answer.entropy, entropy, eb, "entropy")
    assert torch.equal(answer.top_tokens.cpu(), order)
    _within(answer.top_logprobs, top_lp, tb, "top log probabilities")
    for k in range(more):
        x, r = torch.randn(windows, 256, generator=g).cuda(), torch.randn(windows, 256, generator=g).cuda()
        rows, states = layer.rows.cpu(), layer.states.cpu()
        got = layer(bl, x, r, None, slots.cuda())
        _check(layer, x, r, list(range(windows + 1)), slots, None, rows, states, got)


def test_single_rows_captured_once_and_replayed(bl):
    """A captured step of the whole layer continues its states from replay to replay as eager steps do."""
    places, replays = 3, 5
    g = torch.Generator().manual_seed(41)
    inputs = [torch.randn(places, 256, generator=g).cuda() for _ in range(replays)]
    slots = torch.tensor([2, 0, 1], dtype=torch.int32).cuda()
    eager, captured = Layer(42, places), Layer(42, places)
    residual = torch.randn(places, 256, generator=g).cuda()
    ids = torch.tensor([3, 0, 250]).cuda()
    x = inputs[0].clone()

    def step(layer, x):
        out = layer(bl, x, residual, None, slots)["last"]
        return out.y, bl.token_logprobs(out.y, ids, top=4)

    expect = [step(eager, v) for v in inputs]
    scratch = Layer(42, places)
    step(scratch, x)  # libraries' first calls stay out of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, answer = step(captured, x)
    for v, (ey, ea) in zip(inputs, expect):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ey)
        for a, b in zip(answer, ea):
            assert torch.equal(a, b)
    assert torch.equal(captured.states, eager.states) and torch.equal(captured.rows, eager.rows)


def test_two_calls_at_once_on_two_streams(bl):
    """Layers of their own on two streams, many calls in flight, against the same calls one by one."""
    g = torch.Generator().manual_seed(51)
    rows = 600
    x, r = torch.randn(rows, 256, generator=g).cuda(), torch.randn(rows, 256, generator=g).cuda()
    starts = torch.tensor([0, rows], dtype=torch.int32).cuda()
    slots = torch.zeros(1, dtype=torch.int32).cuda()
    alone = [Layer(52, 1), Layer(53, 1)]
    expect = [[layer(bl, x, r, starts, slots)["last"].y for _ in range(4)] for layer in alone]
    both, streams, got = [Layer(52, 1), Layer(53, 1)], [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    torch.cuda.synchronize()
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(both[k](bl, x, r, starts, slots)["last"].y)
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(got[k], expect[k]):
            assert torch.equal(a, b)
        assert torch.equal(both[k].states, alone[k].states)

"""A decoder's layer over the stack's frames: keys and values by a product over the frames, then norm, query product,
cross attention, output product with the residual, norm to 8 bits and a feed-forward pair, for packed prompts and row
by row. Every operator is checked against its 64-bit definition on the inputs it got."""

import pytest
import torch

import workloads
from tests import decoder_plain as plain
from tests import sequence_plain

pytestmark = pytest.mark.gpu

HEADS, KEY_HEADS, WIDTH, MODEL, INNER = 4, 2, 64, 256, 512


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _within(got, ref, bound, what):
    off = (got.cpu().double() - ref).abs()
    assert torch.isfinite(off).all() and (off <= bound).all(), f"{what}: {(off - bound).max():.3e} over the bound"


class Layer:
    def __init__(self, seed, dtype):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, scale=1 / 16: (torch.randn(*s, generator=g) * scale).to(dtype).cuda()  # noqa: E731
        self.dtype = dtype
        self.kv = r(2 * KEY_HEADS * WIDTH, MODEL)
        self.q, self.q_bias = r(HEADS * WIDTH, MODEL), r(HEADS * WIDTH)
        self.out, self.out_bias = r(MODEL, HEADS * WIDTH), r(MODEL)
        self.norms = [r(MODEL, scale=1).abs() + 0.5 for _ in range(2)]
        up, down = torch.randn(INNER, MODEL, generator=g) / 16, torch.randn(MODEL, INNER, generator=g) / 22
        self.up_scales = (up.abs().amax(1) / 448).cuda()
        self.up = (up.cuda() / self.up_scales[:, None]).to(torch.float8_e4m3fn)
        self.up_bias, self.down = r(INNER), down.to(dtype).cuda()

    def memory(self, bl, frames):
        kv = bl.linear(frames.to(self.dtype), self.kv)
        n = KEY_HEADS * WIDTH
        return kv, kv[:, :n].view(-1, KEY_HEADS, WIDTH), kv[:, n:].view(-1, KEY_HEADS, WIDTH)

    def __call__(self, bl, x, k, v, starts, memory_starts, lengths, slots, stream=None):
        """Outputs of every operator; `starts` None: one row a sequence."""
        first = bl.add_rms_norm(x, self.norms[0], stream=stream).y
        q = bl.linear(first, self.q, bias=self.q_bias, stream=stream).view(-1, HEADS, WIDTH)
        if starts is None:
            mix = bl.cross_attention_step(q, k, v, memory_starts, memory_lengths=lengths, slots=slots, stream=stream)
        else:
            mix = bl.cross_attention(q, k, v, starts, memory_starts, memory_lengths=lengths, slots=slots, stream=stream)
        out = bl.linear(mix.view(-1, HEADS * WIDTH), self.out, bias=self.out_bias, residual=x, stream=stream)
        second = bl.add_rms_norm(out, self.norms[1], eight_bit="e4m3", stream=stream)
        up = bl.linear(second.q, self.up, bias=self.up_bias, activation="gelu", x_scales=second.scales,
                       weight_scales=self.up_scales, out_type=self.dtype, stream=stream)
        down = bl.linear(up, self.down, residual=out, stream=stream)
        return {"first": first, "q": q, "mix": mix, "out": out, "second": second, "up": up, "down": down}


def _check(layer, x, k, v, starts, memory_starts, lengths, slots, got):
    cpu = lambda t: t.cpu()  # noqa: E731
    dtype = layer.dtype
    q, bound = plain.linear(cpu(got["first"]), cpu(layer.q), cpu(layer.q_bias), None, None, None, None, 0, dtype)
    _within(got["q"].reshape(q.shape), q, bound, "query")
    mix, bound = plain.attention(cpu(got["q"]), cpu(k), cpu(v), starts, memory_starts, lengths, slots, None, WIDTH ** -0.5,
                                 torch.zeros(got["q"].shape))
    _within(got["mix"], mix, bound, "attention")
    flat = cpu(got["mix"]).reshape(-1, HEADS * WIDTH)
    out, bound = plain.linear(flat, cpu(layer.out), cpu(layer.out_bias), None, cpu(x), None, None, 0, dtype)
    _within(got["out"], out, bound, "output")
    up, bound = plain.linear(cpu(got["second"].q), cpu(layer.up), cpu(layer.up_bias), "gelu", None, cpu(got["second"].scales),
                             cpu(layer.up_scales), 0, dtype)
    _within(got["up"], up, bound, "up")
    down, bound = plain.linear(cpu(got["up"]), cpu(layer.down), None, None, cpu(got["out"]), None, None, 0, dtype)
    _within(got["down"], down, bound, "down")


@pytest.mark.parametrize("dtype", sequence_plain.TYPES, ids=str)
def test_prompts_and_single_rows_over_the_stacks_frames(bl, dtype):
    windows, steps = 3, 57
    plan = bl.Plan(workloads.make_layers(61), windows, steps)
    frames = plan.forward(torch.from_numpy(workloads.make_input(62, windows, steps)).cuda()).view(-1, 256)
    plan.check()
    layer = Layer(63, dtype)
    kv, k, v = layer.memory(bl, frames)
    ref, bound = plain.linear(frames.to(dtype).cpu(), layer.kv.cpu(), None, None, None, None, None, 0, dtype)
    _within(kv, ref, bound, "keys and values")
    g = torch.Generator().manual_seed(64)
    memory_starts, lengths = [j * steps for j in range(windows + 1)], [57, 20, 41]
    whole = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    starts, slots = [0, 30, 30, 101, 140], [2, 0, 1, 0]
    x = torch.randn(140, MODEL, generator=g).to(dtype).cuda()
    got = layer(bl, x, k, v, whole(starts), whole(memory_starts), whole(lengths), whole(slots))
    _check(layer, x, k, v, starts, memory_starts, lengths, slots, got)
    for rows in (3, 40):
        slots = [(5 * i) % 3 for i in range(rows)]
        x = torch.randn(rows, MODEL, generator=g).to(dtype).cuda()
        got = layer(bl, x, k, v, None, whole(memory_starts), whole(lengths), whole(slots))
        _check(layer, x, k, v, None, memory_starts, lengths, slots, got)


def _inputs(dtype, rows, frames, seed, places=2):
    g = torch.Generator().manual_seed(seed)
    whole = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    memory = torch.randn(places * frames, MODEL, generator=g).cuda()
    return (torch.randn(rows, MODEL, generator=g).to(dtype).cuda(), memory, whole([j * frames for j in range(places + 1)]),
            whole([frames - 3 * j for j in range(places)]))


@pytest.mark.parametrize("step", [True, False])
def test_captured_once_and_replayed(bl, step):
    """Every replay, on rows, lengths and memories of its own, gives the eager call's bits; long memories, so that
    frames are split and joined within the graph."""
    dtype, rows, replays = torch.bfloat16, 2 if step else 70, 4
    layer = Layer(71, dtype)
    sets = [_inputs(dtype, rows, 3000, 72 + i) for i in range(replays)]
    whole = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    starts = None if step else whole([0, 65, 70])
    x, memory, memory_starts, lengths = (t.clone() for t in sets[0])
    slots = whole([1, 0])

    def run(x, memory, lengths):
        _, k, v = layer.memory(bl, memory)
        return layer(bl, x, k, v, starts, memory_starts, lengths, slots)["down"]

    expect = []
    for i, (xi, mi, _, li) in enumerate(sets):
        expect.append(run(xi, mi, li - 100 * i))
    run(x, memory, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(x, memory, lengths)
    for i, (xi, mi, _, li) in enumerate(sets):
        x.copy_(xi), memory.copy_(mi), lengths.copy_(li - 100 * i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect[i])
        run(xi, mi, li)  # eager work between the replays
        torch.cuda.synchronize()


def test_two_calls_at_once_on_two_streams(bl):
    layers = [Layer(81, torch.float16), Layer(82, torch.float16)]
    sets = [_inputs(torch.float16, 300, 2500, 83 + i) for i in range(2)]
    whole = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    starts = whole([0, 120, 300])
    memories = [layer.memory(bl, s[1]) for layer, s in zip(layers, sets)]

    def run(i, stream=None):
        x, _, memory_starts, lengths = sets[i]
        return layers[i](bl, x, memories[i][1], memories[i][2], starts, memory_starts, lengths, None, stream)["down"]

    expect = [run(i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            got[i].append(run(i, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, expect[i])


def test_two_calls_at_once_share_no_scratch(bl):
    """The same split calls on two streams at once, their scratch from the allocator of each stream."""
    g = torch.Generator().manual_seed(91)
    x, w = torch.randn(4, 16384, generator=g).cuda(), torch.randn(64, 16384, generator=g).cuda()
    expect = bl.linear(x, w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [bl.linear(x, w, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y, expect) for y in got)


def test_refuses_gradients(bl):
    x = torch.ones(3, 8, device="cuda", requires_grad=True)
    w = torch.ones(4, 8, device="cuda")
    with pytest.raises(TypeError, match="gradient"):
        bl.linear(x, w)
    with pytest.raises(TypeError, match="gradient"):
        bl.linear(w, x)
    q = torch.ones(3, 1, 8, device="cuda", requires_grad=True)
    whole = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="gradient"):
        bl.cross_attention(q, q, q, whole, whole)
    with torch.no_grad():
        assert bl.linear(x, w).shape == (3, 4)
        assert bl.cross_attention(q, q, q, whole, whole).shape == q.shape


def test_binding_refuses_what_does_not_fit(bl):
    x, w = torch.ones(3, 8, device="cuda"), torch.ones(4, 8, device="cuda")
    code, one = torch.ones(3, 8, device="cuda").to(torch.int8), torch.ones(3, device="cuda")
    for call, error in ((lambda: bl.linear(x, w.half()), TypeError), (lambda: bl.linear(x, w[:, :7]), ValueError),
                        (lambda: bl.linear(x, w, activation="tanh"), ValueError),
                        (lambda: bl.linear(x, w, out_type=torch.float16), TypeError),
                        (lambda: bl.linear(x, w, x_scales=one), ValueError),
                        (lambda: bl.linear(code, w, x_scales=one, weight_scales=one), TypeError),
                        (lambda: bl.linear(code, code, weight_scales=one), bl.BilstmError),
                        (lambda: bl.linear(x.t(), w[:, :3]), ValueError),
                        (lambda: bl.linear(x, w, bias=torch.ones(5, device="cuda")), ValueError),
                        (lambda: bl.linear(x, w, slope=float("nan")), bl.BilstmError),
                        (lambda: bl.linear(x, w, out=x), ValueError),
                        (lambda: bl.linear(x, torch.ones(8, 8, device="cuda"), out=x), bl.BilstmError)):
        with pytest.raises(error):
            call()
    q, k = torch.ones(3, 4, 8, device="cuda"), torch.ones(5, 2, 8, device="cuda")
    starts, memory = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 3], [0, 5]))
    for call, error in ((lambda: bl.cross_attention(q, k, k[:4], starts, memory), ValueError),
                        (lambda: bl.cross_attention(q, k[:, :, :7], k, starts, memory), ValueError),
                        (lambda: bl.cross_attention(q, k.half(), k.half(), starts, memory), TypeError),
                        (lambda: bl.cross_attention(q[:, :3], k, k, starts, memory), bl.BilstmError),
                        (lambda: bl.cross_attention(q, k, k, starts.long(), memory), TypeError),
                        (lambda: bl.cross_attention(q, k, k, starts, memory, scale=-1.0), bl.BilstmError),
                        (lambda: bl.cross_attention(q, k, k, starts, memory, mask=torch.ones(4, device="cuda").bool()), ValueError),
                        (lambda: bl.cross_attention(q, k, k, starts, memory, mask=torch.ones(5, device="cuda")), TypeError),
                        (lambda: bl.cross_attention(q, k, k, starts, memory, out=q), bl.BilstmError),
                        (lambda: bl.cross_attention_step(q, k, k, memory), bl.BilstmError),
                        (lambda: bl.cross_attention(q, k, k, starts, memory[:0]), ValueError)):
        with pytest.raises(error):
            call()

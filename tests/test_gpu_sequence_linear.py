"""The matrix product with bias, activation and residual, against 64 bits."""

import pytest
import torch

from tests import decoder_plain as plain
from tests.sequence_plain import TYPES

pytestmark = pytest.mark.gpu

EIGHT = list(plain.EIGHT)
ACTIVATIONS = [None, "relu", "leaky_relu", "gelu", "silu"]


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _make(dtype, rows, inputs, outputs, seed, out_type=None):
    """x, weight, bias, residual and the scales of 8-bit rows, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w = r(rows, inputs), r(outputs, inputs) / inputs ** 0.5
    y = out_type or dtype
    bias, residual = r(outputs).to(y), (r(rows, outputs) * 2).to(y)
    if dtype not in plain.EIGHT:
        return x.to(dtype), w.to(dtype), bias, residual, None, None
    top, scales, codes = plain.EIGHT[dtype], [], []
    for t in (x, w):
        scale = t.abs().amax(1) / top
        q = (t / scale[:, None]).clamp(-top, top)
        codes.append(torch.round(q).to(dtype) if dtype == torch.int8 else q.to(dtype))
        scales.append(scale)
    return codes[0], codes[1], bias, residual, scales[0], scales[1]


def _same(got, value, bound):
    off = (got.cpu().double() - value).abs()
    assert torch.isfinite(off).all() and (off <= bound).all(), f"{(off - bound).max():.3e} over the bound"


def _check(bl, x, w, bias, residual, xs, ws, kind=None, slope=0.01, out_type=None, **more):
    to = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = out_type or (x.dtype if xs is None else torch.bfloat16)
    got = bl.linear(to(x), to(w), bias=to(bias), activation=kind, residual=to(residual), x_scales=to(xs), weight_scales=to(ws),
                    slope=slope, out_type=out_type, **more)
    assert got.dtype == y
    _same(got, *plain.linear(x, w, bias, kind, residual, xs, ws, slope, y))
    return got


@pytest.mark.parametrize("dtype", TYPES + EIGHT, ids=str)
@pytest.mark.parametrize("rows", [1, 2, 3, 15, 16, 17, 33, 63, 64, 65, 129, 300])
@pytest.mark.parametrize("inputs, outputs", [(1, 1), (8, 5), (16, 16), (77, 130), (128, 64), (256, 257), (600, 40)])
def test_sizes(bl, dtype, rows, inputs, outputs):
    x, w, bias, residual, xs, ws = _make(dtype, rows, inputs, outputs, rows + inputs, torch.bfloat16 if dtype in EIGHT else None)
    _check(bl, x, w, bias, residual, xs, ws)


@pytest.mark.parametrize("dtype", TYPES + EIGHT, ids=str)
@pytest.mark.parametrize("rows, inputs, outputs", [(2100, 320, 2050), (1111, 777, 999), (4096, 64, 4096), (700, 1000, 1300), (4200, 72, 4200),
                                                   (6000, 40, 2600)])
def test_many_rows(bl, dtype, rows, inputs, outputs):
    x, w, bias, residual, xs, ws = _make(dtype, rows, inputs, outputs, 3, torch.bfloat16 if dtype in EIGHT else None)
    _check(bl, x, w, bias, residual, xs, ws)


@pytest.mark.parametrize("dtype", TYPES + EIGHT, ids=str)
@pytest.mark.parametrize("rows", [1, 7, 40, 200])
@pytest.mark.parametrize("inputs, outputs", [(8192, 24), (5120, 200), (4097, 33)])
def test_long_sums(bl, dtype, rows, inputs, outputs):
    x, w, bias, residual, xs, ws = _make(dtype, rows, inputs, outputs, 4, torch.bfloat16 if dtype in EIGHT else None)
    _check(bl, x, w, bias, residual, xs, ws)


@pytest.mark.parametrize("out_type", TYPES, ids=str)
@pytest.mark.parametrize("dtype", TYPES + EIGHT, ids=str)
@pytest.mark.parametrize("kind", ACTIVATIONS)
@pytest.mark.parametrize("rows", [5, 200])
def test_epilogues(bl, out_type, dtype, kind, rows):
    if dtype not in EIGHT and dtype != out_type:
        pytest.skip("y is of x's type")
    x, w, bias, residual, xs, ws = _make(dtype, rows, 96, 72, 5, out_type)
    for b in (None, bias * 3):
        for r in (None, residual):
            _check(bl, x, w, b, r, xs, ws, kind, out_type=out_type)
    _check(bl, x, w, bias, None, xs, ws, kind, slope=-2.5, out_type=out_type)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_activations_far_out(bl, dtype):
    """Arguments from -100 to 100: tails that vanish, and values that pass through."""
    v = torch.linspace(-100, 100, 4001).to(dtype)
    x, w = v[:, None].contiguous(), torch.ones(1, 1, dtype=dtype)
    for kind in ACTIVATIONS:
        _check(bl, x, w, None, None, None, None, kind)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [3, 150])
def test_infinities_and_not_numbers(bl, dtype, rows):
    """They reach the outputs that the formula says, and no others."""
    x, w, bias, residual, _, _ = _make(dtype, rows, 70, 50, 6)
    clean = bl.linear(x.cuda(), w.cuda(), bias=bias.cuda())
    x[1, 3], x[2, 69] = float("nan"), float("inf")
    got = bl.linear(x.cuda(), w.cuda(), bias=bias.cuda())
    assert torch.isnan(got[1]).all()
    assert torch.equal(got[2].cpu().float(), torch.sign(w[:, 69].float()) * float("inf"))
    assert torch.equal(got[3:], clean[3:]) and torch.equal(got[0], clean[0])
    big = torch.finfo(dtype).max
    x = torch.full((rows, 2), big, dtype=dtype)
    w = torch.tensor([[0.5, 0.0], [0.0, -0.25], [0.0, 0.0]], dtype=dtype)
    got = bl.linear(x.cuda(), w.cuda()).cpu().double()
    assert torch.equal(got, torch.tensor([[big * 0.5, big * -0.25, 0.0]], dtype=torch.float64).expand(rows, 3))


@pytest.mark.parametrize("dtype", TYPES + EIGHT, ids=str)
@pytest.mark.parametrize("rows", [4, 150])
@pytest.mark.parametrize("offset", [0, 1, 3, 16])
def test_strides_and_alignments(bl, dtype, rows, offset):
    inputs, outputs = 96, 80
    y = torch.bfloat16 if dtype in EIGHT else dtype
    x, w, bias, residual, xs, ws = _make(dtype, rows, inputs, outputs, 7, y)

    def inside(t, kind):
        store = torch.zeros(t.shape[0], t.shape[1] + 2 * offset + (4 if offset == 3 else 0), dtype=torch.float32).to(kind).cuda()
        view = store[:, offset: offset + t.shape[1]]
        view.copy_(t)
        return store, view

    _, xv = inside(x, dtype)
    _, wv = inside(w, dtype)
    _, rv = inside(residual, y)
    store, out = inside(torch.zeros(rows, outputs), y)
    store.fill_(9.0)
    got = bl.linear(xv, wv, bias=bias.cuda(), residual=rv, x_scales=None if xs is None else xs.cuda(),
                    weight_scales=None if ws is None else ws.cuda(), out=out)
    assert got is out
    ref = plain.linear(x, w, bias, None, residual, xs, ws, 0.01, y)
    _same(out, *ref)
    rest = torch.ones(store.shape[1], dtype=torch.bool)
    rest[offset: offset + outputs] = False
    assert (store[:, rest.cuda()] == 9).all()
    # in place of the residual
    got = bl.linear(xv, wv, bias=bias.cuda(), residual=rv, x_scales=None if xs is None else xs.cuda(),
                    weight_scales=None if ws is None else ws.cuda(), out=rv)
    _same(got, *ref)


@pytest.mark.parametrize("eight", ["e4m3", "int8"])
@pytest.mark.parametrize("rows", [1, 30, 260])
def test_takes_the_norms_rows(bl, eight, rows):
    g = torch.Generator().manual_seed(8)
    x, gain = torch.randn(rows, 512, generator=g).to(torch.bfloat16), torch.rand(512, generator=g).to(torch.bfloat16)
    normed = bl.add_rms_norm(x.cuda(), gain.cuda(), eight_bit=eight)
    code = normed.q.dtype
    _, w, bias, _, _, ws = _make(code, 1, 512, 96, 9, torch.bfloat16)
    got = bl.linear(normed.q, w.cuda(), bias=bias.cuda(), activation="silu", x_scales=normed.scales, weight_scales=ws.cuda())
    _same(got, *plain.linear(normed.q.cpu(), w, bias, "silu", None, normed.scales.cpu(), ws, 0.01, torch.bfloat16))


@pytest.mark.parametrize("rows", [3, 20, 40, 300])
def test_sums_of_int8_are_exact(bl, rows):
    """Sums beyond 2^24, split or not, are rounded once: equal to the exact sum in float32."""
    inputs, outputs = 32768, 40
    g = torch.Generator().manual_seed(10)
    x = torch.randint(-128, 128, (rows, inputs), generator=g).to(torch.int8)
    w = torch.randint(-128, 128, (outputs, inputs), generator=g).to(torch.int8)
    x[0], w[0] = 127, 127
    w[1, : inputs // 2], w[1, inputs // 2:] = 127, -127  # what cancels over the splits
    w[1, 5] = 126
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    got = bl.linear(x.cuda(), w.cuda(), x_scales=one(rows), weight_scales=one(outputs), out_type=torch.float32)
    assert torch.equal(got.cpu(), (x.long() @ w.long().t()).float())


@pytest.mark.parametrize("rows", [40, 300])
def test_a_row_does_not_depend_on_its_neighbours(bl, rows):
    """float32 sums that are not finite are computed again, and the others stay as they were."""
    x, w, _, _, _, _ = _make(torch.float32, rows, 300, 200, 11)
    clean = bl.linear(x.cuda(), w.cuda())
    x[rows - 2] = torch.finfo(torch.float32).max  # rounds to infinity in bf16
    got = bl.linear(x.cuda(), w.cuda())
    rest = torch.arange(rows) != rows - 2
    assert torch.equal(got[rest.cuda()], clean[rest.cuda()])
    w = torch.zeros(200, 300)
    w[:, 7] = 0.5
    got = bl.linear(x.cuda(), w.cuda())
    assert torch.equal(got[rows - 2].cpu(), torch.full((200,), torch.finfo(torch.float32).max / 2))


def test_nothing_to_do(bl):
    for dtype in TYPES:
        w = torch.ones(5, 3, dtype=dtype, device="cuda")
        assert bl.linear(torch.ones(0, 3, dtype=dtype, device="cuda"), w).shape == (0, 5)

"""The matrix product at the edges of its range: e4m3 products that differ much, operands of any size, and its largest tiles
over several steps."""

import pytest
import torch

from tests import decoder_plain as plain
from tests.sequence_plain import TYPES

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _ones(n):
    return torch.ones(n, device="cuda")


@pytest.mark.parametrize("out_type", TYPES, ids=str)
@pytest.mark.parametrize("rows, inputs, outputs", [(1, 256, 40), (20, 256, 40), (40, 256, 40), (300, 250, 33), (40, 4096, 24),
                                                   (4100, 256, 4100), (4100, 250, 4100)])
def test_products_of_e4m3_far_below_their_neighbours_count(bl, out_type, rows, inputs, outputs):
    """Of eight neighbouring products one is 2^17 and cancels against the next eight's; the others are 4. All are whole
    numbers, and so are their sums, below 2^24: any order of additions in float32 is exact."""
    x, w = torch.full((rows, inputs), 2.0), torch.full((outputs, inputs), 2.0)
    whole = inputs // 16 * 16
    x[:, :whole:8] = 448.0
    w[:, :whole:16], w[:, 8:whole:16] = 448.0, -448.0
    x[::3, 1::2] = 1.0
    got = bl.linear(x.to(E4M3).cuda(), w.to(E4M3).cuda(), x_scales=_ones(rows), weight_scales=_ones(outputs), out_type=out_type)
    want = (x[:2].double() @ w[:1].double().t()).to(out_type).cuda()  # rows of two kinds, all outputs alike
    assert bool((got[::3] == want[0]).all()) and bool((got[1::3] == want[-1]).all())


@pytest.mark.parametrize("out_type", TYPES, ids=str)
@pytest.mark.parametrize("width", [16, 5])
def test_every_code_of_e4m3(bl, out_type, width):
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3)
    x, w = torch.zeros(256, width).to(E4M3), torch.zeros(7, width).to(E4M3)
    x[:, 3], w[2, 3] = codes, torch.ones(()).to(E4M3)
    want = codes.float().to(out_type)
    for rows in (slice(0, 256), slice(0, 30), slice(120, 150), slice(230, 256)):
        n = want[rows].shape[0]
        got = bl.linear(x[rows].cuda(), w.cuda(), x_scales=_ones(n), weight_scales=_ones(7), out_type=out_type)[:, 2].cpu()
        assert torch.equal(got.nan_to_num(nan=-1000), want[rows].nan_to_num(nan=-1000))
        back = bl.linear(w.cuda(), x[rows].cuda(), x_scales=_ones(7), weight_scales=_ones(n), out_type=out_type)[2].cpu()
        assert torch.equal(back.nan_to_num(nan=-1000), want[rows].nan_to_num(nan=-1000))


@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("inputs", [64, 77])
@pytest.mark.parametrize("x_size, w_size", [(1e-33, 1e30), (1e-35, 1e33), (1e-37, 1e35), (1e30, 1e-36), (1e-20, 1e-15), (1e-37, 1.0),
                                            (1e15, 1e12), (1e20, 1e10), (1e25, 1e10)])
def test_float32_operands_of_any_size(bl, rows, inputs, x_size, w_size):
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(rows, inputs, generator=g) * x_size, torch.randn(50, inputs, generator=g) * w_size
    bias, residual = torch.randn(50, generator=g) * x_size * w_size, torch.randn(rows, 50, generator=g) * x_size * w_size
    x[abs(x) < 2e-38], w[abs(w) < 2e-38] = 0, 0  # normal numbers
    value, bound = plain.linear(x, w, bias, None, residual, None, None, 0, torch.float32)
    off = (bl.linear(x.cuda(), w.cuda(), bias=bias.cuda(), residual=residual.cuda()).cpu().double() - value).abs()
    assert torch.isfinite(off).all() and (off <= bound).all(), f"{((off - bound) / bound).max():.3e} of the bound over it"


def _codes(dtype, rows, inputs, g):
    """Rows of a type, and of 8-bit types their scales."""
    x = torch.randn(rows, inputs, generator=g, device="cuda")
    if dtype not in plain.EIGHT:
        return x.to(dtype), None
    scale = x.abs().amax(1) / plain.EIGHT[dtype]
    q = x / scale[:, None]
    return (torch.round(q) if dtype == torch.int8 else q).to(dtype), scale


@pytest.mark.parametrize("out_type", TYPES, ids=str)
@pytest.mark.parametrize("dtype", TYPES + list(plain.EIGHT), ids=str)
@pytest.mark.parametrize("rows, outputs", [(4200, 4200), (5100, 5000)])
@pytest.mark.parametrize("extra", [0, 1])
def test_large_tiles_over_many_steps(bl, out_type, dtype, rows, outputs, extra):
    """One tile of 256 x 256 and more for every CU, halved ones in the last round or not, over six steps and a rest, with
    everything that an epilogue takes; with an element more the rows lie at any element."""
    if dtype not in plain.EIGHT and dtype != out_type:
        pytest.skip("y is of x's type")
    g = torch.Generator(device="cuda").manual_seed(rows)
    inputs = 816 // torch.finfo(dtype).bits * 8 + extra if dtype != torch.int8 else 816 + extra
    (x, xs), (w, ws) = _codes(dtype, rows, inputs, g), _codes(dtype, outputs, inputs, g)
    ws = None if ws is None else ws / inputs ** 0.5
    bias = torch.randn(outputs, generator=g, device="cuda").to(out_type)
    residual = torch.randn(rows, outputs, generator=g, device="cuda").to(out_type)
    got = bl.linear(x, w, bias=bias, activation="gelu", residual=residual, x_scales=xs, weight_scales=ws, out_type=out_type)
    some = torch.cat([torch.arange(0, rows, 137), torch.arange(rows - 9, rows)]).cuda()
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    value, bound = plain.linear(cpu(x[some.long()]), cpu(w), cpu(bias), "gelu", cpu(residual[some]), None if xs is None else cpu(xs[some]),
                                cpu(ws), 0, out_type)
    off = (got[some].cpu().double() - value).abs()
    assert torch.isfinite(off).all() and (off <= bound).all(), f"{(off - bound).max():.3e} over the bound"
    # the other rows: the same product of fewer, in smaller tiles, differs by the order of its sums (below 1e-4 for values of
    # this size: 2 n steps of 2^-24) and so by a step of y at most
    half = rows // 2
    low = bl.linear(x[:half], w[:700], bias=bias[:700], activation="gelu", residual=residual[:half, :700], x_scales=None if xs is None else xs[:half],
                    weight_scales=None if ws is None else ws[:700], out_type=out_type)
    near = torch.finfo(out_type).eps * (1 + low.float().abs()) + 1e-4
    assert ((got[:half, :700].float() - low.float()).abs() <= near).all()


@pytest.mark.parametrize("rows", [3, 150])
def test_float32_operands_down_to_the_smallest(bl, rows):
    """Subnormal numbers count, in any number of rows."""
    x, w = torch.zeros(rows, 40), torch.zeros(24, 40)
    for e in range(24):
        x[:, e], w[e, e] = 2.0 ** -(149 - e) * 3, 2.0 ** 110  # the first is 3 of the smallest
    got = bl.linear(x.cuda(), w.cuda()).cpu()
    assert torch.equal(got, torch.tensor([3 * 2.0 ** (e - 39) for e in range(24)]).expand(rows, 24))
    back = bl.linear(w.cuda(), x.cuda()).cpu()
    assert torch.equal(back, got.t())

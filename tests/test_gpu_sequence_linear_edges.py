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

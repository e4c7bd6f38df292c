"""The root-mean-square norm with the residual's addition and 8-bit outputs, against 64 bits."""

import pytest
import torch

from tests import sequence_plain as plain

pytestmark = pytest.mark.gpu

EIGHT = {"e4m3": (448.0, 2.0 ** -4, 2.0 ** -10), "int8": (127.0, 0.0, 0.5)}  # top, half step relative, half step


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _inputs(dtype, rows, width, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g).to(dtype)
    r = (torch.randn(rows, width, generator=g) * scale).to(dtype)
    return x, r, (torch.rand(width, generator=g) + 0.5).to(dtype)


def _check(got, x, r, w, eps, eight):
    y, s, error = plain.norm(x, w, eps, r)
    dtype = x.dtype
    if r is not None:
        assert ((got.residual.cpu().double() - s).abs() <= plain.rounded(s, 0 * s, torch.float32) + plain.rounded(s, 0 * s, dtype)).all()
    if got.y is not None:
        off = (got.y.cpu().double() - y).abs()
        assert (off <= plain.rounded(y, error, dtype)).all(), (off - plain.rounded(y, error, dtype)).max()
    if eight:
        top, relative, step = EIGHT[eight]
        scale = got.scales.cpu().double()[:, None]
        most = y.abs().amax(1, keepdim=True)
        expect = torch.where(most > 0, most / top, 1.0)
        # the scale carries y's relative error and two roundings
        slack = (error / y.abs().clamp(min=1e-300)).max() + 4 * plain.U32
        assert ((scale - expect).abs() <= slack * expect).all()
        value = got.q.cpu().double() * scale
        # half a step of the code at y's place, y's own error and the scale's (in y's size)
        bound = relative * y.abs() + step * expect + error + 3 * slack * y.abs() + slack * expect
        assert ((value - y).abs() <= bound).all(), ((value - y).abs() - bound).max()


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width", [1, 7, 64, 100, 256, 1000, 2048, 4097, 8200, 40000])
@pytest.mark.parametrize("eight", [None, "e4m3", "int8"])
@pytest.mark.parametrize("residual", [False, True])
def test_matches_the_definition(bl, dtype, width, eight, residual):
    rows = 5
    x, r, w = _inputs(dtype, rows, width, width)
    r = r if residual else None
    got = bl.add_rms_norm(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(), eight_bit=eight, keep_y=True)
    assert (got.q is None) == (eight is None) and (got.residual is None) == (not residual)
    _check(got, x, r, w, 1e-5, eight)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width", [33, 512, 2500, 40000])
def test_in_place_and_strided(bl, dtype, width):
    """Outputs in the inputs' own memory, rows of wider buffers, and the same bits as apart from it."""
    x, r, w = _inputs(dtype, 6, width, 1)
    apart = bl.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
    wide = torch.zeros(6, 2 * width + 8, dtype=dtype, device="cuda")
    xv, rv = wide[:, :width], wide[:, width + 8:]
    xv.copy_(x)
    rv.copy_(r)
    got = bl.add_rms_norm(xv, w.cuda(), residual=rv, out=xv, residual_out=rv)
    assert torch.equal(xv, apart.y) and torch.equal(rv, apart.residual) and got.y is xv
    assert not wide[:, width: width + 8].any()
    xv.copy_(x)
    rv.copy_(r)
    bl.add_rms_norm(xv, w.cuda(), residual=rv, out=rv, residual_out=xv)
    assert torch.equal(rv, apart.y) and torch.equal(xv, apart.residual)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("eight", ["e4m3", "int8"])
def test_edge_rows(bl, dtype, eight):
    """Zeros, one large value, tiny values, and rows that are not numbers."""
    x = torch.zeros(6, 96, dtype=dtype)
    x[1, 17] = 100.0
    x[2] = torch.finfo(dtype).smallest_normal
    x[3, 5] = float("nan")
    x[4, 5] = float("inf")
    x[5] = 1.0
    w = torch.ones(96, dtype=dtype)
    got = bl.add_rms_norm(x.cuda(), w.cuda(), 1e-5, eight_bit=eight, keep_y=True)
    for i in (0, 1, 2, 5):
        one = bl.NormResult(got.y[i: i + 1], got.q[i: i + 1], got.scales[i: i + 1], None)
        if i == 2 and dtype != torch.float16:
            # far below the least scale 2^-100: codes of zero
            assert got.scales[2].item() == 2.0 ** -100 and not got.q[2].float().any()
        else:
            _check(one, x[i: i + 1], None, w, 1e-5, eight)
    assert got.scales[0].item() == 1.0 and not got.q[0].float().any() and not got.y[0].any()
    assert torch.isnan(got.scales[3:5]).all() and torch.isnan(got.y[3]).all() and torch.isnan(got.y[4, 5])


def test_many_rows_and_none(bl):
    x, r, w = _inputs(torch.float32, 18848, 256, 2)
    got = bl.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
    _check(got, x, r, w, 1e-5, None)
    none = bl.add_rms_norm(x[:0].cuda(), w.cuda(), residual=r[:0].cuda(), eight_bit="e4m3")
    assert none.q.shape == (0, 256) and none.scales.shape == (0,)


def test_captured_graph_and_stream(bl):
    x, r, w = (t.cuda() for t in _inputs(torch.bfloat16, 40, 1024, 3))
    expect = bl.add_rms_norm(x, w, residual=r, eight_bit="e4m3")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = bl.add_rms_norm(x, w, residual=r, eight_bit="e4m3", stream=side)
    side.synchronize()
    assert torch.equal(other.scales, expect.scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bl.add_rms_norm(x, w, residual=r, eight_bit="e4m3")
    for k in range(3):
        x.copy_(torch.randn(40, 1024, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        again = bl.add_rms_norm(x, w, residual=r, eight_bit="e4m3")
        assert torch.equal(got.q.view(torch.uint8), again.q.view(torch.uint8))
        assert torch.equal(got.scales, again.scales) and torch.equal(got.residual, again.residual)


def test_the_binding_refuses_what_the_operators_do_not_take(bl):
    """Types, shapes, devices, strides within a row, gradients: said before anything runs."""
    x, r, w = (t.cuda() for t in _inputs(torch.float32, 4, 64, 5))
    for error, call in (
            (TypeError, lambda: bl.add_rms_norm(x.cpu(), w)),
            (TypeError, lambda: bl.add_rms_norm(x, w.cpu())),
            (TypeError, lambda: bl.add_rms_norm(x, w.double())),
            (TypeError, lambda: bl.add_rms_norm(x.double(), w.double())),
            (TypeError, lambda: bl.add_rms_norm(x, [1.0] * 64)),
            (ValueError, lambda: bl.add_rms_norm(x, w[:63])),
            (ValueError, lambda: bl.add_rms_norm(x[0], w)),
            (ValueError, lambda: bl.add_rms_norm(x.t().contiguous().t(), w)),
            (ValueError, lambda: bl.add_rms_norm(x, w, eight_bit="int4")),
            (ValueError, lambda: bl.add_rms_norm(x, w, residual_out=r)),
            (ValueError, lambda: bl.add_rms_norm(x, w, keep_y=False)),
            (TypeError, lambda: bl.add_rms_norm(x, w.clone().requires_grad_())),
            (bl.BilstmError, lambda: bl.add_rms_norm(x, w, eps=-1.0)),
            (bl.BilstmError, lambda: bl.add_rms_norm(x, w, residual=r, out=r[:, :], residual_out=r)),
            (bl.BilstmError, lambda: bl.add_rms_norm(x[:1].expand(4, 64), w, out=x))):
        with pytest.raises(error):
            call()
    with torch.no_grad():
        assert bl.add_rms_norm(x, w.clone().requires_grad_()).y.shape == x.shape


CODES = {"e4m3": (448.0, lambda v: v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)),
         "int8": (127.0, lambda v: torch.round(v).clamp(-127.0, 127.0).to(torch.int8))}


@pytest.mark.parametrize("width", [64, 1000, 2048, 4097, 20000])
@pytest.mark.parametrize("eight", ["e4m3", "int8"])
def test_codes_are_those_of_the_quotients(bl, width, eight):
    """The scale is max|y| / top and a code the nearest to y / scale, in float32 as y is: bit for bit, in every
    form of the kernel. A row has about 2^-18 values a code's rounding tells apart in the quotient's last bit."""
    rows = (1 << 21) // width
    x, r, w = _inputs(torch.float32, rows, width, 31)
    got = bl.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), eight_bit=eight, keep_y=True)
    top, code = CODES[eight]
    y, scales = got.y.cpu(), got.scales.cpu()
    assert torch.equal(scales, y.abs().amax(1) / top)
    expect = code(y / scales[:, None])
    assert torch.equal(got.q.cpu().view(torch.uint8), expect.view(torch.uint8))


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width", [96, 3000, 40000])
@pytest.mark.parametrize("eight", ["e4m3", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_weights_that_are_not_numbers(bl, dtype, width, eight, bad):
    """What is not a number in y makes the row's scale none, wherever it came from."""
    x, _, w = _inputs(dtype, 3, width, 32)
    x[1, 7] = 0.0
    w[7] = bad
    got = bl.add_rms_norm(x.cuda(), w.cuda(), eight_bit=eight, keep_y=True)
    assert torch.isnan(got.scales).all()
    assert not torch.isfinite(got.y[:, 7]).any() and torch.isfinite(got.y[:, 8:]).all()


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("width", [1, 96, 3000, 9000, 40000])
@pytest.mark.parametrize("eight", [None, "e4m3", "int8"])
@pytest.mark.parametrize("eps", [0.0, 1e-42])
def test_tiny_rows_without_eps(bl, dtype, width, eight, eps):
    """Squares below float32's range, down to its smallest number, and rows of zeros. plain.norm's bound holds
    for them as for any row: sums of squares of values times a power of two round as others do."""
    x, _, w = _inputs(dtype, 6, width, 33)
    x[0] = 0.0
    small = [1e-18, 1e-25, 1e-38, 1e-44] if dtype != torch.float16 else [1e-2, 1e-3, 1e-5, 6e-8]
    for i, size in enumerate(small):
        x[1 + i] = (torch.sign(x[1 + i].float()) * (0.5 + torch.rand(width, generator=torch.Generator().manual_seed(i))) * size).to(dtype)
        if not x[1 + i].any():
            x[1 + i] = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    eps = float(torch.tensor(eps, dtype=torch.float32))  # what the call gets
    got = bl.add_rms_norm(x.cuda(), w.cuda(), eps, eight_bit=eight, keep_y=True)
    rest = bl.NormResult(got.y[1:], None if eight is None else got.q[1:], None if eight is None else got.scales[1:], None)
    _check(rest, x[1:], None, w, eps, eight)
    assert not got.y[0].any()
    if eight:
        assert got.scales[0].item() == 1.0 and not got.q[0].float().any()


def test_tiny_rows_in_place(bl):
    """The sum with a residual comes back unchanged from rows that are looked at a second time."""
    for width in (96, 3000, 9000, 40000):
        x, r, w = _inputs(torch.float32, 4, width, 34)
        x, r = x * 1e-30, r * 1e-30
        xg, rg = x.cuda(), r.cuda()
        apart = bl.add_rms_norm(x.cuda(), w.cuda(), 0.0, residual=r.cuda())
        bl.add_rms_norm(xg, w.cuda(), 0.0, residual=rg, out=rg, residual_out=xg)
        assert torch.equal(xg.cpu(), x + r) and torch.equal(rg, apart.y) and torch.equal(apart.residual, xg)


def test_the_binding_refuses_forward_mode_tangents(bl):
    """These operators have no derivatives of either mode."""
    import torch.autograd.forward_ad as fw
    x, r, w = (t.cuda() for t in _inputs(torch.float32, 4, 64, 36))
    tokens = torch.zeros(4, dtype=torch.int64, device="cuda")
    starts = torch.tensor([0, 4], dtype=torch.int32).cuda()
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones_like(x))
        for call in (lambda: bl.add_rms_norm(dual, w), lambda: bl.add_rms_norm(x, w, residual=dual),
                     lambda: bl.token_logprobs(dual, tokens), lambda: bl.causal_conv(dual, x.new_ones(64, 2), starts),
                     lambda: bl.causal_conv_step(x, x.new_ones(64, 2), fw.make_dual(x.new_zeros(4, 1, 64), x.new_ones(4, 1, 64))),
                     lambda: bl.selective_scan(dual.view(4, 2, 32), x.new_ones(4, 2), -x.new_ones(2), x.new_ones(4, 1, 16),
                                               x.new_ones(4, 1, 16), starts)):
            with pytest.raises(TypeError, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(TypeError, match="tangent"):
                call()
        assert bl.add_rms_norm(x, w).y.shape == x.shape
        assert bl.add_rms_norm(fw.unpack_dual(dual).primal, w).y.shape == x.shape
    assert bl.add_rms_norm(x, w).y.shape == x.shape


def test_an_error_from_before_is_not_the_calls(bl):
    """An error that an earlier, refused HIP call left behind is neither reported by a sound call nor taken away."""
    import ctypes
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
    assert len(paths) == 1
    hip = ctypes.CDLL(paths.pop())
    x, r, w = (t.cuda() for t in _inputs(torch.float32, 4, 64, 35))
    starts = torch.tensor([0, 4], dtype=torch.int32).cuda()
    tokens, large = torch.zeros(4, dtype=torch.int64, device="cuda"), x.new_zeros(4, 20000)
    taps, rows, states = x.new_ones(64, 2), x.new_zeros(4, 1, 64), x.new_zeros(4, 2, 32, 16)
    heads, dt, a, b = x.view(4, 2, 32), x.new_ones(4, 2), -x.new_ones(2), x.new_ones(4, 1, 16)
    many, many_dt, many_b = x.new_ones(400, 2, 32), x.new_ones(400, 2), x.new_ones(400, 1, 16)
    whole = torch.tensor([0, 400], dtype=torch.int32).cuda()
    cases = [lambda: bl.add_rms_norm(x, w, residual=r, eight_bit="int8"), lambda: bl.causal_conv(x, taps, starts),
             lambda: bl.causal_conv_step(x, taps, rows), lambda: bl.token_logprobs(x, tokens, top=2),
             lambda: bl.token_logprobs(large, tokens, top=2), lambda: bl.selective_scan(heads, dt, a, b, b, starts),
             lambda: bl.selective_scan(many, many_dt, a, many_b, many_b, whole),
             lambda: bl.selective_scan_step(heads, dt, a, b, b, states)]
    for case in cases:
        case()
    torch.cuda.synchronize()
    for case in cases:
        refused = hip.hipSetDevice(1 << 20)
        assert refused != 0
        try:
            case()
        finally:
            left = hip.hipGetLastError()
        assert left == refused
    torch.cuda.synchronize()

"""Log probabilities of given tokens, entropy and top alternatives, against 64 bits."""

import pytest
import torch

from tests import sequence_plain as plain

pytestmark = pytest.mark.gpu

# groups of lanes (up to 1024, up to 2048 for few alternatives), one tile, several tiles, odd sizes around their borders
VOCABULARIES = [1, 2, 7, 8, 9, 31, 33, 129, 255, 257, 512, 513, 1024, 1025, 2048, 2049, 5000, 8185, 8186, 8189, 8190, 8193, 16377, 16378, 16390, 40001]


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


def _logits(dtype, rows, v, seed, scale=4.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, v, generator=g) * scale).to(dtype), torch.randint(0, v, (rows, 3), generator=g)


def _same(got, value, bound, what):
    got = got.cpu().double()
    fine = torch.isfinite(value)
    assert torch.equal(torch.isnan(got), torch.isnan(value)), what
    assert torch.equal(got[~fine & ~torch.isnan(value)], value[~fine & ~torch.isnan(value)]), what
    off = (got - value)[fine].abs()
    assert (off <= bound[fine]).all(), f"{what}: {(off - bound[fine]).max():.3e} over the bound"


def _check(r, logits, tokens, top):
    (given, entropy, order, top_lp), (gb, eb, tb) = plain.logprobs(logits, tokens, top)
    _same(r.logprobs, given, gb, "logprobs")
    _same(r.entropy, entropy, eb, "entropy")
    if top:
        assert torch.equal(r.top_tokens.cpu(), order)
        _same(r.top_logprobs, top_lp, tb, "top_logprobs")


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("vocabulary", VOCABULARIES)
@pytest.mark.parametrize("top", [0, 1, 8, 32])
def test_matches_the_definition(bl, dtype, vocabulary, top):
    top = min(top, vocabulary)
    logits, tokens = _logits(dtype, 9, vocabulary, vocabulary)
    _check(bl.token_logprobs(logits.cuda(), tokens.cuda(), top=top), logits, tokens, top)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("vocabulary,top", [(7, 7), (200, 20), (400, 20), (1000, 20), (1500, 8), (1500, 20), (6000, 20), (20001, 20)])
def test_masks(bl, dtype, vocabulary, top):
    """Rows with few tokens left, with none, masks of the type's lowest value, one token, equal logits."""
    logits, tokens = _logits(dtype, 8, vocabulary, 3)
    keep = torch.arange(vocabulary) % 997 == 5
    logits[0, ~keep] = float("-inf")
    logits[1] = float("-inf")
    logits[2] = torch.finfo(dtype).min
    logits[3, ~keep] = torch.finfo(dtype).min
    logits[4] = float("-inf")
    logits[4, vocabulary - 1] = -3.0
    logits[5] = 1.5
    logits[6, ::2] = -0.0
    logits[6, 1::2] = 0.0
    logits[7, : vocabulary - 1] = float("-inf")
    tokens[:, 0] = 5
    tokens[:, 1] = vocabulary - 1
    r = bl.token_logprobs(logits.cuda(), tokens.cuda(), top=top)
    _check(r, logits, tokens, top)
    assert torch.isinf(r.logprobs[1]).all() and r.entropy[1].item() == 0.0
    assert r.top_tokens[1].tolist() == list(range(top))


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
@pytest.mark.parametrize("vocabulary", [50, 9000])
def test_not_numbers_and_tokens_outside(bl, dtype, vocabulary):
    logits, tokens = _logits(dtype, 4, vocabulary, 4)
    logits[0, 3] = float("nan")
    logits[1, 4] = float("inf")
    logits[2, vocabulary - 1] = float("nan")
    logits[2, :9] = float("-inf")
    tokens[3] = torch.tensor([-1, vocabulary, 2 ** 40])
    r = bl.token_logprobs(logits.cuda(), tokens.cuda(), top=2)
    assert torch.isnan(r.logprobs).all()
    assert torch.isnan(r.entropy[:3]).all() and torch.isfinite(r.entropy[3])
    assert torch.isnan(r.top_logprobs[:3]).all()
    assert r.top_tokens[:3, 0].tolist() == [3, 4, vocabulary - 1]


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_ties_fall_to_the_lowest_token(bl, dtype):
    """Logits of few values: more equal ones than a tile's list holds, over several tiles."""
    g = torch.Generator().manual_seed(6)
    for vocabulary, values in ((300, 3), (8000, 40), (30000, 9), (30000, 1)):
        logits = torch.randint(0, values, (5, vocabulary), generator=g).to(dtype)
        r = bl.token_logprobs(logits.cuda(), torch.zeros(5, dtype=torch.int64).cuda(), top=32)
        assert torch.equal(r.top_tokens.cpu(), torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :32])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8, 1e20, 1e37])
@pytest.mark.parametrize("vocabulary", [100, 20000])
def test_logits_of_any_size(bl, dtype, size, vocabulary):
    """Far from zero, alone and with the spread of ordinary logits, on both sides."""
    logits, tokens = _logits(dtype, 6, vocabulary, 21, scale=1.0)
    logits[:2] = logits[:2] * size
    logits[2:4] = logits[2:4] - size
    logits[4:] = logits[4:] + size
    _check(bl.token_logprobs(logits.cuda(), tokens.cuda(), top=5), logits, tokens, 5)


def test_rising_logits(bl):
    """Every tile beats the one before it."""
    logits = torch.arange(50000, dtype=torch.float32).repeat(3, 1) * 1e-3
    r = bl.token_logprobs(logits.cuda(), torch.full((3,), 49999).cuda(), top=16)
    assert r.top_tokens[1].tolist() == list(range(49999, 49999 - 16, -1))
    assert r.logprobs.shape == (3,)


@pytest.mark.parametrize("dtype", plain.TYPES, ids=str)
def test_strided_rows_of_every_alignment(bl, dtype):
    wide = (torch.randn(17, 9011, generator=torch.Generator().manual_seed(7)) * 3).to(dtype)
    logits = wide[:, 1:9010]
    tokens = torch.randint(0, 9009, (17, 1), generator=torch.Generator().manual_seed(8))
    _check(bl.token_logprobs(wide.cuda()[:, 1:9010], tokens.cuda(), top=5), logits, tokens, 5)


def test_row_offsets_past_32_bits(bl):
    stride = (1 << 30) + 1
    base = torch.zeros(2 * stride + 5000, dtype=torch.bfloat16, device="cuda")
    view = base.as_strided((3, 5000), (stride, 1))
    logits, tokens = _logits(torch.bfloat16, 3, 5000, 9)
    view.copy_(logits)
    _check(bl.token_logprobs(view, tokens.cuda(), top=4), logits, tokens, 4)


def test_largest_vocabulary_and_one_row(bl):
    logits, tokens = _logits(torch.bfloat16, 1, 1 << 20, 10)
    _check(bl.token_logprobs(logits.cuda(), tokens.cuda(), top=32), logits, tokens, 32)


def test_no_rows_and_no_tokens(bl):
    r = bl.token_logprobs(torch.zeros(0, 9).cuda(), torch.zeros(0, 2, dtype=torch.int64).cuda(), top=3)
    assert r.logprobs.shape == (0, 2) and r.top_tokens.shape == (0, 3)
    logits, _ = _logits(torch.float32, 4, 9000, 11)
    r = bl.token_logprobs(logits.cuda(), torch.zeros(4, 0, dtype=torch.int64).cuda())
    _check(r, logits, torch.zeros(4, 0, dtype=torch.int64), 0)


def test_after_the_heads(bl):
    """The heads' output, log probabilities of seven classes, normalised again changes nothing."""
    lp = torch.log_softmax(torch.randn(100, 7, generator=torch.Generator().manual_seed(12)), 1)
    label = torch.randint(0, 7, (100, 1), generator=torch.Generator().manual_seed(13))
    _check(bl.token_logprobs(lp.cuda(), label.cuda(), top=3), lp, label, 3)


def test_captured_graphs_do_not_share_scratch(bl):
    """Two graphs captured one after the other, replayed at the same time on two streams."""
    a, ta = _logits(torch.float32, 16, 60000, 14)
    b, tb = _logits(torch.float32, 16, 60000, 15)
    a, ta, b, tb = a.cuda(), ta.cuda(), b.cuda(), tb.cuda()
    expect = [bl.token_logprobs(a, ta, top=8), bl.token_logprobs(b, tb, top=8)]
    graphs, got = [], []
    for z, t in ((a, ta), (b, tb)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(bl.token_logprobs(z, t, top=8))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for g, e in zip(got, expect):
            for x, y in zip(g, e):
                assert torch.equal(x, y)
            for x in g:
                x.zero_()

"""Calls of the sequence operators whose launches have more work-items than 32 bits count: every row is computed."""

import pytest
import torch

pytestmark = pytest.mark.gpu

MANY = (1 << 24) + 5  # workgroups of 256: a little more than 2^32 work-items


@pytest.fixture(scope="module")
def bl():
    import bidirectional_lstm_sequence_amd as bl
    return bl


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.is_available() and torch.cuda.mem_get_info()[1] < 200 << 30:
        pytest.skip("needs a card of 200 GB or more")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows, width", [(MANY, 1028)])
def test_norm(bl, rows, width):
    x = torch.full((rows, width), 2.0, device="cuda")
    y = bl.add_rms_norm(x, torch.ones(width, device="cuda"), 0.0, out=x).y
    assert y.data_ptr() == x.data_ptr() and bool((y.view(-1) == 1.0).all())


@pytest.mark.parametrize("rows, vocabulary", [(4 * MANY, 257), (MANY, 2049)])
def test_log_probabilities(bl, rows, vocabulary):
    """Groups of lanes, four rows a workgroup, and a tile a row."""
    logits = torch.zeros(rows, vocabulary, dtype=torch.bfloat16, device="cuda")
    r = bl.token_logprobs(logits, torch.zeros(rows, dtype=torch.int64, device="cuda"))
    expect = -torch.log(torch.tensor(float(vocabulary)))
    for got, value in ((r.logprobs, expect), (r.entropy, -expect)):
        assert abs(got.min().item() - value) < 1e-5 and abs(got.max().item() - value) < 1e-5


def test_scan_step(bl):
    """One head of one row a workgroup: D = dt, S = S exp(-D) + D, y = the sum of 16 states and x."""
    heads = 1024
    rows = MANY // heads + 1
    one = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    state = torch.zeros(rows, heads, 32, 16, device="cuda")
    y = bl.selective_scan_step(one(rows, heads, 32), one(rows, heads), -torch.ones(heads, device="cuda"), one(rows, 1, 16),
                               one(rows, 1, 16), state, d=torch.ones(heads, device="cuda"), softplus=False)
    assert bool((y == 17.0).all()) and bool((state.view(-1) == 1.0).all())


def test_scan(bl):
    """256 workgroups a sequence of one row."""
    heads = 1024
    rows = MANY // 256 + 1
    one = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y = bl.selective_scan(one(rows, heads, 32), one(rows, heads), -torch.ones(heads, device="cuda"), one(rows, 1, 16),
                          one(rows, 1, 16), torch.arange(rows + 1, dtype=torch.int32, device="cuda"),
                          d=torch.ones(heads, device="cuda"), softplus=False)
    assert bool((y == 17.0).all())

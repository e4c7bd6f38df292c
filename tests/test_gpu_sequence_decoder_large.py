"""Cross attention and the matrix product where offsets pass 32 bits."""

import pytest
import torch

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("step", [False, True])
def test_memories_behind_four_gigabytes(bl, step):
    """Keys and values of 2^32 elements and more: a memory at their end against the same rows alone."""
    groups, width, held = 8, 128, 2200000
    kv = torch.zeros(held, 2 * groups * width, dtype=torch.bfloat16, device="cuda")
    assert kv.numel() > 1 << 32
    g = torch.Generator().manual_seed(1)
    tail = torch.randn(500, 2 * groups * width, generator=g).to(torch.bfloat16).cuda()
    kv[-500:] = tail
    n = groups * width
    q = torch.randn(2, 32, width, generator=g).to(torch.bfloat16).cuda()
    whole = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(rows, memory_starts, slots):
        k, v = rows[:, :n].view(-1, groups, width), rows[:, n:].view(-1, groups, width)
        if step:
            return bl.cross_attention_step(q, k, v, whole(memory_starts), slots=whole(slots))
        return bl.cross_attention(q, k, v, whole([0, 1, 2]), whole(memory_starts), slots=whole(slots))

    got = run(kv, [0, held - 500, held - 200, held], [1, 2])
    alone = run(tail, [0, 0, 300, 500], [1, 2])
    assert (got.float() - alone.float()).abs().max() < 0.05 and got.abs().max() > 0


def test_outputs_behind_four_gigabytes(bl):
    rows, outputs = (1 << 22) + 77, 1032
    x = torch.ones(rows, 16, dtype=torch.bfloat16, device="cuda")
    x[-1] = 2
    w = torch.ones(outputs, 16, dtype=torch.bfloat16, device="cuda")
    y = bl.linear(x, w)
    assert y.numel() > 1 << 32
    assert bool((y[:-1].view(-1) == 16).all()) and bool((y[-1] == 32).all())
    x8 = torch.ones(rows, 15, dtype=torch.int8, device="cuda")  # rows at any byte
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = bl.linear(x8, torch.ones(outputs, 15, dtype=torch.int8, device="cuda"), x_scales=one(rows), weight_scales=one(outputs), out=y)
    assert bool((y.view(-1) == 15).all())


def test_weights_behind_four_gigabytes(bl):
    inputs, outputs = 65536, 65600
    w = torch.ones(outputs, inputs, dtype=torch.int8, device="cuda")
    w[-1] = 2
    x = torch.ones(3, inputs, dtype=torch.int8, device="cuda")
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = bl.linear(x, w, x_scales=one(3), weight_scales=one(outputs), out_type=torch.float32)
    assert bool((y[:, :-1] == inputs).all()) and bool((y[:, -1] == 2 * inputs).all())


def test_wide_strides(bl):
    """Rows further apart than the kernels' tiles of rows reach with 32-bit offsets."""
    g = torch.Generator().manual_seed(2)
    apart = 6 << 20
    store = torch.zeros(70 * apart, dtype=torch.float16, device="cuda")
    x = store.view(70, apart)[:, :64]
    x.copy_(torch.randn(70, 64, generator=g))
    w = torch.randn(72, 64, generator=g).half().cuda()
    assert torch.equal(bl.linear(x, w), bl.linear(x.contiguous(), w))
    assert torch.equal(bl.linear(w, x), bl.linear(w, x.contiguous()))
    far = torch.zeros(140, 10 << 20, dtype=torch.float16, device="cuda")[:, :64]
    far.copy_(torch.randn(140, 64, generator=g))
    k = far.view(140, 1, 64)
    q = torch.randn(5, 2, 64, generator=g).half().cuda()
    whole = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    got = bl.cross_attention(q, k, k, whole([0, 5]), whole([0, 140]))
    near = bl.cross_attention(q, k.contiguous(), k.contiguous(), whole([0, 5]), whole([0, 140]))
    assert torch.equal(got, near)

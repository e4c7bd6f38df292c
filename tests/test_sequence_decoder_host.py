"""Refusals of cross attention and of the matrix product: the entry points check their arguments before
they touch a device, so this runs without a GPU. Pointers are numbers that nothing reads."""

import ctypes

import pytest

P = 1 << 20  # a 16-byte aligned address that no check follows


@pytest.fixture(scope="module")
def bl():
    import os

    import bidirectional_lstm_sequence_amd as bl
    if not os.path.exists(bl.LIB_PATH):
        from bidirectional_lstm_sequence_amd import _build
        _build.build()
    bl.library()
    return bl


def status(bl, name, packed):
    return bl.STATUS[getattr(bl.library(), name)(packed, None)]


def pack(form, f):
    flat = []
    for v in f.values():
        flat.extend(v if isinstance(v, tuple) else (v,))
    return form.pack(*flat)


def attention_args(**over):
    """64 rows of 4 heads of 32 in 3 sequences, 5 memories of 200 rows of 2 heads."""
    f = dict(device=0, type=1, rows=64, memory_rows=200, heads=4, groups=2, width=32, sequences=3, places=5, scale=0.2,
             reserved0=0, reserved1=0, q=(P, 64 * 128, 128), k=(2 * P, 200 * 64, 64), v=(3 * P, 200 * 64, 64),
             starts=(4 * P, 4), slots=(5 * P, 3), memory_starts=(6 * P, 6), memory_lengths=(7 * P, 5), mask=(8 * P, 200),
             y=(9 * P, 64 * 128, 128), scratch=(20 * P, 1 << 30))
    f.update(over)
    return f


ATTENTION_BAD = [
    (dict(type=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(heads=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(groups=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(groups=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(heads=65538), "BILSTM_INVALID_ARGUMENT"),
    (dict(width=0), "BILSTM_UNSUPPORTED"),
    (dict(width=257), "BILSTM_UNSUPPORTED"),
    (dict(rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(memory_rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(memory_rows=(1 << 30) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(sequences=(1 << 30) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(places=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(scale=0.0), "BILSTM_INVALID_ARGUMENT"),
    (dict(scale=-1.0), "BILSTM_INVALID_ARGUMENT"),
    (dict(scale=float("nan")), "BILSTM_INVALID_ARGUMENT"),
    (dict(scale=float("inf")), "BILSTM_INVALID_ARGUMENT"),
    (dict(reserved0=1), "BILSTM_INVALID_ARGUMENT"),
    (dict(reserved1=1), "BILSTM_INVALID_ARGUMENT"),
    (dict(q=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(q=(P + 1, 64 * 128, 128)), "BILSTM_INVALID_ARGUMENT"),
    (dict(q=(P, 64 * 128 - 1, 128)), "BILSTM_BUFFER_LENGTH"),
    (dict(q=(P, 64 * 128, 127)), "BILSTM_INVALID_ARGUMENT"),
    (dict(k=(2 * P, 199 * 64, 64)), "BILSTM_BUFFER_LENGTH"),
    (dict(k=(2 * P, 1 << 62, 1 << 58)), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(v=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(v=(3 * P, 200 * 64, 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(starts=(4 * P, 3)), "BILSTM_BUFFER_LENGTH"),
    (dict(starts=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(starts=(4 * P + 2, 4)), "BILSTM_INVALID_ARGUMENT"),
    (dict(slots=(5 * P, 4)), "BILSTM_BUFFER_LENGTH"),
    (dict(slots=(0, 0), places=2, memory_starts=(6 * P, 3), memory_lengths=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(memory_starts=(6 * P, 5)), "BILSTM_BUFFER_LENGTH"),
    (dict(memory_starts=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(memory_lengths=(7 * P, 4)), "BILSTM_BUFFER_LENGTH"),
    (dict(mask=(8 * P, 199)), "BILSTM_BUFFER_LENGTH"),
    (dict(y=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(y=(9 * P, 64 * 128, 100)), "BILSTM_INVALID_ARGUMENT"),
    (dict(y=(P, 64 * 128, 128)), "BILSTM_INVALID_ARGUMENT"),  # q
    (dict(y=(3 * P - 2, 64 * 128, 128)), "BILSTM_INVALID_ARGUMENT"),  # v
    (dict(y=(8 * P, 64 * 128, 128)), "BILSTM_INVALID_ARGUMENT"),  # the mask
    (dict(y=(6 * P, 64 * 128, 128)), "BILSTM_INVALID_ARGUMENT"),  # memory_starts
]


@pytest.mark.parametrize("over, expected", ATTENTION_BAD, ids=lambda v: str(v)[:60])
def test_attention_refuses(bl, over, expected):
    assert status(bl, "bilstm_cross_attention", pack(bl.sequence._ATTENTION, attention_args(**over))) == expected
    assert bl.last_error().startswith("cross_attention:")


@pytest.mark.parametrize("over, expected", [
    (dict(slots=(5 * P, 3)), "BILSTM_BUFFER_LENGTH"),
    (dict(slots=(0, 0)), "BILSTM_INVALID_ARGUMENT"),  # 64 rows, 5 memories
    (dict(width=300), "BILSTM_UNSUPPORTED"),
    (dict(slots=(5 * P, 64), y=(5 * P, 64 * 128, 128)), "BILSTM_INVALID_ARGUMENT"),
], ids=str)
def test_attention_step_refuses(bl, over, expected):
    f = dict(slots=(5 * P, 64), starts=(0, 0))
    f.update(over)
    assert status(bl, "bilstm_cross_attention_step", pack(bl.sequence._ATTENTION, attention_args(**f))) == expected
    assert bl.last_error().startswith("cross_attention_step:")


def test_attention_accepts_what_the_header_allows(bl):
    """Sound arguments pass every check: without a device the call then says so, and nothing was read."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are numbers: nothing may be launched")
    form = bl.sequence._ATTENTION
    for over in (dict(), dict(memory_lengths=(0, 0), mask=(0, 0)), dict(slots=(0, 0)),
                 dict(k=(2 * P, 200 * 128, 128), v=(2 * P + 128, 200 * 128 - 64, 128)),  # side by side
                 dict(q=(P, 64 * 256, 256), y=(P + 256, 64 * 256 - 128, 256)),
                 dict(memory_rows=0, k=(0, 0, 0), v=(0, 0, 0), mask=(0, 0)),
                 dict(places=0, memory_starts=(6 * P, 1), memory_lengths=(0, 0))):
        assert status(bl, "bilstm_cross_attention", pack(form, attention_args(**over))) == "BILSTM_UNSUPPORTED"
        assert "no HIP device" in bl.last_error()
    step = attention_args(slots=(5 * P, 64), starts=(0, 0), sequences=77)
    assert status(bl, "bilstm_cross_attention_step", pack(form, step)) == "BILSTM_UNSUPPORTED"
    assert status(bl, "bilstm_cross_attention", pack(form, attention_args(rows=0))) == "BILSTM_OK"
    assert status(bl, "bilstm_cross_attention", pack(form, attention_args(sequences=0, starts=(0, 0)))) == "BILSTM_OK"


def linear_args(**over):
    """64 rows of 32 inputs and 48 outputs, bfloat16."""
    f = dict(device=0, type=1, rows=64, inputs=32, outputs=48, eight=0, activation=0, slope=0.0, reserved=0,
             x=(P, 64 * 32, 32), weight=(2 * P, 48 * 32, 32), bias=(3 * P, 48), residual=(4 * P, 64 * 48, 48),
             x_scales=(0, 0), weight_scales=(0, 0), y=(5 * P, 64 * 48, 48), scratch=(20 * P, 1 << 30))
    f.update(over)
    return f


SCALED = dict(eight=1, x_scales=(6 * P, 64), weight_scales=(7 * P, 48))
LINEAR_BAD = [
    (dict(type=-1), "BILSTM_INVALID_ARGUMENT"),
    (dict(eight=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(inputs=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(outputs=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(activation=5), "BILSTM_INVALID_ARGUMENT"),
    (dict(activation=-1), "BILSTM_INVALID_ARGUMENT"),
    (dict(slope=float("nan")), "BILSTM_INVALID_ARGUMENT"),
    (dict(slope=float("inf")), "BILSTM_INVALID_ARGUMENT"),
    (dict(reserved=1), "BILSTM_INVALID_ARGUMENT"),
    (dict(rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(rows=(1 << 31) - 1023), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(inputs=(1 << 28) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(outputs=(1 << 28) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(SCALED, eight=2, inputs=(1 << 16) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(x=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P + 1, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P, 64 * 32 - 1, 32)), "BILSTM_BUFFER_LENGTH"),
    (dict(x=(P, 64 * 32, 31)), "BILSTM_INVALID_ARGUMENT"),
    (dict(weight=(2 * P, 47 * 32, 32)), "BILSTM_BUFFER_LENGTH"),
    (dict(bias=(3 * P, 47)), "BILSTM_BUFFER_LENGTH"),
    (dict(residual=(4 * P, 64 * 47, 48)), "BILSTM_BUFFER_LENGTH"),
    (dict(x_scales=(6 * P, 64)), "BILSTM_INVALID_ARGUMENT"),
    (dict(weight_scales=(6 * P, 48)), "BILSTM_INVALID_ARGUMENT"),
    (dict(SCALED, x_scales=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(SCALED, x_scales=(6 * P, 63)), "BILSTM_BUFFER_LENGTH"),
    (dict(SCALED, weight_scales=(7 * P, 49)), "BILSTM_BUFFER_LENGTH"),
    (dict(SCALED, weight_scales=(7 * P + 2, 48)), "BILSTM_INVALID_ARGUMENT"),
    (dict(y=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(y=(P, 64 * 48, 48)), "BILSTM_INVALID_ARGUMENT"),  # x
    (dict(y=(2 * P, 64 * 48, 48)), "BILSTM_INVALID_ARGUMENT"),  # the weight
    (dict(y=(3 * P, 64 * 48, 48)), "BILSTM_INVALID_ARGUMENT"),  # the bias
    (dict(y=(4 * P + 2, 64 * 48, 48)), "BILSTM_INVALID_ARGUMENT"),  # the residual, one element on
    (dict(y=(4 * P, 64 * 49, 49)), "BILSTM_INVALID_ARGUMENT"),  # the residual with another stride
    (dict(SCALED, y=(6 * P, 64 * 48, 48)), "BILSTM_INVALID_ARGUMENT"),  # the scales
]


@pytest.mark.parametrize("over, expected", LINEAR_BAD, ids=lambda v: str(v)[:60])
def test_linear_refuses(bl, over, expected):
    assert status(bl, "bilstm_linear", pack(bl.sequence._LINEAR, linear_args(**over))) == expected
    assert bl.last_error().startswith("linear:")


def test_linear_accepts_what_the_header_allows(bl):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are numbers: nothing may be launched")
    form = bl.sequence._LINEAR
    for over in (dict(), dict(bias=(0, 0), residual=(0, 0, 0)), dict(y=(4 * P, 64 * 48, 48)), dict(SCALED),
                 dict(SCALED, eight=2, type=0), dict(x=(P, 64 * 64, 64), y=(P + 64, 64 * 64 - 32, 64), outputs=32,
                                                    weight=(2 * P, 32 * 32, 32), bias=(0, 0), residual=(0, 0, 0))):
        assert status(bl, "bilstm_linear", pack(form, linear_args(**over))) == "BILSTM_UNSUPPORTED"
        assert "no HIP device" in bl.last_error()
    assert status(bl, "bilstm_linear", pack(form, linear_args(rows=0))) == "BILSTM_OK"


def scratch_of(bl, name, packed):
    need = ctypes.c_uint64(1)
    assert getattr(bl.library(), name)(packed, ctypes.byref(need)) == 0
    return need.value


def test_scratch_is_checked(bl):
    """What a call needs beyond its outputs: one byte less, misaligned, over an input or an output is refused."""
    form = bl.sequence._LINEAR
    f = dict(rows=8, inputs=8192, outputs=64, x=(P, 8 * 8192, 8192), weight=(2 * P, 64 * 8192, 8192), bias=(0, 0),
             residual=(0, 0, 0), y=(5 * P, 8 * 64, 64))
    need = scratch_of(bl, "bilstm_linear_scratch", pack(form, linear_args(**f)))
    assert need > 0
    for scratch, expected in (((20 * P, need - 1), "BILSTM_BUFFER_LENGTH"), ((0, 0), "BILSTM_INVALID_ARGUMENT"),
                              ((20 * P + 8, need), "BILSTM_INVALID_ARGUMENT"), ((P, need), "BILSTM_INVALID_ARGUMENT"),
                              ((5 * P, need), "BILSTM_INVALID_ARGUMENT")):
        assert status(bl, "bilstm_linear", pack(form, linear_args(**f, scratch=scratch))) == expected
    form = bl.sequence._ATTENTION
    f = dict(rows=2, memory_rows=200000, sequences=1, places=1, q=(P, 256, 128), k=(200 * P, 200000 * 64, 64),
             v=(300 * P, 200000 * 64, 64), starts=(4 * P, 2), slots=(0, 0), memory_starts=(6 * P, 2), memory_lengths=(0, 0),
             mask=(0, 0), y=(9 * P, 256, 128))
    need = scratch_of(bl, "bilstm_cross_attention_scratch", pack(form, attention_args(**f)))
    assert need > 0
    for scratch, expected in (((20 * P, need - 1), "BILSTM_BUFFER_LENGTH"), ((0, 0), "BILSTM_INVALID_ARGUMENT"),
                              ((20 * P + 4, need), "BILSTM_INVALID_ARGUMENT"), ((P, need), "BILSTM_INVALID_ARGUMENT"),
                              ((9 * P, need), "BILSTM_INVALID_ARGUMENT")):
        assert status(bl, "bilstm_cross_attention", pack(form, attention_args(**f, scratch=scratch))) == expected
    assert scratch_of(bl, "bilstm_cross_attention_scratch", pack(form, attention_args(rows=0))) == 0
    assert scratch_of(bl, "bilstm_cross_attention_step_scratch", pack(form, attention_args(rows=0))) == 0
    assert scratch_of(bl, "bilstm_linear_scratch", pack(bl.sequence._LINEAR, linear_args(rows=0))) == 0


@pytest.mark.parametrize("name", ["bilstm_cross_attention", "bilstm_cross_attention_step", "bilstm_linear"])
def test_no_arguments(bl, name):
    assert bl.STATUS[getattr(bl.library(), name)(None, None)] == "BILSTM_INVALID_ARGUMENT"


@pytest.mark.parametrize("name", ["bilstm_cross_attention_scratch", "bilstm_cross_attention_step_scratch",
                                  "bilstm_linear_scratch"])
def test_scratch_without_arguments(bl, name):
    need = ctypes.c_uint64()
    assert bl.STATUS[getattr(bl.library(), name)(None, ctypes.byref(need))] == "BILSTM_INVALID_ARGUMENT"
    packed = pack(bl.sequence._LINEAR, linear_args()) if "linear" in name else pack(bl.sequence._ATTENTION, attention_args())
    assert bl.STATUS[getattr(bl.library(), name)(packed, None)] == "BILSTM_INVALID_ARGUMENT"


def test_binding_refuses(bl):
    """What the binding sees before a device: host tensors, unknown names."""
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="CUDA"):
        bl.linear(x, x)
    with pytest.raises(TypeError, match="CUDA"):
        bl.cross_attention(x.view(4, 1, 8), x.view(4, 1, 8), x.view(4, 1, 8), torch.zeros(2, dtype=torch.int32),
                           torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="seq_starts"):
        bl.cross_attention(x, x, x, None, x)

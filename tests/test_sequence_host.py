"""Refusals of the causal sequence operators: the entry points check their arguments before they
touch a device, so this runs without a GPU. Pointers are numbers that nothing reads."""

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


def conv_args(**over):
    """64 rows of 32 channels in 3 sequences, 4 taps, a cache of 5 places."""
    f = dict(device=0, type=0, rows=64, channels=32, taps=4, sequences=3, places=5, silu=1, reserved=0,
             x=(P, 64 * 32, 32), weight=(2 * P, 128), bias=(3 * P, 32), starts=(4 * P, 4), state=(5 * P, 5 * 96),
             slots=(6 * P, 3), fresh=(7 * P, 3), y=(8 * P, 64 * 32, 32))
    f.update(over)
    return f


def pack(form, f):
    flat = []
    for v in f.values():
        flat.extend(v if isinstance(v, tuple) else (v,))
    return form.pack(*flat)


CONV_BAD = [
    (dict(type=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(type=-1), "BILSTM_INVALID_ARGUMENT"),
    (dict(channels=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(taps=1), "BILSTM_UNSUPPORTED"),
    (dict(taps=5), "BILSTM_UNSUPPORTED"),
    (dict(rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(sequences=(1 << 30) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(reserved=1), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(0, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P + 2, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P, 64 * 32 - 1, 32)), "BILSTM_BUFFER_LENGTH"),
    (dict(x=(P, 1 << 62, 31)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P, 1 << 62, 1 << 60)), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(weight=(2 * P, 127)), "BILSTM_BUFFER_LENGTH"),
    (dict(weight=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(bias=(3 * P, 31)), "BILSTM_BUFFER_LENGTH"),
    (dict(starts=(4 * P, 3)), "BILSTM_BUFFER_LENGTH"),
    (dict(starts=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(state=(5 * P, 4 * 96)), "BILSTM_BUFFER_LENGTH"),
    (dict(state=(0, 0)), "BILSTM_INVALID_ARGUMENT"),  # slots without a state
    (dict(slots=(6 * P, 2)), "BILSTM_BUFFER_LENGTH"),
    (dict(slots=(0, 0), places=2, state=(5 * P, 2 * 96)), "BILSTM_INVALID_ARGUMENT"),
    (dict(fresh=(7 * P, 4)), "BILSTM_BUFFER_LENGTH"),
    (dict(y=(P + 64 * 32 * 4 - 4, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # one element shared with x
    (dict(y=(5 * P, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # the state
    (dict(y=(2 * P, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # the weights
    (dict(x=(P, 64 * 64, 64), y=(P + 124, 64 * 64, 64)), "BILSTM_INVALID_ARGUMENT"),  # columns 0..31 and 31..62
]


@pytest.mark.parametrize("over, expected", CONV_BAD, ids=lambda v: str(v)[:60])
def test_conv_refuses(bl, over, expected):
    assert status(bl, "bilstm_causal_conv", pack(bl.sequence._CONV, conv_args(**over))) == expected
    assert bl.last_error().startswith("causal_conv:")


def test_conv_step_refuses(bl):
    step = dict(slots=(6 * P, 64), places=64, state=(5 * P, 64 * 96))
    form = bl.sequence._CONV
    assert status(bl, "bilstm_causal_conv_step", pack(form, conv_args(**step, taps=7))) == "BILSTM_UNSUPPORTED"
    over = dict(step, state=(0, 0))
    assert status(bl, "bilstm_causal_conv_step", pack(form, conv_args(**over))) == "BILSTM_INVALID_ARGUMENT"
    over = dict(step, slots=(6 * P, 63))
    assert status(bl, "bilstm_causal_conv_step", pack(form, conv_args(**over))) == "BILSTM_BUFFER_LENGTH"
    assert bl.STATUS[bl.library().bilstm_causal_conv_step(None, None)] == "BILSTM_INVALID_ARGUMENT"


def test_conv_accepts_what_the_header_allows(bl):
    """Sound arguments pass every check: without a device the call then says so, and nothing was read."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are numbers: nothing may be launched")
    form = bl.sequence._CONV
    for over in (dict(), dict(bias=(0, 0)), dict(state=(0, 0), slots=(0, 0), fresh=(0, 0)),
                 dict(x=(P, 64 * 64, 64), y=(P + 128, 64 * 64, 64)),  # columns side by side
                 dict(x=(P, 63 * 100 + 32, 100))):
        assert status(bl, "bilstm_causal_conv", pack(form, conv_args(**over))) == "BILSTM_UNSUPPORTED"
        assert "no HIP device" in bl.last_error()
    # nothing to do: no device is needed
    assert status(bl, "bilstm_causal_conv", pack(form, conv_args(rows=0))) == "BILSTM_OK"
    assert status(bl, "bilstm_causal_conv", pack(form, conv_args(sequences=0, starts=(0, 0)))) == "BILSTM_OK"


def scan_args(**over):
    """64 rows of 4 heads of 64 channels and 32 states in 3 sequences, a cache of 5 places."""
    f = dict(device=0, type=1, rows=64, heads=4, width=64, groups=2, states=32, sequences=3, places=5, softplus=1,
             reserved=0, x=(P, 64 * 256, 256), dt=(2 * P, 64 * 4, 4), b=(3 * P, 64 * 64, 64), c=(4 * P, 64 * 64, 64),
             z=(5 * P, 64 * 256, 256), a=(6 * P, 4), d=(7 * P, 4), dt_bias=(8 * P, 4), starts=(9 * P, 4),
             state=(10 * P, 5 * 4 * 64 * 32), slots=(12 * P, 3), fresh=(13 * P, 3), y=(14 * P, 64 * 256, 256),
             scratch=(20 * P, 1 << 30))
    f.update(over)
    return f


SCAN_BAD = [
    (dict(type=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(heads=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(groups=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(groups=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(width=48), "BILSTM_UNSUPPORTED"),
    (dict(heads=1 << 20), "BILSTM_DIMENSION_OVERFLOW"),  # 2^31 floats a state
    (dict(states=8), "BILSTM_UNSUPPORTED"),
    (dict(states=512), "BILSTM_UNSUPPORTED"),
    (dict(rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(sequences=(1 << 30) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(reserved=1), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P + 1, 64 * 256, 256)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P, 64 * 256 - 1, 256)), "BILSTM_BUFFER_LENGTH"),
    (dict(dt=(2 * P, 64 * 4, 3)), "BILSTM_INVALID_ARGUMENT"),
    (dict(dt=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(b=(3 * P, 64 * 63, 63)), "BILSTM_INVALID_ARGUMENT"),
    (dict(c=(4 * P, 100, 64)), "BILSTM_BUFFER_LENGTH"),
    (dict(z=(5 * P, 100, 256)), "BILSTM_BUFFER_LENGTH"),
    (dict(a=(6 * P, 3)), "BILSTM_BUFFER_LENGTH"),
    (dict(a=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(d=(7 * P, 5)), "BILSTM_BUFFER_LENGTH"),
    (dict(dt_bias=(8 * P + 2, 4)), "BILSTM_INVALID_ARGUMENT"),
    (dict(starts=(9 * P, 3)), "BILSTM_BUFFER_LENGTH"),
    (dict(state=(10 * P, 5 * 4 * 64 * 32 - 1)), "BILSTM_BUFFER_LENGTH"),
    (dict(state=(10 * P + 4, 5 * 4 * 64 * 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(state=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(slots=(12 * P, 4)), "BILSTM_BUFFER_LENGTH"),
    (dict(fresh=(13 * P, 2)), "BILSTM_BUFFER_LENGTH"),
    (dict(y=(P, 64 * 256, 256)), "BILSTM_INVALID_ARGUMENT"),
    (dict(y=(5 * P, 64 * 256, 256)), "BILSTM_INVALID_ARGUMENT"),
    (dict(state=(P, 5 * 4 * 64 * 32)), "BILSTM_INVALID_ARGUMENT"),
]


@pytest.mark.parametrize("over, expected", SCAN_BAD, ids=lambda v: str(v)[:60])
def test_scan_refuses(bl, over, expected):
    assert status(bl, "bilstm_scan", pack(bl.sequence._SCAN, scan_args(**over))) == expected
    assert bl.last_error().startswith("scan:")


def test_scan_step_refuses(bl):
    step = dict(slots=(12 * P, 64))
    form = bl.sequence._SCAN
    assert status(bl, "bilstm_scan_step", pack(form, scan_args(**step, state=(0, 0)))) == "BILSTM_INVALID_ARGUMENT"
    assert status(bl, "bilstm_scan_step", pack(form, scan_args(slots=(12 * P, 3)))) == "BILSTM_BUFFER_LENGTH"
    assert status(bl, "bilstm_scan_step", pack(form, scan_args(slots=(0, 0)))) == "BILSTM_INVALID_ARGUMENT"
    assert status(bl, "bilstm_scan_step", pack(form, scan_args(**step, width=16))) == "BILSTM_UNSUPPORTED"


def test_scan_scratch(bl):
    """None for whole sequences; else a state and a decay for every block of as many rows as a run has, and
    a state for every sequence that can be split."""
    need = ctypes.c_uint64()
    form = bl.sequence._SCAN

    def scratch(**sizes):
        f = dict(rows=4096, heads=64, width=64, groups=1, states=128, sequences=1)
        f.update(sizes)
        assert bl.library().bilstm_scan_scratch(pack(form, scan_args(**f)), ctypes.byref(need)) == 0
        return need.value

    def bytes_of(blocks, first):
        return ((blocks + first) * 64 * 64 * 128 + blocks * 64) * 4

    assert scratch() == bytes_of(4096 // 256, 1)
    assert scratch(rows=90) == 0 and scratch(rows=0) == 0 and scratch(sequences=0, rows=64) == 0
    assert scratch(rows=4096, sequences=1024) == bytes_of(16, 17)  # one of them may have all the rows
    assert scratch(rows=16384, sequences=24) == bytes_of(21, 22)
    assert scratch(rows=65536, sequences=256) == bytes_of(85, 86)
    bad = pack(form, scan_args(width=7))
    assert bl.STATUS[bl.library().bilstm_scan_scratch(bad, ctypes.byref(need))] == "BILSTM_UNSUPPORTED"


@pytest.mark.parametrize("name", ["bilstm_causal_conv", "bilstm_causal_conv_step", "bilstm_scan", "bilstm_scan_step",
                                  "bilstm_add_rms_norm", "bilstm_token_logprobs"])
def test_no_arguments(bl, name):
    assert bl.STATUS[getattr(bl.library(), name)(None, None)] == "BILSTM_INVALID_ARGUMENT"


def norm_args(**over):
    """64 rows of 32 with a residual and an e4m3 output."""
    f = dict(device=0, type=1, rows=64, width=32, eight=1, eps=1e-5, reserved=0, x=(P, 64 * 32, 32),
             residual=(2 * P, 64 * 32, 32), weight=(3 * P, 32), residual_out=(4 * P, 64 * 32, 32), y=(0, 0, 0),
             q=(5 * P, 64 * 32, 32), scales=(6 * P, 64))
    f.update(over)
    return f


NORM_BAD = [
    (dict(type=9), "BILSTM_INVALID_ARGUMENT"),
    (dict(eight=3), "BILSTM_INVALID_ARGUMENT"),
    (dict(width=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(eps=-1e-6), "BILSTM_INVALID_ARGUMENT"),
    (dict(eps=float("nan")), "BILSTM_INVALID_ARGUMENT"),
    (dict(eps=float("inf")), "BILSTM_INVALID_ARGUMENT"),
    (dict(reserved=2), "BILSTM_INVALID_ARGUMENT"),
    (dict(rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(x=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(x=(P + 1, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(residual=(2 * P, 64 * 32 - 1, 32)), "BILSTM_BUFFER_LENGTH"),
    (dict(weight=(3 * P, 33)), "BILSTM_BUFFER_LENGTH"),
    (dict(scales=(6 * P, 63)), "BILSTM_BUFFER_LENGTH"),
    (dict(scales=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(q=(0, 0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(eight=0), "BILSTM_INVALID_ARGUMENT"),  # q and scales without a type
    (dict(eight=0, q=(0, 0, 0), scales=(0, 0)), "BILSTM_INVALID_ARGUMENT"),  # no output at all
    (dict(q=(P, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # 8-bit rows over x
    (dict(residual_out=(2 * P + 2, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # the residual, one element on
    (dict(residual_out=(2 * P, 64 * 33, 33)), "BILSTM_INVALID_ARGUMENT"),  # the residual with another stride
    (dict(y=(4 * P, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # two outputs in one place
    (dict(y=(3 * P, 64 * 32, 32)), "BILSTM_INVALID_ARGUMENT"),  # the weights
    (dict(scales=(5 * P + 64, 64)), "BILSTM_INVALID_ARGUMENT"),  # inside q
]


@pytest.mark.parametrize("over, expected", NORM_BAD, ids=lambda v: str(v)[:60])
def test_norm_refuses(bl, over, expected):
    assert status(bl, "bilstm_add_rms_norm", pack(bl.sequence._NORM, norm_args(**over))) == expected
    assert bl.last_error().startswith("add_rms_norm:")


def logprob_args(**over):
    """16 rows of 20000 tokens, two given, top 4."""
    f = dict(device=0, type=0, rows=16, vocabulary=20000, given=2, top=4, reserved=0, logits=(P, 16 * 20000, 20000),
             tokens=(4 * P, 32), logprobs=(5 * P, 32), entropy=(6 * P, 16), top_tokens=(7 * P, 64),
             top_logprobs=(8 * P, 64), scratch=(9 * P, 16 * 3 * 48))
    f.update(over)
    return f


LOGPROB_BAD = [
    (dict(type=4), "BILSTM_INVALID_ARGUMENT"),
    (dict(vocabulary=0), "BILSTM_INVALID_ARGUMENT"),
    (dict(vocabulary=(1 << 20) + 1), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(rows=1 << 31), "BILSTM_DIMENSION_OVERFLOW"),
    (dict(top=33), "BILSTM_INVALID_ARGUMENT"),
    (dict(vocabulary=3), "BILSTM_INVALID_ARGUMENT"),  # top 4 of 3
    (dict(given=1025), "BILSTM_INVALID_ARGUMENT"),
    (dict(reserved=1), "BILSTM_INVALID_ARGUMENT"),
    (dict(logits=(P + 2, 16 * 20000, 20000)), "BILSTM_INVALID_ARGUMENT"),
    (dict(logits=(P, 16 * 20000 - 1, 20000)), "BILSTM_BUFFER_LENGTH"),
    (dict(tokens=(4 * P + 4, 32)), "BILSTM_INVALID_ARGUMENT"),
    (dict(tokens=(4 * P, 31)), "BILSTM_BUFFER_LENGTH"),
    (dict(logprobs=(5 * P, 16)), "BILSTM_BUFFER_LENGTH"),
    (dict(entropy=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(top_tokens=(7 * P, 63)), "BILSTM_BUFFER_LENGTH"),
    (dict(top_logprobs=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(scratch=(9 * P, 16 * 3 * 48 - 1)), "BILSTM_BUFFER_LENGTH"),
    (dict(scratch=(9 * P + 8, 1 << 20)), "BILSTM_INVALID_ARGUMENT"),
    (dict(scratch=(0, 0)), "BILSTM_INVALID_ARGUMENT"),
    (dict(entropy=(P, 16)), "BILSTM_INVALID_ARGUMENT"),
    (dict(top_logprobs=(7 * P, 64)), "BILSTM_INVALID_ARGUMENT"),
]


@pytest.mark.parametrize("over, expected", LOGPROB_BAD, ids=lambda v: str(v)[:60])
def test_logprobs_refuse(bl, over, expected):
    assert status(bl, "bilstm_token_logprobs", pack(bl.sequence._LOGPROBS, logprob_args(**over))) == expected
    assert bl.last_error().startswith("token_logprobs")


def test_logprobs_scratch(bl):
    """Tiles of 8192 float32 or 16384 16-bit logits whose rows may start up to 3 or 7 tokens into a
    vector; 16 bytes and a key of 8 for each top token a tile; none where one launch is enough."""
    need = ctypes.c_uint64()
    for kind, sizes in ((0, ((1024, 0), (1025, 0), (8189, 0), (8190, 2), (20000, 3), (1 << 20, 129))),
                        (1, ((1024, 0), (8190, 0), (16377, 0), (16378, 2), (20000, 2), (1 << 20, 65)))):
        for vocabulary, tiles in sizes:
            packed = pack(bl.sequence._LOGPROBS, logprob_args(type=kind, vocabulary=vocabulary))
            assert bl.library().bilstm_token_logprobs_scratch(packed, ctypes.byref(need)) == 0
            assert need.value == 16 * tiles * (16 + 8 * 4)


def test_sound_arguments_reach_the_device(bl):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are numbers: nothing may be launched")
    for over in (dict(), dict(residual_out=(2 * P, 64 * 32, 32)), dict(y=(P, 64 * 32, 32)),
                 dict(residual=(0, 0, 0), residual_out=(0, 0, 0))):
        assert status(bl, "bilstm_add_rms_norm", pack(bl.sequence._NORM, norm_args(**over))) == "BILSTM_UNSUPPORTED"
    for over in (dict(), dict(given=0, tokens=(0, 0), logprobs=(0, 0)), dict(vocabulary=500, scratch=(0, 0))):
        assert status(bl, "bilstm_token_logprobs", pack(bl.sequence._LOGPROBS, logprob_args(**over))) == "BILSTM_UNSUPPORTED"
    for over in (dict(), dict(z=(0, 0, 0), d=(0, 0), dt_bias=(0, 0)), dict(state=(0, 0), slots=(0, 0), fresh=(0, 0))):
        assert status(bl, "bilstm_scan", pack(bl.sequence._SCAN, scan_args(**over))) == "BILSTM_UNSUPPORTED"
        assert "no HIP device" in bl.last_error()
    assert status(bl, "bilstm_scan", pack(bl.sequence._SCAN, scan_args(rows=0))) == "BILSTM_OK"
    assert status(bl, "bilstm_add_rms_norm", pack(bl.sequence._NORM, norm_args(rows=0))) == "BILSTM_OK"
    assert status(bl, "bilstm_token_logprobs", pack(bl.sequence._LOGPROBS, logprob_args(rows=0))) == "BILSTM_OK"


def test_structures_have_the_header_sizes(bl):
    """The packed layouts are the C structures of bilstm.h: 4- and 8-byte members without holes."""
    assert ctypes.sizeof(ctypes.c_void_p) == 8
    assert bl.sequence._CONV.size == 40 + 2 * 24 + 6 * 16
    assert bl.sequence._SCAN.size == 48 + 6 * 24 + 8 * 16
    assert bl.sequence._NORM.size == 32 + 5 * 24 + 2 * 16
    assert bl.sequence._LOGPROBS.size == 32 + 24 + 6 * 16


def test_binding_refuses_before_the_library(bl):
    import torch
    x = torch.zeros(4, 8)
    starts = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        bl.causal_conv(x, torch.zeros(8, 4), starts)
    with pytest.raises(TypeError):
        bl.causal_conv_step(x, torch.zeros(8, 4), torch.zeros(4, 3, 8))
    with pytest.raises(TypeError):
        bl.add_rms_norm(x, torch.ones(8))
    with pytest.raises(TypeError):
        bl.token_logprobs(x, torch.zeros(4, dtype=torch.int64))


def test_steps_ignore_what_the_header_says(bl):
    """starts, fresh and the number of sequences are not read in the single-token forms, whatever they hold."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are numbers: nothing may be launched")
    conv = dict(slots=(6 * P, 64), places=64, state=(5 * P, 64 * 96))
    scan = dict(slots=(12 * P, 64))
    for over in (dict(), dict(starts=(8 * P, 1), fresh=(8 * P, 7)), dict(starts=(5 * P + 1, 1 << 40), fresh=(5 * P, 1)),
                 dict(sequences=(1 << 32) - 1)):
        args = pack(bl.sequence._CONV, conv_args(**conv, **over))
        assert status(bl, "bilstm_causal_conv_step", args) == "BILSTM_UNSUPPORTED", bl.last_error()
        assert "no HIP device" in bl.last_error()
        args = pack(bl.sequence._SCAN, scan_args(**scan, **over))
        assert status(bl, "bilstm_scan_step", args) == "BILSTM_UNSUPPORTED", bl.last_error()
        assert "no HIP device" in bl.last_error()


def _long_scan(**over):
    """4096 rows of 64 heads, two sequences: long enough that sequences are split and scratch is needed."""
    f = dict(rows=4096, heads=64, width=64, groups=1, states=32, sequences=2, places=5, x=(P, 4096 * 4096, 4096),
             dt=(64 * P, 4096 * 64, 64), b=(65 * P, 4096 * 32, 32), c=(66 * P, 4096 * 32, 32), z=(0, 0, 0), a=(67 * P, 64),
             d=(0, 0), dt_bias=(0, 0), starts=(68 * P, 3), state=(70 * P, 5 * 4096 * 32), slots=(80 * P, 2),
             fresh=(81 * P, 2), y=(128 * P, 4096 * 4096, 4096), scratch=(256 * P, 1 << 40))
    f.update(over)
    return scan_args(**f)


def test_scan_scratch_is_checked(bl):
    """What a split sequence writes to scratch stays inside it and apart from everything else."""
    import torch
    form, need = bl.sequence._SCAN, ctypes.c_uint64()
    assert bl.library().bilstm_scan_scratch(pack(form, _long_scan()), ctypes.byref(need)) == 0
    assert need.value > 0
    for scratch, expected in (((256 * P, need.value - 1), "BILSTM_BUFFER_LENGTH"),
                              ((256 * P, 0), "BILSTM_BUFFER_LENGTH"),
                              ((0, 0), "BILSTM_INVALID_ARGUMENT"),
                              ((0, need.value), "BILSTM_INVALID_ARGUMENT"),
                              ((256 * P + 8, need.value), "BILSTM_INVALID_ARGUMENT"),
                              ((P, need.value), "BILSTM_INVALID_ARGUMENT"),  # x
                              ((65 * P, need.value), "BILSTM_INVALID_ARGUMENT"),  # b and what follows
                              ((70 * P + 5 * 4096 * 32 * 4 - 16, need.value), "BILSTM_INVALID_ARGUMENT"),  # the state's last floats
                              ((128 * P - need.value // 16 * 16 + 16, need.value), "BILSTM_INVALID_ARGUMENT"),  # into y
                              ((128 * P, need.value), "BILSTM_INVALID_ARGUMENT")):
        assert status(bl, "bilstm_scan", pack(form, _long_scan(scratch=scratch))) == expected, scratch
        assert bl.last_error().startswith("scan:")
    if not torch.cuda.is_available():  # else something would be launched
        for scratch in ((256 * P, need.value), (256 * P, need.value + 5)):
            assert status(bl, "bilstm_scan", pack(form, _long_scan(scratch=scratch))) == "BILSTM_UNSUPPORTED"
            assert "no HIP device" in bl.last_error()
        # sequences that are not split need none, whatever is passed for it
        for scratch in ((0, 0), (256 * P + 1, 3)):
            short = scan_args(scratch=scratch)
            assert status(bl, "bilstm_scan", pack(form, short)) == "BILSTM_UNSUPPORTED"

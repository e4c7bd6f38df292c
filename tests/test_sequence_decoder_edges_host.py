"""Refusals at the edges of what cross attention takes; without a GPU, as in test_sequence_decoder_host.py."""

import pytest
import torch

from tests.test_sequence_decoder_host import attention_args, bl, pack, status  # noqa: F401


@pytest.mark.parametrize("scale", [2.0 ** 127, 1e-40])
def test_scales_up_to_2_to_the_127th(bl, scale):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("the pointers are numbers: nothing may be launched")
    assert status(bl, "bilstm_cross_attention", pack(bl.sequence._ATTENTION, attention_args(scale=scale))) == "BILSTM_UNSUPPORTED"
    assert "no HIP device" in bl.last_error()


def test_larger_scales_are_refused(bl):  # noqa: F811
    """Their product with log2 e leaves float32."""
    for scale in (1.8e38, 2.9e38):
        assert status(bl, "bilstm_cross_attention", pack(bl.sequence._ATTENTION, attention_args(scale=scale))) == "BILSTM_INVALID_ARGUMENT"
        assert "scale" in bl.last_error()

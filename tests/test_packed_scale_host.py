"""svdq_attention refuses scales whose multiple by log2 e leaves fp32's range, before any device is touched."""
import pytest

import bit_diffusion_amd as bd

FAKE = 1 << 20


def call(scale):
    return bd.lib().svdq_attention(5, 7, 4, 2, 64, 2, scale, 0.0, 0, FAKE, FAKE, None, None, FAKE, 256, FAKE, 128, FAKE, 128, 2 * FAKE, 100,
                                   None, 0, None)


@pytest.mark.parametrize("scale,status,word", [(2.0 ** 127 * (1 + 2.0 ** -23), bd.SVDQ_ERR_UNSUPPORTED_CONFIG, "scale"),
                                               (3.4e38, bd.SVDQ_ERR_UNSUPPORTED_CONFIG, "scale"), (float("inf"), bd.SVDQ_ERR_INVALID_ARG, "scale"),
                                               (2.0 ** 127, bd.SVDQ_ERR_INVALID_ARG, "out_stride"), (2.0 ** -149, bd.SVDQ_ERR_INVALID_ARG, "out_stride")])
def test_scale(scale, status, word):
    """The last two pass this check and fail at the result's rows, which are too close."""
    assert call(scale) == status
    assert word in bd.svdq_last_error()

"""Sizes at the ends of their types (CPU only): refused before anything is enqueued."""
import pytest

import gated_deltanet_chunked_rule_amd as gdr
from gated_deltanet_chunked_rule_amd import layer


def fake(n):   # aligned, never dereferenced: validation fails first
    return 0x10000 * (n + 1)


def last():
    return gdr.load_library().gdr_last_error().decode()


@pytest.mark.parametrize("D", [2 ** 30 + 1, 2 ** 31 - 600, 2 ** 31 - 8, 2 ** 31 - 1])
def test_convolution_refuses_channels_whose_numbers_leave_an_int(D):
    # D + 7 and the step's D + 511 are formed in 32 bits
    sh = layer._ConvShape(1, 1, D, 4, 0, 0, 1, 0)
    f, s = layer._entry("gdr_causal_conv_fwd"), layer._entry("gdr_causal_conv_step")
    assert f(sh, fake(0), fake(1), None, None, None, fake(2), None, None) == -2 and "2^30" in last()
    assert s(sh, fake(0), fake(1), None, fake(2), 4, None, fake(3), None) == -2 and "2^30" in last()
    assert layer._entry("gdr_causal_conv_bwd_workspace_size")(sh) == 0

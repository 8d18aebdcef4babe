"""Sizes of the convolution that 32 bits cannot hold (CPU only, tensors without
storage): refused, where their low 32 bits would be taken for a size."""
import torch

import gated_deltanet_chunked_rule_amd as gdr
from test_block_refusals import OnDevice
from test_layer_refusals import raises


def test_convolution_refuses_sizes_beyond_32_bits():
    m = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="meta").as_subclass(OnDevice)  # noqa: E731
    n = 2 ** 32 + 8
    x, w = m(1, n, 8), m(8, 4)
    raises("T must be below", gdr.gdr_causal_conv_fwd, x, w)
    raises("T must be below", gdr.gdr_causal_conv_bwd, x, w, None, x)
    raises("T must be below", gdr.causal_conv, x, w)
    raises("B must be below", gdr.gdr_causal_conv_fwd, m(n, 1, 8), w)
    raises("D must be below", gdr.gdr_causal_conv_fwd, m(1, 1, n), m(n, 4))
    raises("rows must be below", gdr.gdr_causal_conv_step, x[0], m(n, 3, 8), w)

"""Pools of states and tables of offsets that 32 bits cannot count (CPU only,
tensors without storage)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
from gated_deltanet_chunked_rule_amd import layer
from test_block_refusals import OnDevice
from test_layer_refusals import raises


def meta(*s, dtype=torch.float32):
    return torch.empty(*s, dtype=dtype, device="meta").as_subclass(OnDevice)


@pytest.mark.parametrize("n,slots", [(3, 3), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 + 5, 2 ** 31 - 1), (2 ** 32 + 4, 2 ** 31 - 1)])
def test_a_pool_is_as_long_as_slots_can_name(n, slots):
    state = meta(n, 8)
    assert layer._pool(state, "state", (8,), torch.float32, 0, 2, meta(2, dtype=torch.int32))[1] == slots


def test_tables_of_offsets_beyond_32_bits():
    x, A, table = meta(1, 6, 8), meta(8), meta(2 ** 32 + 3, dtype=torch.int32)
    raises("offsets must be below", gdr.gdr_linear_scan_fwd, x, x, x, A, None, table)
    raises("offsets must be below", gdr.gdr_causal_conv_fwd, x, meta(8, 4), None, None, table)

"""The gradient of the linear recurrence where its join does its work: a strand
of it holds several tiles of 48 tokens from 3073 tokens on, and slow decays carry
states and gradients across strands."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import check
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

CASES = [
    # B, T, D, type, cu, largest -A
    (1, 7000, 6, F32, None, 1e-3),
    (1, 7000, 6, BF, None, 1e-3),
    (1, 7100, 18, F32, [0, 40, 3500, 3500, 7093], 2e-3),     # ends inside tiles, an empty one, tokens behind the last
    (1, 7100, 33, BF, [5, 2400, 2401, 7100], 2e-3),
    (2, 3600, 3, F32, None, 1e-3),                            # the second row starts at a tile's first token
    (1, 6300, 130, BF, [0, 6300], 0.05),                      # two columns of channels
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_gradient_across_strands(k):
    B, T, D, dtype, cu, most = CASES[k]
    g = gen(1300 + k)
    N = B if cu is None else len(cu) - 1
    x, r, i, dy = (randn(g, B, T, D, dtype=dtype) for _ in range(4))
    A, h0, dht = -most * torch.rand(D, generator=g), randn(g, N, D), randn(g, N, D)
    table = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, ht = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i, A, h0)), table, output_final_state=True)
    got = gdr.gdr_linear_scan_bwd(*(cuda(t) for t in (x, r, i, A, dy, h0, dht)), table)
    ry, rye, rh, rhe, _, _ = ref.linear_scan(x, r, i, A, h0, cu)
    check(y, ry, rye, "y")
    check(ht, rh, rhe, "final state")
    for name, t, (v, b) in zip(("dx", "dr", "di", "dA", "dh0"), got, ref.linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)):
        check(t, v, b, name)

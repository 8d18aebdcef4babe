"""The gradient of the norms around a block where its persistent workgroups take
more than one step of several rows each, the last one ragged.

A sum of rows is added from a lane's steps (3 at most here), a workgroup's rows
(16), and partial rows of 512 workgroups in 64 strands of 8: 90 roundings of
2^-24 at most, 2^-17 of the magnitudes, beside the 2^-18 that the reference's
bound has for each of them."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import check
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# 512 workgroups of 16, 8, 4 and 2 rows
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,dim", [(8200, 100), (16391, 128), (4103, 200), (2050, 500), (4099, 300), (1027, 1000)])
def test_second_steps_of_several_rows(rows, dim, dtype):
    g = gen(rows + dim)
    x, gate, dy, dres = (randn(g, rows, dim, dtype=dtype) for _ in range(4))
    residual = randn(g, rows, dim, dtype=dtype, std=2.0)
    post, pre, scale = ((1 + randn(g, dim, std=0.1)).to(dtype), (1 + randn(g, dim, std=0.1)).to(dtype), randn(g, dim, std=0.5).to(dtype))
    h = ref.block_norm(x, post, residual, pre, gate, scale)[2].to(dtype)
    got = gdr.gdr_block_norm_bwd(*(cuda(t) for t in (x, post, h, pre, dy, gate, scale, dres)), eps=ref.EPS)
    want = ref.block_norm_bwd(x, post, h, pre, dy, gate, scale, dres)
    for name, t, (v, b) in zip(("dx", "dh", "dpost", "dpre", "dgate", "dscale"), got, want):
        check(t, v, 3 * b if t.dim() == 1 else b, name)
    bad = [t.clone() for t in (x, h, dy)]
    bad[0][rows - 1, 3] = bad[1][rows - 1, 3] = bad[2][rows - 1, 3] = float("nan")     # in the last step
    again = gdr.gdr_block_norm_bwd(*(cuda(t) for t in (bad[0], post, bad[1], pre, bad[2], gate, scale, dres)), eps=ref.EPS)
    for k in (0, 1, 4):
        assert torch.equal(again[k][:-1], got[k][:-1])

"""Norms with eps = 0 of rows whose mean square lies below fp32's normal numbers.

The squares' sum is then held in steps of 2^-149: each of its n additions is off
by 2^-150 at most, and so is the mean, 2^-149 in all, so that the root's
reciprocal is off by delta = 2^-150 / mean beside its own roundings.  An output
that is of degree k in it is off by k delta more."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import SLACK, check
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(7, 60), (40, 128), (33, 300), (9, 1000), (5, 2048), (4, 4096), (3, 6000), (2, 9000)]


def delta(t):
    return 2.0 ** -150 / float(t.double().square().mean(-1).min())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("small", ["x", "h"])
def test_block_norm_of_tiny_rows(rows, dim, dtype, small):
    g = gen(rows + dim)
    tiny, one = 2e-20, 1.0
    x = randn(g, rows, dim, std=tiny if small == "x" else one).to(dtype)
    residual = randn(g, rows, dim, std=tiny if small == "h" else one).to(dtype)
    post = ((1 + randn(g, dim, std=0.1)) * (tiny if small == "h" else one)).to(dtype)
    pre, gate, dy = (1 + randn(g, dim, std=0.1)).to(dtype), randn(g, rows, dim).to(dtype), randn(g, rows, dim).to(dtype)
    y, h = gdr.gdr_block_norm_fwd(*(cuda(t) for t in (x, post, residual, pre, gate)), eps=0.0)
    ry, rye, rh, rhe = ref.block_norm(x, post, residual, pre, gate, eps=0.0)
    if small == "x":
        off = delta(x) * (rh - residual.double()).abs()
        mean = rh.square().mean(-1, keepdim=True)
        check(y, ry, rye + off * pre.double().abs() / mean.sqrt() + ry.abs() * (rh.abs() * off).mean(-1, keepdim=True) / mean, "y")
        check(h, rh, rhe + off, "h")
    else:
        check(y, ry, rye + delta(rh) * ry.abs(), "y")
        check(h, rh, rhe, "h")
    h = rh.to(dtype)
    got = gdr.gdr_block_norm_bwd(*(cuda(t) for t in (x, post, h, pre, dy, gate)), eps=0.0)
    want = ref.block_norm_bwd(x, post, h, pre, dy, gate, eps=0.0)
    more = 1 + 4 * delta(x if small == "x" else h) / SLACK           # a gradient is of degree three in it
    for name, t, (v, b) in zip(("dx", "dh", "dpost", "dpre", "dgate"), got, want):
        check(t, v, b * more, name)

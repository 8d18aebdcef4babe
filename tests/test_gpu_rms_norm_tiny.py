"""The norm with eps = 0 of rows whose mean square lies below fp32's normal
numbers (test_gpu_norm_tiny.py states what fp32 then holds of it)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
import layer_reference as ref
from layer_reference import gen, randn
from test_gpu_layer import cuda
from test_gpu_norm_tiny import BF, F32, SIZES, delta

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -18


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_rms_norm_of_tiny_rows(rows, dim, dtype):
    g = gen(rows + dim)
    x, residual = (randn(g, rows, dim, std=2e-20).to(dtype) for _ in range(2))
    weight, gate, dy = (1 + randn(g, dim, std=0.1)).to(dtype), randn(g, rows, dim).to(dtype), randn(g, rows, dim).to(dtype)
    ry, my, rh = ref.norm(x, weight, residual, gate, eps=0.0)
    off = delta(rh)
    y, _, h = gdr.gdr_rms_norm_fwd(*(cuda(t) for t in (x, weight, residual, gate)), eps=0.0)
    ref.check(y, ry, my, SLACK + off, "y")
    assert bool(((h.cpu().double() - rh).abs() <= ref.HALF[dtype] * rh.abs()).all())
    q, scales, _ = gdr.gdr_rms_norm_fwd(*(cuda(t) for t in (x, weight, residual, gate)), eps=0.0, quant=True)
    rs, bound = ref.e4m3_parts(ry)
    assert bool(((scales.cpu().double() - rs).abs() <= (SLACK + off) * rs).all())
    wide = scales.cpu().double().repeat_interleave(128, -1)[..., :dim]
    assert bool(((q.cpu().float().double() * wide - ry).abs() <= bound + off * my).all())
    h = h.cpu()
    for name, t, want in zip(("dh", "dw", "dgate"), gdr.gdr_rms_norm_bwd(*(cuda(t) for t in (h, weight, dy, gate)), eps=0.0),
                             ref.norm_bwd(h, weight, dy, gate, eps=0.0)):
        ref.check(t, *want, SLACK + 3 * delta(h), name)      # of degree three at most

"""The norm at sizes where its kernels take another path: short rows two to a
lane group, and gradients whose workgroups walk over several rows each."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
import layer_reference as ref
from layer_reference import check, gen, randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
cuda = lambda t: None if t is None else t.to("cuda")  # noqa: E731


@pytest.mark.parametrize("rows,dim,dtype,residual,gated", [
    (65536, 64, BF, False, False), (65536 + 7, 128, BF, False, True), (65536 + 17, 100, F32, True, False), (65536 + 31, 128, BF, True, True),
    (32768 + 3, 256, BF, False, True), (32768 + 9, 200, F32, True, True), (16384 + 1, 512, BF, True, False), (16384 + 5, 300, F32, False, True),
    (65535, 128, BF, False, True),     # one below: a row a lane group
])
def test_norm_fwd_of_many_short_rows(rows, dim, dtype, residual, gated):
    g = gen(rows + dim)
    x, w = randn(g, rows, dim, dtype=dtype), (1 + randn(g, dim, std=0.2)).to(dtype)
    r = randn(g, rows, dim, dtype=dtype, std=2) if residual else None
    z = randn(g, rows, dim + 8, dtype=dtype)[:, 4:4 + dim] if gated else None
    y, _, h = gdr.gdr_rms_norm_fwd(cuda(x), cuda(w), cuda(r), None if z is None else cuda(z._base)[:, 4:4 + dim])
    check(y, *ref.norm(x, w, r, z)[:2], label="y")
    if residual:
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(dtype))


@pytest.mark.parametrize("rows,dim,dtype,gated,dres", [
    (2 * 16384 + 5, 128, BF, True, False), (16384 + 1, 64, F32, False, True), (8192 * 2 + 3, 256, BF, True, True), (4096 * 2 + 1, 300, F32, True, False),
    (2048 * 3 + 1, 700, BF, False, True), (1024 + 5, 2048, BF, True, True), (1100, 4096, BF, False, True), (600, 4096, F32, True, True),
    (520, 8192, BF, True, True), (300, 9000, BF, True, True), (513, 16384, BF, False, False),
])
def test_norm_bwd_over_several_rows_a_workgroup(rows, dim, dtype, gated, dres):
    g = gen(rows + dim)
    h, dy, w = randn(g, rows, dim, dtype=dtype), randn(g, rows, dim, dtype=dtype), (1 + randn(g, dim, std=0.2)).to(dtype)
    z, s = randn(g, rows, dim, dtype=dtype) if gated else None, randn(g, rows, dim, dtype=dtype) if dres else None
    got = gdr.gdr_rms_norm_bwd(cuda(h), cuda(w), cuda(dy), cuda(z), cuda(s))
    want = ref.norm_bwd(h, w, dy, z, s)
    check(got[0], *want[0], label="dh")
    # about 3 rows a lane, 16 lane groups, 16 workgroups a strand and 64 strands are added one after another: 100
    # roundings of 2^-24, beside those of the terms
    check(got[1], *want[1], slack=2.0 ** -17, label="dw")
    if gated:
        check(got[2], *want[2], label="dgate")

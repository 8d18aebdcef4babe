"""The convolution over nearly 2^31 rows of one token: tiles of tokens and
sequences together are more than an int counts."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
import layer_reference as ref
from layer_reference import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_rows_whose_items_leave_an_int():
    B, W = 0x7fff0000, 2
    fill = lambda seed: torch.empty(B, 1, 1, device="cuda", dtype=BF).normal_(generator=torch.Generator(device="cuda").manual_seed(seed))  # noqa: E731
    x, h0 = fill(1), fill(2)
    w, b = torch.tensor([[0.5, -1.5]], device="cuda", dtype=BF), torch.tensor([0.25], device="cuda", dtype=BF)
    y, ht = gdr.gdr_causal_conv_fwd(x, w, b, h0, output_final_state=True)
    places = [slice(0, 50), slice(B // 2, B // 2 + 50), slice(B - 50, B)]
    for at in places:
        ry, my = ref.conv(x[at], w, b, h0[at])[:2]
        check(y[at], ry, my, label="y")
        assert torch.equal(ht[at], x[at])
    del ht
    dx, _, _, dh0 = gdr.gdr_causal_conv_bwd(x, w, b, y, h0)
    for at in places:
        vx, vh, vw, vb = (t[at].cpu().double() if t.dim() == 3 else t.cpu().double() for t in (x, h0, w, b))
        z = vb + vw[0, 1] * vx + vw[0, 0] * vh
        s = torch.sigmoid(z)
        dz = y[at].cpu().double() * s * (1 + z * (1 - s))
        check(dx[at], dz * vw[0, 1], dz.abs() * 1.5, label="dx")
        check(dh0[at], dz * vw[0, 0], dz.abs() * 0.5, label="dh0")
    del x, h0, y, dx, dh0
    torch.cuda.empty_cache()

"""Accuracy of the layer operators where single terms dominate: bounds that give
each term the rounding that it takes and no more (layer_reference.py has the
plain 64-bit forms)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
import layer_reference as ref
from layer_reference import check, gen, randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def run_scan(c, cu=None, **kw):
    H, P = c["x"].shape[2:]
    G, N = c["B"].shape[2:]
    row = c["row"].to("cuda")
    x, B, C = (t.unflatten(-1, s) for t, s in zip(row.split([H * P, G * N, G * N], -1), ((H, P), (G, N), (G, N))))
    dev = {n: c[n].to("cuda") for n in ("dt", "A", "D", "bias", "h0")}
    return gdr.gdr_ssm_scan_fwd(x, dev["dt"], dev["A"], B, C, dev["D"], dev["bias"], dev["h0"], None if cu is None else cu.to("cuda"),
                                output_final_state=True, **kw)


# -------------------------------------------------------------------- scan --
@pytest.mark.parametrize("T,H,G,P,N,dtype", [(200, 4, 1, 64, 128, BF), (130, 4, 2, 32, 32, BF), (300, 3, 1, 128, 64, BF), (70, 8, 2, 64, 32, BF),
                                             (150, 2, 1, 64, 64, F32)])
def test_scan_skip_term_is_not_rounded_before_the_output(T, H, G, P, N, dtype):
    # D x in fp32: y's own half step, the bf16 roundings of the scan's products (as in test_scan), and a few fp32 ones of D x
    g = gen(400 + T)
    c = ref.scan_inputs(g, 1, T, H, G, P, N, dtype)
    c["D"] = 60 + randn(g, H, std=20.0)
    y, _ = run_scan(c)
    ry, rm, _, _ = ref.scan(*(c[n] for n in ("x", "dt", "A", "B", "C")), None, c["bias"], c["h0"])
    skip = c["D"].double()[:, None] * c["x"].double()
    check(y, ry + skip, rm * (2.0 ** -8 if dtype == BF else 2.0 ** -17) + skip.abs() * 2.0 ** -20, slack=1.0, label="y")
    c["row"][..., H * P + G * N:] = 0       # C = 0: nothing but D x is left
    y, _ = run_scan(c)
    check(y, skip, skip.abs(), slack=2.0 ** -20, label="D x")

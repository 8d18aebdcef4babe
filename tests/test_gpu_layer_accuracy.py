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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("step", [100.0, 62464.0, 2.0 ** 60])
def test_scan_after_a_token_that_forgets_everything(step, dtype):
    # one token of a chunk whose log-decay is -1600 to -2^64: the decays between later tokens are as exact as before it
    c = ref.scan_inputs(gen(9), 1, 130, 4, 1, 64, 64, dtype)
    c["A"] = torch.tensor([-16.0, -4.0, -1.0, -2.5])
    c["dt"][0, 20] = step
    c["dt"][0, 70] = step
    y, ht = run_scan(c)
    ry, rm, rh, rhm = ref.scan(*(c[n] for n in ("x", "dt", "A", "B", "C", "D", "bias", "h0")))
    check(y, ry, rm, slack=2.0 ** -8 if dtype == BF else 2.0 ** -17, label="y")
    check(ht, rh, rhm, slack=2.0 ** -17, label="state")


# -------------------------------------------------------------------- norm --
def e4m3_of(x, w, z=None, eps=1e-6):
    """(8-bit values, scales) of the norm of rows in 64 bits, on the GPU; the quotient y / scale is rounded to fp32 and
    from there to 8 bits, so that what ties in fp32 goes to the even value."""
    h, w = x.double(), w.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w
    if z is not None:
        y = y * (z.double() / (1 + torch.exp(-z.double())))
    y = y.unflatten(-1, (-1, 128))
    s = (y.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 448).float()
    v = (y / s.double()).float().double()
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / unit) * unit).flatten(-2), s[..., 0]


@pytest.mark.parametrize("lo,hi", [(-15.0, -10.0), (-30.0, -15.0), (-40.0, -30.0), (-85.0, -40.0), (-10.0, 10.0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_to_8_bits_of_strongly_negative_gates(lo, hi, dtype):
    # 2^25 values: every one the rounding of its 64-bit value, wherever the gates of a group lie
    g = torch.Generator(device="cuda").manual_seed(int(-lo))
    rows = 1 << 16
    w = (1 + 0.2 * torch.randn(128, generator=g, device="cuda")).to(dtype)
    wrong = 0
    for _ in range(4):
        x = torch.randn(rows, 128, generator=g, device="cuda").to(dtype)
        z = (lo + (hi - lo) * torch.rand(rows, 128, generator=g, device="cuda")).to(dtype)
        q, s, _ = gdr.gdr_rms_norm_fwd(x, w, None, z, quant=True)
        want, scale = e4m3_of(x, w, z)
        wrong += int((q.double() != want).sum())
        # the fp32 chain's scale: 30 roundings and exp's argument, rounded at |z| log2 e
        assert bool(((s / scale - 1).abs() <= (30 + 2 * max(0.0, -lo)) * 2.0 ** -24).all())
    # a value whose 64-bit sum was added in another order may still differ where its fp32 rounding ties to 2^-50
    print("wrong", wrong, flush=True)
    assert wrong <= 1


@pytest.mark.parametrize("dim,dtype", [(128, BF), (128, F32), (256, BF), (512, F32), (2048, BF)])
def test_norm_to_8_bits_without_a_gate(dim, dtype):
    # 2^25 values, as above
    g = torch.Generator(device="cuda").manual_seed(dim)
    w = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(dtype)
    wrong = 0
    for _ in range(4):
        x = torch.randn(2 ** 23 // dim, dim, generator=g, device="cuda").to(dtype)
        q, s, _ = gdr.gdr_rms_norm_fwd(x, w, quant=True)
        want, scale = e4m3_of(x, w)
        wrong += int((q.double() != want).sum())
        assert bool(((s / scale - 1).abs() <= 30 * 2.0 ** -24).all())
    print("wrong", wrong, flush=True)
    assert wrong <= 1


@pytest.mark.parametrize("dim,dtype,gated", [(64, BF, False), (128, BF, True), (128, F32, False), (256, BF, True), (200, F32, True)])
def test_norm_to_8_bits_of_a_row_does_not_depend_on_its_neighbours(dim, dtype, gated):
    g = torch.Generator(device="cuda").manual_seed(dim)
    rows = 20001
    x, z = (torch.randn(rows, dim, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(dtype)
    z = z if gated else None
    q, s, _ = gdr.gdr_rms_norm_fwd(x, w, None, z, quant=True)
    for first in (1, 2, 3, 5, 9):      # other rows share the wave
        q1, s1, _ = gdr.gdr_rms_norm_fwd(x[first:], w, None, None if z is None else z[first:], quant=True)
        assert torch.equal(q[first:].view(torch.uint8), q1.view(torch.uint8))
        assert torch.equal(s[first:], s1)
    for r in (0, 777, rows - 1):       # alone
        q1, s1, _ = gdr.gdr_rms_norm_fwd(x[r:r + 1], w, None, None if z is None else z[r:r + 1], quant=True)
        assert torch.equal(q[r:r + 1].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[r:r + 1], s1)


@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_norm_to_8_bits_of_gates_that_are_zero_or_strongly_negative(zero):
    # lanes whose gates are all zero, of either sign, beside lanes whose gates decide the range that is looked at again
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = 1 << 16
    w = torch.ones(128, device="cuda", dtype=F32)
    wrong = 0
    for _ in range(4):
        x = torch.randn(rows, 128, generator=g, device="cuda")
        z = -40 + 10 * torch.rand(rows, 128, generator=g, device="cuda")
        z[:, 32:48] = zero
        q, _, _ = gdr.gdr_rms_norm_fwd(x, w, None, z, quant=True)
        wrong += int((q.double() != e4m3_of(x, w, z)[0]).sum())
    print("wrong", wrong, flush=True)
    assert wrong <= 1

"""States and gradients that are infinite stay so until their sequence ends,
wherever the token axis is cut: what token by token gives (inf a + b = inf)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


# decays around e^-0.2, whose products vanish in fp32 over some tiles, and around e^-4, over a few waves of one
@pytest.mark.parametrize("dtype,rate", [(BF, -0.4), (BF, -8.0), (F32, -0.4), (F32, -8.0)])
def test_an_infinite_state_stays_infinite(dtype, rate):
    g = gen(int(-10 * rate))
    T, D, cu = 6000, 40, [0, 5500, 5990]
    x, r, i = (randn(g, 1, T, D, dtype=dtype) for _ in range(3))
    A, h0 = torch.full((D,), rate), randn(g, 2, D)
    want = torch.zeros(T, D)
    for start, channel, value in ((0, 3, INF), (200, 4, -INF), (3333, 5, INF), (5499, 6, INF), (5500, 7, -INF)):
        x[0, start, channel] = value
        want[start:5500 if start < 5500 else 5990, channel] = value
    h0[0, 8], h0[1, 9] = -INF, INF
    want[:5500, 8], want[5500:5990, 9] = -INF, INF
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, ht = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i, A)), cuda(h0), table, output_final_state=True)
    y, ht = y[0].float().cpu(), ht.cpu()
    at = torch.isinf(want)
    assert torch.equal(y[at], want[at]) and bool(torch.isfinite(y[~at]).all())
    last = torch.stack([want[5499], want[5989]])
    at = torch.isinf(last)
    assert torch.equal(ht[at], last[at]) and bool(torch.isfinite(ht[~at]).all())


@pytest.mark.parametrize("dtype,rate", [(BF, -0.4), (BF, -8.0), (F32, -0.4), (F32, -8.0)])
def test_an_infinite_gradient_of_the_state_stays_infinite(dtype, rate):
    g = gen(int(-20 * rate))
    T, D, cu = 6000, 40, [0, 5500, 5990]
    x, r, i, dy = (randn(g, 1, T, D, dtype=dtype) for _ in range(4))
    A, h0, dht = torch.full((D,), rate), randn(g, 2, D), randn(g, 2, D)
    want, want0 = torch.zeros(T, D), torch.zeros(2, D)
    for token, channel, value in ((5499, 3, INF), (5000, 4, -INF), (0, 5, INF), (5989, 6, INF), (5500, 7, -INF)):
        dy[0, token, channel] = value
        n = int(token >= 5500)
        want[cu[n]:token + 1, channel] = want0[n, channel] = value
    dht[0, 8] = -INF
    want[:5500, 8] = want0[0, 8] = -INF
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    dx, dr, di, dA, dh0 = gdr.gdr_linear_scan_bwd(*(cuda(t) for t in (x, r, i, A, dy)), cuda(h0), cuda(dht), table)
    dx, dh0 = dx[0].float().cpu(), dh0.cpu()       # dx = g sqrt(1 - a^2) sigmoid(i): g's sign
    at, at0 = torch.isinf(want), torch.isinf(want0)
    assert torch.equal(dx[at], want[at]) and bool(torch.isfinite(dx[~at]).all())
    assert torch.equal(dh0[at0], want0[at0]) and bool(torch.isfinite(dh0[~at0]).all())
    clean = ~(at.any(0) | at0.any(0))
    assert all(bool(torch.isfinite(t.float().cpu()[..., clean]).all()) for t in (dr, di, dA))


def test_a_decay_of_zero_makes_an_infinite_state_nan():
    T, D = 3000, 4
    x, r, i = (torch.zeros(1, T, D) for _ in range(3))
    x[0, 0] = INF
    r[0, 1500] = 100.0                       # a = e^-200, zero in fp32
    r[0, :1500] = r[0, 1501:] = -10.0        # a = e^(-200 sigmoid(-10)), 0.991
    A = torch.full((D,), -200.0)
    y, _ = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i, A)))
    assert bool((y[0, :1500] == INF).all()) and bool(torch.isnan(y[0, 1500:]).all())


def test_nan_of_either_sign_stays_to_the_end_of_its_sequence():
    g = gen(31)
    T, D, cu = 5000, 12, [0, 4000, 4980]
    x, r, i, dy = (randn(g, 1, T, D) for _ in range(4))
    A, h0 = torch.full((D,), -0.5), randn(g, 2, D)
    want, behind = torch.zeros(T, D, dtype=torch.bool), torch.zeros(T, D, dtype=torch.bool)
    for t, channel, bits in ((100, 3, 0x7fc00000), (100, 4, -0x400000), (3999, 5, -0x400000), (4000, 6, -1), (4979, 7, 0x7fffffff)):
        end = 4000 if t < 4000 else 4980
        r.view(torch.int32)[0, t, channel] = bits             # the decay is NaN
        want[t:end, channel] = True
        behind[(0 if t < 4000 else 4000):end, channel] = True
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, ht = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i, A)), cuda(h0), table, output_final_state=True)
    assert torch.equal(torch.isnan(y[0]).cpu(), want)
    assert torch.equal(torch.isnan(ht).cpu(), torch.stack([want[3999], want[4979]]))
    grads = gdr.gdr_linear_scan_bwd(*(cuda(t) for t in (x, r, i, A, dy)), cuda(h0), None, table)
    first = torch.stack([behind[3999], behind[4979]])
    assert torch.equal(torch.isnan(grads[4]).cpu(), first)     # every gradient in front goes through that decay
    for t in grads[:3]:
        assert not torch.isnan(t[0].cpu()[~behind]).any()
    assert torch.equal(torch.isnan(grads[3]).cpu(), first.any(0))

"""The packed operators on offsets that decrease or leave the tensor (device
tables are not checked on the host): nothing outside their buffers changes, and
runs that the table still names start from their own sequence's state."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
import layer_reference as ref
from gated_deltanet_chunked_rule_amd import layer
from layer_reference import check, gen, randn

pytestmark = pytest.mark.gpu
GUARD = 1 << 20


def guarded(n):
    whole = torch.full((n + 2 * GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
    return whole, whole[GUARD:GUARD + n]


def untouched(whole):
    return bool((whole[:GUARD] == 0x5a).all() and (whole[-GUARD:] == 0x5a).all())


@pytest.mark.parametrize("T,cu", [(20, [0, 10, 5, 20]), (150, [0, 70, 30, 150]), (640, [0, 200, 100, 640]), (640, [640, 0, 640, 3, 500]),
                                  (640, [-7, 900, 100, 2 ** 31 - 1, -2 ** 31, 640])])
def test_scan_on_tables_that_decrease(T, cu):
    N = len(cu) - 1
    c = ref.scan_inputs(gen(T), 1, T, 4, 1, 64, 64, torch.bfloat16, seqs=N)
    d = {n: c[n].contiguous().to("cuda") for n in ("x", "dt", "A", "B", "C", "D", "bias", "h0")}
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = layer._bytes("gdr_ssm_scan_fwd_workspace_size", layer._SsmShape(1, T, 4, 1, 64, 64, N, 0, 1, 0, 0, 0, 0))
    whole, ws = guarded(n)
    ws.zero_()
    y, ht = gdr.gdr_ssm_scan_fwd(*(d[n] for n in ("x", "dt", "A", "B", "C", "D", "bias", "h0")), table, output_final_state=True, workspace=ws)
    assert untouched(whole) and bool(torch.isfinite(y).all())
    if T <= 150:   # one segment: the run behind the first decrease, alone
        at, s = cu[1], 2
        ye, he = gdr.gdr_ssm_scan_fwd(*(d[n][:, at:].contiguous() for n in ("x", "dt")), d["A"], *(d[n][:, at:].contiguous() for n in ("B", "C")),
                                      d["D"], d["bias"], d["h0"][s:s + 1].contiguous(), output_final_state=True)
        assert torch.equal(y[:, at:], ye) and torch.equal(ht[s], he[0])


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [20, 0, 20, 3], [-7, 90, 10, 2 ** 31 - 1, -2 ** 31, 20]])
def test_convolution_on_tables_that_decrease(cu):
    N, T, D = len(cu) - 1, 20, 24
    g = gen(N)
    x, dy, w, h0, dht = (randn(g, *s).to("cuda") for s in ((1, T, D), (1, T, D), (D, 4), (N, 3, D), (N, 3, D)))
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, ht = gdr.gdr_causal_conv_fwd(x, w, None, h0, table, output_final_state=True)
    whole, ws = guarded(layer._bytes("gdr_causal_conv_bwd_workspace_size", layer._ConvShape(1, T, D, 4, N, 1, 1, 0)))
    grads = gdr.gdr_causal_conv_bwd(x, w, None, dy, h0, dht, table, workspace=ws)
    assert untouched(whole)
    assert all(bool(torch.isfinite(t).all()) for t in (y, ht, *grads[:2], grads[3]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[0] * 200, [0, 0, 300] + [0] * 150 + [500, 0, 7] + [0] * 40, [900] + [0] * 63, [0] * 129 + [130]])
def test_scan_of_a_batch_that_is_mostly_empty(lens, dtype):
    # a table with room for more sequences than there are: the empty ones keep their states, whichever workgroup copies them
    T, N, H = 900, len(lens), 6
    c = ref.scan_inputs(gen(N), 1, T, H, 2, 32, 32, dtype, seqs=N)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    d = {n: c[n].contiguous().to("cuda") for n in ("x", "dt", "A", "B", "C", "D", "bias", "h0")}
    for h0 in (d["h0"], None):
        y, ht = gdr.gdr_ssm_scan_fwd(*(d[n] for n in ("x", "dt", "A", "B", "C", "D", "bias")), h0, cu.to("cuda"), output_final_state=True)
        ry, rm, rh, rhm = ref.scan(*(c[n] for n in ("x", "dt", "A", "B", "C", "D", "bias")), None if h0 is None else c["h0"], cu)
        check(y, ry, rm, slack=2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -17, label="y")
        check(ht, rh, rhm, slack=2.0 ** -17, label="states")
        empty = torch.tensor([n for n in range(N) if lens[n] == 0])
        want = c["h0"][empty] if h0 is not None else torch.zeros_like(c["h0"][empty])
        assert torch.equal(ht.cpu()[empty], want)

"""The gated linear recurrence on the GPU against its plain 64-bit form
(block_reference.py states how the bounds come about)."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import check
from layer_reference import gen, randn
from test_gpu_layer import cuda, sliced

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SCAN = [
    # B, T, D, type, cu, carried, largest -A
    (1, 1, 1, F32, None, True, 1.0),
    (1, 1, 256, BF, None, False, 1.0),
    (2, 9, 67, BF, None, True, 1.0),             # odd rows
    (3, 64, 256, F32, None, False, 20.0),
    (2, 65, 300, BF, None, True, 0.05),
    (1, 200, 513, F32, None, True, 1.0),         # a column of one channel
    (1, 130, 8, BF, [0, 1, 1, 3, 64, 64, 129, 130], True, 1.0),     # empty and one token, sequences that start at a tile
    (1, 130, 70, F32, [5, 5, 17, 44, 100], True, 1.0),              # tokens before the first and behind the last sequence
    (1, 700, 260, BF, [0, 333, 600, 700], False, 1.0),
    (1, 4, 24, BF, [0, 0, 0], True, 1.0),        # no sequence has a token
    (1, 1500, 40, F32, None, True, 1e-4),        # nearly no decay
]


def scan_case(k, B, T, D, dtype, cu, carried, most):
    g = gen(700 + k)
    N = B if cu is None else len(cu) - 1
    row = randn(g, B, T, 2 * D, dtype=dtype)
    return dict(x=randn(g, B, T, D, dtype=dtype), row=row, r=row[..., :D], i=row[..., D:],
                A=-most * torch.rand(D, generator=g), h0=randn(g, N, D) if carried else None,
                cu=None if cu is None else torch.tensor(cu, dtype=torch.int32),
                dy=randn(g, B, T, D, dtype=dtype), dht=randn(g, N, D) if k % 2 else None)


def inputs(c):
    """On the device, as slices of wider rows (a copy of a slice would be dense)."""
    D = c["x"].shape[-1]
    row = sliced(cuda(c["row"]), 3 if D % 2 else 8, 1 if D % 2 else 4)
    return [sliced(cuda(c["x"]), 5, 2), row[..., :D], row[..., D:], cuda(c["A"])]


@pytest.mark.parametrize("k", range(len(SCAN)))
def test_linear_scan_fwd(k):
    c = scan_case(k, *SCAN[k])
    y, ht = gdr.gdr_linear_scan_fwd(*inputs(c), cuda(c["h0"]), cuda(c["cu"]), output_final_state=True)
    ry, rye, rh, rhe, _, _ = ref.linear_scan(c["x"], c["r"], c["i"], c["A"], c["h0"], c["cu"])
    check(y, ry, rye, "y")
    check(ht, rh, rhe, "final state")
    again, none = gdr.gdr_linear_scan_fwd(*inputs(c), cuda(c["h0"]), cuda(c["cu"]))
    assert none is None and torch.equal(again, y)


@pytest.mark.parametrize("k", range(len(SCAN)))
def test_linear_scan_bwd(k):
    c = scan_case(k, *SCAN[k])
    got = gdr.gdr_linear_scan_bwd(*inputs(c), cuda(c["dy"]), cuda(c["h0"]), cuda(c["dht"]), cuda(c["cu"]))
    want = ref.linear_scan_bwd(c["x"], c["r"], c["i"], c["A"], c["dy"], c["h0"], c["dht"], c["cu"])
    for name, t, (v, b) in zip(("dx", "dr", "di", "dA", "dh0"), got, want):
        if name == "dh0" and c["h0"] is None:
            assert t is None
        else:
            check(t, v, b, name)


@pytest.mark.parametrize("dtype,rows,D", [(BF, 1, 1), (BF, 3, 260), (F32, 5, 67), (BF, 200, 2560), (F32, 33, 1024)])
def test_linear_scan_step(dtype, rows, D):
    g = gen(40 + rows)
    x, row = randn(g, rows, D, dtype=dtype), randn(g, rows, 2 * D, dtype=dtype)
    A, state = -torch.rand(D, generator=g), randn(g, rows + 2, D)
    slots = torch.randperm(rows + 2, generator=g)[:rows].to(torch.int32)
    if rows > 2:
        slots[1] = -1             # padding
        slots[2] = slots[0]       # named twice
    dev = cuda(state)
    wide = cuda(row)
    y = gdr.gdr_linear_scan_step(sliced(cuda(x), 4, 1), wide[:, :D], wide[:, D:], cuda(A), dev, slots=cuda(slots))
    live = [k for k in range(rows) if not (rows > 2 and k in (1, 2))]
    at = slots[live].long()
    ry, rye, rh, rhe, _, _ = ref.linear_scan(x[live][:, None], row[live][:, None, :D], row[live][:, None, D:], A, state[at])
    check(y[live], ry[:, 0], rye[:, 0], "y")
    check(dev[at.cuda()], rh, rhe, "state")
    untouched = torch.ones(rows + 2, dtype=torch.bool)
    untouched[at] = False
    assert torch.equal(dev.cpu()[untouched], state[untouched])
    if rows > 2:
        assert not y[1:3].any()


def test_prompt_then_tokens_is_the_longer_prompt():
    g = gen(8)
    T, D, n = 70, 300, 5
    x, r, i = (randn(g, 1, T + n, D, dtype=F32) for _ in range(3))
    A = -torch.rand(D, generator=g)
    full, _ = gdr.gdr_linear_scan_fwd(cuda(x), cuda(r), cuda(i), cuda(A))
    _, state = gdr.gdr_linear_scan_fwd(*(cuda(t[:, :T].contiguous()) for t in (x, r, i)), cuda(A), output_final_state=True)
    ry, rye, _, _, _, _ = ref.linear_scan(x, r, i, A)
    check(full, ry, rye, "prompt")
    for k in range(n):
        y = gdr.gdr_linear_scan_step(*(cuda(t[:, T + k].contiguous()) for t in (x, r, i)), cuda(A), state)
        check(y, ry[:, T + k], rye[:, T + k], f"token {k}")


def test_many_short_sequences():
    g = gen(9)
    lens = [(7 * k) % 5 for k in range(1500)]      # more than the table that is staged
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    T, D = int(cu[-1]), 12
    x, r, i, dy = (randn(g, 1, T, D) for _ in range(4))
    A, h0, dht = -torch.rand(D, generator=g), randn(g, 1500, D), randn(g, 1500, D)
    y, ht = gdr.gdr_linear_scan_fwd(cuda(x), cuda(r), cuda(i), cuda(A), cuda(h0), cuda(cu), output_final_state=True)
    ry, rye, rh, rhe, _, _ = ref.linear_scan(x, r, i, A, h0, cu)
    check(y, ry, rye, "y")
    check(ht, rh, rhe, "final state")
    got = gdr.gdr_linear_scan_bwd(cuda(x), cuda(r), cuda(i), cuda(A), cuda(dy), cuda(h0), cuda(dht), cuda(cu))
    for t, (v, b) in zip(got, ref.linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)):
        check(t, v, b)


def test_values_that_are_not_finite_stay_in_their_sequence_and_channel():
    g = gen(10)
    T, D, cu = 300, 20, torch.tensor([0, 90, 128, 250], dtype=torch.int32)
    x, r, i, dy = (randn(g, 1, T, D) for _ in range(4))
    A, h0, dht = -torch.rand(D, generator=g), randn(g, 3, D), randn(g, 3, D)
    clean = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i)), cuda(A), cuda(h0), cuda(cu), output_final_state=True)
    grads = gdr.gdr_linear_scan_bwd(*(cuda(t) for t in (x, r, i)), cuda(A), cuda(dy), cuda(h0), cuda(dht), cuda(cu))
    bad = [t.clone() for t in (x, r, i)]
    bad[0][0, 100, 3] = float("nan")
    bad[1][0, 110, 4] = float("nan")
    bad[0][0, 120, 5] = float("inf")
    for t in bad:
        t[0, 250:] = float("nan")          # behind the last sequence
    bad_dy = dy.clone()
    bad_dy[0, 250:] = float("nan")
    y, ht = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in bad), cuda(A), cuda(h0), cuda(cu), output_final_state=True)
    touched = torch.zeros(T, D, dtype=torch.bool)
    touched[100:128, 3] = touched[110:128, 4] = touched[120:128, 5] = True
    same = ~touched.cuda()
    assert torch.equal(y[0][same], clean[0][0][same]) and not torch.isfinite(y[0][~same]).any()
    keep = torch.ones(3, D, dtype=torch.bool)
    keep[1, 3:6] = False
    assert torch.equal(ht[keep.cuda()], clean[1][keep.cuda()]) and not y[0, 250:].any()
    got = gdr.gdr_linear_scan_bwd(*(cuda(t) for t in bad), cuda(A), cuda(bad_dy), cuda(h0), cuda(dht), cuda(cu))
    other = torch.ones(T, D, dtype=torch.bool)
    other[90:128, 3:6] = False
    for a, b in zip(got[:3], grads[:3]):
        assert torch.equal(a[0][other.cuda()], b[0][other.cuda()])
    columns = torch.ones(D, dtype=torch.bool)
    columns[3:6] = False
    assert torch.equal(got[3][columns.cuda()], grads[3][columns.cuda()])
    assert torch.equal(got[4][keep.cuda()], grads[4][keep.cuda()])


def test_extreme_gates():
    """Decays of one and of zero, gates far on either side, and no decay rate at all."""
    D = 8
    r = torch.tensor([-200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 3.0]).expand(1, 5, D).contiguous()
    i = torch.tensor([0.0, -100.0, 100.0, 5.0, -5.0, 0.0, 1.0, 2.0]).expand(1, 5, D).contiguous()
    g = gen(11)
    x, dy = randn(g, 1, 5, D), randn(g, 1, 5, D)
    h0 = randn(g, 1, D)
    for rate in (0.0, -1e-6, -1.0, -50.0, -1e4):
        A = torch.full((D,), rate)
        y, ht = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i, A)), cuda(h0), output_final_state=True)
        grads = gdr.gdr_linear_scan_bwd(*(cuda(t) for t in (x, r, i, A)), cuda(dy), cuda(h0))
        assert all(bool(torch.isfinite(t).all()) for t in (y, ht, *grads)), rate
        ry, rye, _, _, _, _ = ref.linear_scan(x, r, i, A, h0)
        # an exponential's argument of 200 is off by 200 half steps: 2^-16 of the terms
        mag = h0.double().abs() + x.double().abs().sum(1)
        check(y, ry, rye + 2.0 ** -15 * mag, f"rate {rate}")


def test_autograd_matches_the_plain_calls_and_refuses_dropped_gradients():
    g = gen(12)
    c = scan_case(3, *SCAN[2])
    leaves = [cuda(c[n]).detach().clone().requires_grad_(True) for n in ("x", "r", "i", "A")]
    h0 = cuda(c["h0"]).requires_grad_(True)
    y, ht = gdr.linear_scan(*leaves, h0, output_final_state=True)
    dy, dht = cuda(randn(g, *y.shape, dtype=y.dtype)), cuda(randn(g, *ht.shape))
    grads = torch.autograd.grad((y * dy).sum() + (ht * dht).sum(), [*leaves, h0])
    with torch.no_grad():
        want = gdr.gdr_linear_scan_bwd(*(t.detach() for t in leaves), dy, h0.detach(), dht)
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
    with pytest.raises(gdr.GdrError, match="linear_scan"):
        gdr.gdr_linear_scan_fwd(*leaves)
    y, _ = gdr.linear_scan(*leaves)
    assert _ is None and torch.autograd.grad(y.float().sum(), leaves)[0].shape == y.shape


def test_captured_prompt_replays_with_other_offsets_and_inputs():
    g = gen(13)
    T, D = 200, 256
    x, r, i = (cuda(randn(g, 1, T, D, dtype=BF)) for _ in range(3))
    A, cu = cuda(-torch.rand(D, generator=g)), torch.tensor([0, 60, 200], dtype=torch.int32, device="cuda")
    h0 = cuda(randn(g, 2, D))
    call = lambda: gdr.gdr_linear_scan_fwd(x, r, i, A, h0, cu, output_final_state=True)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ht = call()
    for n in range(4):
        cu.copy_(torch.tensor([0, 50 + 40 * n, 190 + n]))
        x.copy_(cuda(randn(gen(50 + n), 1, T, D, dtype=BF)))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(y, want[0]) and torch.equal(ht, want[1])


def test_two_streams_and_another_current_stream():
    g = gen(14)
    x, r, i = (cuda(randn(g, 1, 900, 512, dtype=BF)) for _ in range(3))
    A = cuda(-torch.rand(512, generator=g))
    want, _ = gdr.gdr_linear_scan_fwd(x, r, i, A)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([gdr.gdr_linear_scan_fwd(x, r, i, A)[0] for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for ts in got for t in ts)


def test_no_tokens():
    g = gen(15)
    D = 40
    for B, cu in ((3, None), (1, [0, 0, 0])):
        N = B if cu is None else len(cu) - 1
        e = torch.empty(B, 0, D, device="cuda")
        A, h0, dht = cuda(-torch.rand(D, generator=g)), cuda(randn(g, N, D)), cuda(randn(g, N, D))
        y, ht = gdr.gdr_linear_scan_fwd(e, e, e, A, h0, cu, output_final_state=True)
        assert y.shape == e.shape and torch.equal(ht, h0)
        dx, dr, di, dA, dh0 = gdr.gdr_linear_scan_bwd(e, e, e, A, e, h0, dht, cu)
        assert dx.shape == dr.shape == di.shape == e.shape and not dA.any() and torch.equal(dh0, dht)
        assert not gdr.gdr_linear_scan_fwd(e, e, e, A, None, cu, output_final_state=True)[1].any()


def test_squares_below_the_normal_numbers():
    """1 - a^2 of 2e-39 and less: the factor counts as zero, and no gradient becomes infinite."""
    g = gen(16)
    x, i, dy = (randn(g, 1, 40, 12) for _ in range(3))
    r = torch.full((1, 40, 12), -21.0)
    for rate in (-1e-30, -1e-38, -1e-25):
        A = torch.full((12,), rate)
        got = gdr.gdr_linear_scan_fwd(*(cuda(t) for t in (x, r, i, A)))[0], *gdr.gdr_linear_scan_bwd(*(cuda(t) for t in (x, r, i, A)), cuda(dy))[:4]
        assert all(bool(torch.isfinite(t).all()) for t in got), rate
        assert float(got[0].abs().max()) <= 1e-15 and float(got[1].abs().max()) <= 1e-14


@pytest.mark.parametrize("dtype,T,D", [(BF, 3000, 300), (F32, 1300, 514), (BF, 9000, 32)])
def test_a_workspace_of_any_content_serves_call_after_call(dtype, T, D):
    g = gen(17)
    shape = gdr.layer._LinearScanShape(1, T, D, 1, 0 if dtype == BF else 1, 0, 0, 0)
    n = [gdr.layer._bytes(f"gdr_linear_scan_{k}_workspace_size", shape) for k in ("fwd", "bwd")]
    kept = [torch.randint(0, 256, (m,), dtype=torch.uint8, device="cuda") for m in n]
    A = cuda(-torch.rand(D, generator=g))
    for k in range(8):
        x, r, i, dy = (cuda(randn(gen(100 * k + j), 1, T, D, dtype=dtype)) for j in range(4))
        y, ht = gdr.gdr_linear_scan_fwd(x, r, i, A, output_final_state=True, workspace=kept[0])
        grads = gdr.gdr_linear_scan_bwd(x, r, i, A, dy, workspace=kept[1])
        fresh = [torch.full((m,), 255 * (k % 2), dtype=torch.uint8, device="cuda") for m in n]
        want = gdr.gdr_linear_scan_fwd(x, r, i, A, output_final_state=True, workspace=fresh[0])
        assert torch.equal(y, want[0]) and torch.equal(ht, want[1])
        for a, b in zip(grads[:4], gdr.gdr_linear_scan_bwd(x, r, i, A, dy, workspace=fresh[1])):
            assert torch.equal(a, b)
    cpu = [t.cpu() for t in (x, r, i)]
    ry, rye, rh, rhe, _, _ = ref.linear_scan(*(t[..., :8] for t in cpu), A.cpu()[:8])
    check(y[..., :8].contiguous(), ry, rye, "y")
    check(ht[:, :8].contiguous(), rh, rhe, "final state")

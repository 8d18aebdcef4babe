"""Tensors of more than 2^31 values, the residual's place taken by h, and a
captured training step of the linear recurrence."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import check
from gated_deltanet_chunked_rule_amd import layer
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def big(rows, width, seed):
    torch.manual_seed(seed)
    return torch.empty(rows, width, device="cuda", dtype=BF).normal_()


def test_linear_scan_beyond_32_bits():
    T, D, last = 66000, 32832, 300           # 2.17e9 values
    x, dy = big(T, D, 1)[None], big(T, D, 2)[None]
    A = cuda(-torch.rand(D, generator=gen(1)))
    cu = torch.tensor([0, 1000, T - last, T], dtype=torch.int32, device="cuda")
    y, ht = gdr.gdr_linear_scan_fwd(x, x, x, A, None, cu, output_final_state=True)
    cols = torch.tensor([0, 1, 127, 128, 16000, D - 2, D - 1], device="cuda")
    some = lambda t: t[0, T - last:][:, cols][None]  # noqa: E731
    v, g, a = some(x).cpu(), some(dy).cpu(), A[cols].cpu()
    ry, rye, rh, rhe, _, _ = ref.linear_scan(v, v, v, a)
    check(some(y), ry, rye, "y")
    check(ht[2:, cols], rh, rhe, "final state")
    del y
    grads = gdr.gdr_linear_scan_bwd(x, x, x, A, dy, cu_seqlens=cu)
    for t, (value, bound) in zip(grads[:3], ref.linear_scan_bwd(v, v, v, a, g)):
        check(some(t), value, bound)


def test_linear_scan_of_the_most_channels():
    T, D = 50, 2 ** 25
    x = big(T, D, 7)[None]
    A = torch.full((D,), -0.5, device="cuda")
    cols = torch.tensor([0, 1, 2 ** 24 + 77, D - 1], device="cuda")
    some = lambda t: t[..., cols]  # noqa: E731
    y, _ = gdr.gdr_linear_scan_fwd(x, x, x, A)
    v, a = some(x).cpu(), some(A).cpu()
    ry, rye, _, _, _, _ = ref.linear_scan(v, v, v, a)
    check(some(y), ry, rye, "y")
    del y
    grads = gdr.gdr_linear_scan_bwd(x, x, x, A, x)
    for t, (value, bound) in zip(grads[:4], ref.linear_scan_bwd(v, v, v, a, v)):
        check(some(t), value, bound)


def test_block_norm_beyond_32_bits():
    rows, dim = 131200, 16384                # 2.15e9 values
    x = big(rows, dim, 3)
    w = torch.ones(dim, device="cuda", dtype=BF)
    y, h = gdr.gdr_block_norm_fwd(x, w, x, w)
    at = slice(rows - 3, rows)
    ry, rye, rh, rhe = ref.block_norm(x[at], w, x[at], w)
    check(y[at], ry, rye, "y")
    check(h[at], rh, rhe, "h")
    dx, dh = gdr.gdr_block_norm_bwd(x, w, h, w, y)[:2]
    (vx, bx), (vh, bh) = ref.block_norm_bwd(x[at], w, h[at], w, y[at])[:2]
    check(dx[at], vx, bx, "dx")
    check(dh[at], vh, bh, "dh")


def test_product_beyond_32_bits():
    M, N, K = 66000, 32896, 48               # 2.17e9 outputs
    g = torch.Generator(device="cuda").manual_seed(4)
    whole = lambda n: torch.randint(-128, 128, (n, K), generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    q, w, s, ws = whole(M), whole(N), torch.rand(M, generator=g, device="cuda") + 0.1, torch.rand(N, generator=g, device="cuda") + 0.1
    y = gdr.gdr_matmul_i8(q, s, w, ws)
    for rows in (slice(0, 3), slice(M - 3, M)):
        check(y[rows], *ref.matmul_i8(q[rows], s[rows], w, ws))
    wide = torch.zeros(5000, 2 ** 19, device="cuda", dtype=torch.int8)     # 2.6e9 bytes between the first and the last row
    wide[:, :K] = q[:5000]
    assert torch.equal(gdr.gdr_matmul_i8(wide[:, :K], s[:5000], w[:500], ws[:500]), y[:5000, :500])
    qx, sx = gdr.gdr_quantize_rows(big(M, 32768, 5))
    rq, rs = ref.quantize(big(M, 32768, 5)[-2:])
    assert torch.equal(qx[-2:].cpu(), rq) and torch.equal(sx[-2:].cpu(), rs)


def test_product_of_the_most_columns():
    N, K = 2 ** 29, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    w = torch.randint(-128, 128, (N // 8, K * 8), generator=g, device="cuda", dtype=torch.int8).view(N, K)
    q, s, ws = w[5:6], torch.full((1,), 0.25, device="cuda"), torch.full((N,), 0.5, device="cuda")
    y = gdr.gdr_matmul_i8(q, s, w, ws)
    for at in (slice(0, 300), slice(2 ** 28 - 9, 2 ** 28 + 9), slice(N - 300, N)):
        check(y[:, at], *ref.matmul_i8(q, s, w[at], ws[at]))


@pytest.mark.parametrize("T,cu", [(20, [0, 10, 5, 20]), (150, [0, 70, 30, 150]), (640, [640, 0, 640, 3, 500]),
                                  (640, [-7, 900, 100, 2 ** 31 - 1, -2 ** 31, 640])])
def test_recurrence_on_tables_that_decrease(T, cu):
    g, D, N = gen(T), 200, len(cu) - 1
    x, r, i, dy = (cuda(randn(g, 1, T, D, dtype=BF)) for _ in range(4))
    A, h0, dht = cuda(-torch.rand(D, generator=g)), cuda(randn(g, N, D)), cuda(randn(g, N, D))
    table, guard = torch.tensor(cu, dtype=torch.int32, device="cuda"), 1 << 20
    spaces = []
    for name in ("gdr_linear_scan_fwd_workspace_size", "gdr_linear_scan_bwd_workspace_size"):
        n = layer._bytes(name, layer._LinearScanShape(1, T, D, N, 0, 0, 0, 0))
        spaces.append(torch.full((n + 2 * guard,), 0x5a, dtype=torch.uint8, device="cuda"))
    y, _ = gdr.gdr_linear_scan_fwd(x, r, i, A, h0, table, output_final_state=True, workspace=spaces[0][guard:-guard])
    grads = gdr.gdr_linear_scan_bwd(x, r, i, A, dy, h0, dht, table, workspace=spaces[1][guard:-guard])
    for w in spaces:
        assert bool((w[:guard] == 0x5a).all() and (w[-guard:] == 0x5a).all())
    assert all(bool(torch.isfinite(t).all()) for t in (y, *grads[:4]))
    again, _ = gdr.gdr_linear_scan_fwd(x, r, i, A, h0, table)
    assert torch.equal(again, y)
    if T <= 150:   # the tokens from the first decrease on are a run of the last sequence that holds them
        at = cu[1]
        v = [t[:, at:].cpu() for t in (x, r, i)]
        check(y[:, at:], *ref.linear_scan(*v, A.cpu(), h0[2:3].cpu())[:2], "the run behind the decrease")


def test_h_takes_the_residuals_place():
    g = gen(6)
    for rows, dim in ((37, 100), (9, 4096), (300, 128)):
        x, residual, w = cuda(randn(g, rows, dim, dtype=BF)), cuda(randn(g, rows, dim, dtype=BF)), cuda(randn(g, dim, dtype=BF))
        y, h = gdr.gdr_block_norm_fwd(x, w, residual, w)
        into, out = residual.clone(), torch.empty_like(y)
        shape = layer._BlockNormShape(rows, dim, 0, 1e-6, 0, 0, 0)
        layer._call(0, layer._entry("gdr_block_norm_fwd"), shape, x.data_ptr(), into.data_ptr(), None, w.data_ptr(), w.data_ptr(), None,
                    out.data_ptr(), into.data_ptr())
        assert torch.equal(into, h) and torch.equal(out, y)


def test_captured_training_step_of_the_recurrence():
    g = gen(7)
    T, D = 300, 200
    leaves = [cuda(randn(g, 1, T, D, dtype=BF)).requires_grad_(True) for _ in range(3)] + [cuda(-torch.rand(D, generator=g)).requires_grad_(True),
                                                                                          cuda(randn(g, 2, D)).requires_grad_(True)]
    dy, dht = cuda(randn(g, 1, T, D, dtype=BF)), cuda(randn(g, 2, D))
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")

    def step():
        y, ht = gdr.linear_scan(*leaves, output_final_state=True, cu_seqlens=cu)
        return y, ht, *torch.autograd.grad([y, ht], leaves, [dy, dht])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in range(4):
        with torch.no_grad():
            leaves[0].copy_(cuda(randn(gen(90 + n), 1, T, D, dtype=BF)))
            cu[1] = 60 + 70 * n
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        with torch.no_grad():
            x, r, i, A, h0 = leaves
            y, ht = gdr.gdr_linear_scan_fwd(x, r, i, A, h0, cu, output_final_state=True)
            want = y, ht, *gdr.gdr_linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)
        for a, b in zip(got, want):
            assert torch.equal(a, b)

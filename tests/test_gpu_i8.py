"""Quantised rows and their products on the GPU against their plain 64-bit form."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import check
from layer_reference import gen, randn
from test_gpu_layer import cuda, sliced

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,K,dtype", [(1, 1, F32), (3, 17, BF), (40, 100, F32), (70, 128, BF), (9, 250, BF), (5, 512, F32), (600, 1000, BF),
                                          (33, 2048, F32), (17, 4096, BF), (4, 4100, F32), (6, 8000, BF), (3, 16384, F32), (2, 20001, BF), (2, 32768, F32)])
def test_quantize_rows(rows, K, dtype):
    g = gen(K)
    x = randn(g, rows, K, dtype=dtype, std=3.0)
    x[0] = 0
    if rows > 2:
        x[1] *= 1e-33 if dtype == F32 else 1e-30
        x[2, K // 2] = 1e30
    q, scales = gdr.gdr_quantize_rows(sliced(cuda(x), 5, 1))
    rq, rs = ref.quantize(x)
    assert torch.equal(scales.cpu(), rs) and torch.equal(q.cpu(), rq)
    pad = -(-K // 16) * 16
    assert q.shape == (rows, K) and q.stride() == (pad, 1)
    whole = torch.as_strided(q, (rows, pad), (pad, 1))
    assert not whole[:, K:].any()


def test_quantize_rows_at_ties_and_not_finite():
    x = torch.zeros(6, 40)
    x[:, 0] = 127.0                                       # the scale is one
    x[0, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 125.5, -126.5])
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    x[3, 3] = float("-inf")
    x[4] = -127.0
    q, scales = gdr.gdr_quantize_rows(cuda(x))
    assert q[0, 1:9].tolist() == [0, 2, 2, 0, -2, 126, 126, -126]
    assert scales[[0, 4, 5]].tolist() == [1.0, 1.0, 1.0] and torch.isnan(scales[1:4]).all()
    assert not q[1:4].any() and bool((q[4] == -127).all())


PRODUCTS = [
    # M, N, K, type, bias
    (1, 1, 1, F32, True),
    (1, 64, 64, BF, False),
    (3, 17, 33, BF, True),
    (16, 100, 1000, F32, True),
    (17, 33, 520, BF, False),
    (33, 250, 2048, BF, True),
    (64, 8, 4096, F32, False),
    (65, 40, 129, BF, True),
    (100, 1000, 600, F32, True),
    (129, 300, 257, BF, True),
    (300, 64, 1024, BF, False),
    (1000, 2100, 384, BF, True),
    (1025, 4097, 100, F32, True),
    (2100, 2050, 500, F32, False),
    (4096, 4096, 200, BF, True),
    # each shape of a workgroup's tile with ends in it
    (40, 8150, 70, BF, True),
    (100, 8100, 200, F32, False),
    (250, 8150, 130, BF, False),
    (500, 8100, 257, F32, True),
    (4000, 4090, 300, BF, True),
    (3990, 4085, 129, F32, False),
    (4100, 4099, 130, F32, True),
]


def operands(M, N, K, dtype, bias):
    g = gen(M + 7 * N + K)
    # rows of a wider tensor, anything behind K (sliced on the device: a copy there would be dense)
    pad = lambda n: cuda(torch.randint(-128, 128, (n, -(-K // 16) * 16 + 16), generator=g, dtype=torch.int8))[:, :K]  # noqa: E731
    return pad(M), torch.rand(M, generator=g) + 0.1, pad(N), torch.rand(N, generator=g) + 0.1, randn(g, N) * 50 if bias else None


@pytest.mark.parametrize("k", range(len(PRODUCTS)))
def test_matmul_i8(k):
    M, N, K, dtype, bias = PRODUCTS[k]
    q, s, w, ws, b = operands(M, N, K, dtype, bias)
    y = gdr.gdr_matmul_i8(q, cuda(s), w, cuda(ws), cuda(b), dtype=dtype)
    check(y, *ref.matmul_i8(q, s, w, ws, b), label=f"{M} x {N} x {K}")


@pytest.mark.parametrize("M", [1, 40, 300, 2048])
def test_largest_sums_are_exact(M):
    K, N = 2 ** 17 - 16, 2100 if M == 2048 else 48
    q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = gdr.gdr_matmul_i8(q, one(M), w, one(N), dtype=F32)
    assert bool((y[:, 0] == float(128 * 128 * K)).all()) and bool((y[:, 1] == float(torch.tensor(-128 * 127 * K).float())).all())


def test_a_row_that_is_not_finite_is_nan_alone():
    g = gen(5)
    x = randn(g, 20, 256)
    x[3, 9] = float("nan")
    w, ws = gdr.gdr_quantize_rows(cuda(randn(g, 40, 256)))
    q, s = gdr.gdr_quantize_rows(cuda(x))
    y = gdr.gdr_matmul_i8(q, s, w, ws, dtype=F32)
    keep = torch.arange(20, device="cuda") != 3
    assert torch.isnan(y[3]).all() and torch.isfinite(y[keep]).all()


def test_leading_dimensions_no_rows_and_strided_rows():
    g = gen(6)
    x = cuda(randn(g, 2, 3, 96, dtype=BF))
    w, ws = gdr.gdr_quantize_rows(cuda(randn(g, 50, 96)))
    q, s = gdr.gdr_quantize_rows(x)
    assert q.shape == (2, 3, 96) and s.shape == (2, 3)
    y = gdr.gdr_matmul_i8(q, s, w, ws)
    flat = gdr.gdr_matmul_i8(q.flatten(0, 1), s.flatten(), w, ws)
    assert y.shape == (2, 3, 50) and torch.equal(y.flatten(0, 1), flat)
    wide = torch.randint(-128, 128, (6, 160), generator=g, dtype=torch.int8).cuda()
    wide[:, 32:128] = q.flatten(0, 1)
    assert torch.equal(gdr.gdr_matmul_i8(wide[:, 32:128], s.flatten(), w, ws), flat)
    q, s = gdr.gdr_quantize_rows(x[:0])
    assert gdr.gdr_matmul_i8(q, s, w, ws).shape == (0, 3, 50)


def test_one_row_without_a_leading_dimension():
    g = gen(8)
    x, (w, ws) = cuda(randn(g, 100)), gdr.gdr_quantize_rows(cuda(randn(g, 30, 100)))
    q, s = gdr.gdr_quantize_rows(x)
    assert q.shape == (100,) and s.shape == () and s.dtype == F32
    y = gdr.gdr_matmul_i8(q, s, w, ws, dtype=F32)
    q2, s2 = gdr.gdr_quantize_rows(x[None])
    assert y.shape == (30,) and torch.equal(y, gdr.gdr_matmul_i8(q2, s2, w, ws, dtype=F32)[0])


def test_scales_are_fp32_whatever_the_default_type():
    x = cuda(randn(gen(9), 100, dtype=BF))
    q, s = gdr.gdr_quantize_rows(x)
    torch.set_default_dtype(torch.float64)
    try:
        for v in (x, x[None]):
            q1, s1 = gdr.gdr_quantize_rows(v)
            assert s1.dtype == F32 and torch.equal(q1.flatten(), q) and torch.equal(s1.flatten()[0], s)
    finally:
        torch.set_default_dtype(torch.float32)


def test_captured_projection_replays():
    g = gen(7)
    x, W = cuda(randn(g, 40, 512, dtype=BF)), cuda(randn(g, 300, 512, dtype=BF))
    w, ws = gdr.gdr_quantize_rows(W)
    call = lambda: gdr.gdr_matmul_i8(*gdr.gdr_quantize_rows(x), w, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    for n in range(3):
        x.copy_(cuda(randn(gen(80 + n), 40, 512, dtype=BF)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, call())

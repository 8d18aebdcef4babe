"""What the linear recurrence, the norms around a block and the products in 8
bits refuse, on the host before anything is enqueued (CPU only)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
from gated_deltanet_chunked_rule_amd import layer
from test_layer_refusals import fake, last, raises

P = [fake(i) for i in range(20)]


def swapped(args, at, value):
    return args[:at] + [value] + args[at + 1:]


# --------------------------------------------------------- linear recurrence --
def lin_shape(B=1, T=8, D=16, N=1, dtype=0, xs=0, rs=0, ist=0):
    return layer._LinearScanShape(B, T, D, N, dtype, xs, rs, ist)


FWD = [P[0], P[1], P[2], P[3], None, None, P[4], None, P[5], 1 << 40, None]      # x r i A h0 cu y ht ws bytes stream
BWD = [P[0], P[1], P[2], P[3], None, None, P[4], None, P[5], P[6], P[7], P[8], None, P[9], 1 << 40, None]


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(B=0), -1, "B must be positive"), (dict(T=-1), -1, "T not negative"), (dict(D=0), -1, "D must be positive"),
    (dict(D=2 ** 25 + 1), -2, "2^25"), (dict(dtype=2), -2, "dtype"), (dict(xs=15), -1, "smaller"), (dict(rs=-16), -1, "smaller"),
    (dict(ist=1), -1, "smaller"), (dict(T=2 ** 31 - 1), -2, "too many tokens"), (dict(T=2 ** 24, D=2 ** 20), -2, "too many tokens times channels"),
])
def test_linear_scan_refuses(kw, rc, msg):
    for name, args in (("fwd", FWD), ("bwd", BWD)):
        assert layer._entry("gdr_linear_scan_" + name)(lin_shape(**kw), *args) == rc
        assert msg in last()
        assert layer._entry(f"gdr_linear_scan_{name}_workspace_size")(lin_shape(**kw)) == 0


def test_linear_scan_refuses_pointers_packing_and_workspace():
    f, b, s = (layer._entry("gdr_linear_scan_" + n) for n in ("fwd", "bwd", "step"))
    for f, args, ws in ((f, FWD, 8), (b, BWD, 13)):
        for k in (0, 1, 2):
            assert f(lin_shape(), *swapped(args, k, None)) == -1 and "non-NULL" in last()
            assert f(lin_shape(), *swapped(args, k, P[k] + 1)) == -1 and "aligned" in last()
        assert f(lin_shape(), *swapped(args, 3, None)) == -1 and "non-NULL" in last()
        assert f(lin_shape(), *swapped(args, 3, P[3] + 2)) == -1 and "aligned" in last()
        assert f(lin_shape(), *swapped(args, 4, P[10] + 2)) == -1 and "aligned" in last()
        assert f(lin_shape(B=2), *swapped(args, 5, P[10])) == -1 and "B == 1" in last()
        assert f(lin_shape(N=0), *swapped(args, 5, P[10])) == -1 and "num_seqs" in last()
        assert f(lin_shape(), *swapped(args, ws, None)) == -3
        assert f(lin_shape(), *swapped(args, ws, P[5] + 4)) == -1 and "16-byte" in last()
        assert f(lin_shape(T=1000), *swapped(args, ws + 1, 255)) == -3 and "workspace too small" in last()
        assert f(None, *args) == -1
    f = layer._entry("gdr_linear_scan_fwd")
    for k in (0, 1, 2):
        assert f(lin_shape(), *swapped(FWD, 6, P[k])) == -1 and "overlap" in last()
    assert f(lin_shape(), *swapped(swapped(FWD, 4, P[10]), 7, P[10])) == -1 and "overlap" in last()
    for out in (8, 9, 10):
        for src in (P[0], P[1], P[2], P[4]):
            assert b(lin_shape(), *swapped(BWD, out, src)) == -1 and "overlap" in last()
    assert b(lin_shape(), *swapped(swapped(BWD, 7, P[10]), 12, P[10])) == -1 and "overlap" in last()
    ok = [P[0], P[1], P[2], P[3], P[4], 4, None, P[5], None]
    assert s(lin_shape(T=2), *ok) == -1 and "T == 1" in last()
    assert s(lin_shape(B=5, T=1), *ok) == -1 and "num_slots" in last()
    assert s(lin_shape(T=1), *swapped(ok, 4, None)) == -1 and "non-NULL" in last()
    assert s(lin_shape(T=1), *swapped(ok, 4, P[4] + 2)) == -1 and "aligned" in last()
    assert s(lin_shape(T=1), *swapped(swapped(ok, 5, 0), 6, P[6])) == -1 and "num_slots" in last()


# ------------------------------------------------------- norms around a block --
def norms_shape(rows=4, dim=64, dtype=0, eps=1e-6, xs=0, rs=0, gs=0):
    return layer._BlockNormShape(rows, dim, dtype, eps, xs, rs, gs)


NF = [P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], None]          # x residual gate post pre scale y h
NB = [P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], P[8], P[9], P[10], P[11], P[12], P[13], P[14], 1 << 40, None]


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(rows=-1), -1, "rows"), (dict(dim=0), -1, "positive"), (dict(dim=16385), -2, "at most 16384"), (dict(eps=-1.0), -1, "eps"),
    (dict(eps=float("inf")), -1, "eps"), (dict(xs=63), -1, "smaller"), (dict(rs=-64), -1, "smaller"), (dict(gs=1), -1, "smaller"),
    (dict(rows=1 << 40), -2, "too many rows"), (dict(dtype=4), -2, "dtype"),
])
def test_block_norm_refuses(kw, rc, msg):
    assert layer._entry("gdr_block_norm_fwd")(norms_shape(**kw), *NF) == rc
    assert msg in last()
    assert layer._entry("gdr_block_norm_bwd")(norms_shape(**kw), *NB) == rc
    assert layer._entry("gdr_block_norm_bwd_workspace_size")(norms_shape(**kw)) == 0


def test_block_norm_refuses_pointers_and_workspace():
    f, b = layer._entry("gdr_block_norm_fwd"), layer._entry("gdr_block_norm_bwd")
    assert f(None, *NF) == -1 and b(None, *NB) == -1
    for k in (0, 1, 3, 4, 6, 7):
        assert f(norms_shape(), *swapped(NF, k, None)) == -1 and "non-NULL" in last()
    for k in range(8):
        assert f(norms_shape(), *swapped(NF, k, P[15] + 1)) == -1 and "aligned" in last()
    for out, src in ((6, 0), (6, 1), (6, 2), (6, 7), (7, 0), (7, 2)):
        assert f(norms_shape(), *swapped(NF, out, NF[src])) == -1 and "overlap" in last()
    assert f(norms_shape(rs=80), *swapped(NF, 7, NF[1])) == -1 and "dense" in last()
    for k in (0, 1, 3, 4, 6, 8, 9, 10, 11, 12, 13):
        assert b(norms_shape(), *swapped(NB, k, None)) == -1 and "non-NULL" in last()
    for k in range(14):
        assert b(norms_shape(), *swapped(NB, k, P[15] + 1)) == -1 and "aligned" in last()
    for out in (8, 9, 10):
        for src in (0, 1, 2, 6, 7):
            assert b(norms_shape(), *swapped(NB, out, NB[src])) == -1 and "overlap" in last()
    assert b(norms_shape(), *swapped(NB, 14, None)) == -3
    assert b(norms_shape(), *swapped(NB, 15, 64)) == -3 and "workspace too small" in last()
    assert b(norms_shape(), *swapped(NB, 14, P[14] + 8)) == -1 and "16-byte" in last()


# ------------------------------------------------------------ products in 8 bits --
@pytest.mark.parametrize("kw,rc,msg", [
    (dict(rows=-1), -1, "rows"), (dict(dim=0), -1, "positive"), (dict(dim=32769), -2, "at most 32768"), (dict(dtype=2), -2, "dtype"),
    (dict(xs=99), -1, "smaller"), (dict(qs=96), -1, "smaller"), (dict(qs=120), -1, "multiple of 16"), (dict(rows=1 << 40), -2, "too many rows"),
])
def test_quantize_refuses(kw, rc, msg):
    d = dict(rows=4, dim=100, dtype=0, xs=0, qs=0) | kw
    assert layer._entry("gdr_quantize_rows")(layer._QuantizeShape(*d.values()), P[0], P[1], P[2], None) == rc
    assert msg in last()


def test_quantize_refuses_pointers():
    f, sh = layer._entry("gdr_quantize_rows"), layer._QuantizeShape(4, 100, 0, 0, 0)
    assert f(None, P[0], P[1], P[2], None) == -1
    for args in ((None, P[1], P[2]), (P[0], None, P[2]), (P[0], P[1], None)):
        assert f(sh, *args, None) == -1 and "non-NULL" in last()
    for args in ((P[0] + 1, P[1], P[2]), (P[0], P[1] + 8, P[2]), (P[0], P[1], P[2] + 2)):
        assert f(sh, *args, None) == -1 and "aligned" in last()


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(M=-1), -1, "positive"), (dict(N=0), -1, "positive"), (dict(K=0), -1, "positive"), (dict(K=2 ** 17), -2, "2^17"),
    (dict(M=2 ** 30 + 1), -2, "2^30"), (dict(dtype=7), -2, "dtype"), (dict(xs=16), -1, "smaller"), (dict(ws=40), -1, "multiples of 16"),
    (dict(ws=-48), -1, "smaller"), (dict(xs=2 ** 22 + 16), -2, "2^22"), (dict(M=2 ** 30, N=2 ** 30), -2, "too many rows times columns"),
])
def test_matmul_refuses(kw, rc, msg):
    d = dict(M=4, N=8, K=33, dtype=0, xs=0, ws=0) | kw
    assert layer._entry("gdr_matmul_i8")(layer._MatmulI8Shape(*d.values()), *P[:6], None) == rc
    assert msg in last()


def test_matmul_refuses_pointers():
    f, sh = layer._entry("gdr_matmul_i8"), layer._MatmulI8Shape(4, 8, 33, 0, 0, 0)
    ok = P[:6] + [None]
    assert f(None, *ok) == -1
    for k in (0, 1, 2, 3, 5):
        assert f(sh, *swapped(ok, k, None)) == -1 and "non-NULL" in last()
    for k in (0, 2):
        assert f(sh, *swapped(ok, k, P[k] + 8)) == -1 and "16-byte" in last()
    for k in (1, 3, 4, 5):
        assert f(sh, *swapped(ok, k, P[k] + 1)) == -1 and "elements" in last()


def test_python_checks_run_before_the_library():
    t = torch.zeros
    raises("B, T, D", gdr.gdr_linear_scan_fwd, t(4, 8), t(4, 8), t(4, 8), t(8))
    raises("device tensor", gdr.gdr_linear_scan_fwd, t(1, 4, 8), t(1, 4, 8), t(1, 4, 8), t(8))
    raises("rows, D", gdr.gdr_linear_scan_step, t(1, 4, 8), t(4, 8), t(4, 8), t(8), t(4, 8))
    raises("at least two", gdr.gdr_block_norm_fwd, t(8), t(8), t(8), t(8))
    raises("unsupported dtype", gdr.gdr_block_norm_fwd, t(2, 8, dtype=torch.float16), t(8), t(2, 8), t(8))
    raises("K positive", gdr.gdr_quantize_rows, t(3, 0))
    raises("device tensor", gdr.gdr_quantize_rows, t(3, 8))
    q = t(3, 32, dtype=torch.int8)
    raises("weight", gdr.gdr_matmul_i8, q, t(3), t(32, dtype=torch.int8), t(1))
    raises("shape mismatch", gdr.gdr_matmul_i8, q, t(3), t(4, 16, dtype=torch.int8), t(4))
    raises("unsupported dtype", gdr.gdr_matmul_i8, q, t(3), t(4, 32, dtype=torch.int8), t(4), dtype=torch.float16)
    raises("device tensor", gdr.gdr_matmul_i8, q, t(3), t(4, 32, dtype=torch.int8), t(4))
    leaf = torch.zeros(1, 4, 8, requires_grad=True)
    raises("linear_scan", gdr.gdr_linear_scan_fwd, leaf, t(1, 4, 8), t(1, 4, 8), t(8))
    raises("no gradient", gdr.gdr_linear_scan_step, leaf[0], t(4, 8), t(4, 8), t(8), t(4, 8))
    raises("block_norm", gdr.gdr_block_norm_fwd, t(4, 8), torch.zeros(8, requires_grad=True), t(4, 8), t(8))
    raises("no gradient", gdr.gdr_quantize_rows, leaf)
    raises("no gradient", gdr.gdr_matmul_i8, q, t(3), t(4, 32, dtype=torch.int8), t(4), torch.zeros(4, requires_grad=True))


class OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0, for checks of strides."""

    def get_device(self):
        return 0


def on_device(t):
    return t.as_subclass(OnDevice)


def test_row_strides():
    t = on_device(torch.zeros(4, 6, 40))
    assert layer._flat_rows(t[..., 4:36], "x", (4, 6, 32), torch.float32, 0)[1] == 40
    assert layer._flat_rows(t[:1, :1, :32], "x", (1, 1, 32), torch.float32, 0)[1] == 0
    raises("one stride", layer._flat_rows, t[:, :5, :32], "x", (4, 5, 32), torch.float32, 0)
    raises("contiguous", layer._flat_rows, t[..., ::2], "x", (4, 6, 20), torch.float32, 0)
    raises("overlap", layer._flat_rows, on_device(torch.zeros(32)).expand(5, 32), "x", (5, 32), torch.float32, 0)
    q = on_device(torch.zeros(5, 48, dtype=torch.int8))
    assert layer._i8_rows(q[:, :33], "q", (5, 33), 0)[1] == 48
    raises("multiples of 16", layer._i8_rows, on_device(torch.zeros(5, 33, dtype=torch.int8)), "q", (5, 33), 0)
    short = on_device(torch.zeros(4 * 48 + 33, dtype=torch.int8).as_strided((5, 33), (48, 1)))
    raises("storage must reach", layer._i8_rows, short, "q", (5, 33), 0)


def test_sizes_that_32_bits_cannot_hold():
    m = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="meta").as_subclass(OnDevice)  # noqa: E731
    n = 2 ** 32 + 8                                     # its low 32 bits are a size that would be taken
    x, A = m(1, n, 8), m(8, dtype=torch.float32)
    raises("T must be below", gdr.gdr_linear_scan_fwd, x, x, x, A)
    raises("T must be below", gdr.gdr_linear_scan_bwd, x, x, x, A, x)
    raises("rows must be below", gdr.gdr_linear_scan_step, x[0], x[0], x[0], A, m(n, 8, dtype=torch.float32))
    x, w = m(2, n), m(n)
    raises("dim must be below", gdr.gdr_block_norm_fwd, x, w, x, w)
    raises("dim must be below", gdr.gdr_block_norm_bwd, x, w, x, w, x)
    raises("K must be below", gdr.gdr_quantize_rows, x)
    q, s, w = m(n, 16, dtype=torch.int8), m(n, dtype=torch.float32), m(8, 16, dtype=torch.int8)
    raises("M must be below", gdr.gdr_matmul_i8, q, s, w, m(8, dtype=torch.float32))
    raises("N must be below", gdr.gdr_matmul_i8, w, m(8, dtype=torch.float32), q, s)

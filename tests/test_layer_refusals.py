"""What the operators around the rule refuse, on the host before anything is
enqueued (CPU only), and that the Python prototypes agree with the header."""
import ctypes
import os
import re

import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
from gated_deltanet_chunked_rule_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_prototypes_have_the_headers_arguments():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdr.h")).read(), flags=re.S)
    for name in layer._SIGNATURES:
        args = [a.strip() for a in re.search(r"\b%s\s*\((.*?)\);" % name, text, re.S).group(1).split(",")]
        types = layer._entry(name).argtypes
        assert len(args) == len(types), name
        for a, t in zip(args, types):
            want = (ctypes.c_int64 if a.startswith("int64_t") else ctypes.c_int32 if a.startswith("int32_t")
                    else ctypes.c_float if re.match(r"float \w+$", a) else ctypes.c_size_t if a.startswith("size_t")
                    else None)
            assert (t is want) if want else "*" in a and t not in (ctypes.c_int32, ctypes.c_float, ctypes.c_size_t), (name, a)


def fake(n, off=0):   # aligned, never dereferenced: validation fails first
    return 0x10000 * (n + 1) + off


def last():
    return gdr.load_library().gdr_last_error().decode()


def conv_shape(B=1, T=8, D=16, W=4, N=1, dtype=0, act=1, stride=0):
    return layer._ConvShape(B, T, D, W, N, dtype, act, stride)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(B=0), -1, "B must be positive"), (dict(T=-1), -1, "T not negative"), (dict(D=0), -1, "D must be positive"),
    (dict(W=1), -2, "W must be"), (dict(W=5), -2, "W must be"), (dict(dtype=3), -2, "dtype"), (dict(act=2), -1, "activation"),
    (dict(stride=15), -1, "x_stride"), (dict(T=2 ** 31 - 1), -2, "too many tokens"),
    (dict(T=2 ** 30, D=2 ** 16), -2, "too many tokens times channels"),
])
def test_conv_refuses(kw, rc, msg):
    p = [fake(i) for i in range(9)]
    assert layer._entry("gdr_causal_conv_fwd")(conv_shape(**kw), p[0], p[1], None, None, None, p[2], None, None) == rc
    assert msg in last()
    assert layer._entry("gdr_causal_conv_bwd_workspace_size")(conv_shape(**kw)) == 0


def test_conv_refuses_pointers_packing_and_workspace():
    f, b, s = (layer._entry("gdr_causal_conv_" + n) for n in ("fwd", "bwd", "step"))
    p = [fake(i) for i in range(12)]
    assert f(conv_shape(), None, p[1], None, None, None, p[2], None, None) == -1 and "non-NULL" in last()
    assert f(conv_shape(), p[0] + 1, p[1], None, None, None, p[2], None, None) == -1 and "aligned" in last()
    assert f(conv_shape(dtype=1), p[0] + 2, p[1], None, None, None, p[2], None, None) == -1 and "aligned" in last()
    assert f(conv_shape(B=2), p[0], p[1], None, None, p[3], p[2], None, None) == -1 and "B == 1" in last()
    assert f(conv_shape(N=0), p[0], p[1], None, None, p[3], p[2], None, None) == -1 and "num_seqs" in last()
    assert b(conv_shape(), p[0], p[1], None, None, None, p[2], None, p[3], p[4], None, None, p[5], 4, None) == -3
    assert b(conv_shape(), p[0], p[1], None, None, None, p[2], None, p[3], p[4], None, None, p[5] + 4, 1 << 30, None) == -1
    assert s(conv_shape(T=2), p[0], p[1], None, p[2], 4, None, p[3], None) == -1 and "T == 1" in last()
    assert s(conv_shape(B=5, T=1), p[0], p[1], None, p[2], 4, None, p[3], None) == -1 and "num_slots" in last()
    assert s(conv_shape(T=1), p[0], p[1], None, p[2], 0, p[4], p[3], None) == -1 and "num_slots" in last()


def ssm_shape(B=1, T=8, H=4, G=2, P=64, N=128, seqs=1, dtype=0, softplus=1, xs=0, ds=0, bs=0, cs=0):
    return layer._SsmShape(B, T, H, G, P, N, seqs, dtype, softplus, xs, ds, bs, cs)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(H=5), -1, "multiple of G"), (dict(G=0), -1, "positive"), (dict(P=16), -2, "P must be"), (dict(N=256), -2, "N must be"),
    (dict(softplus=2), -1, "dt_softplus"), (dict(xs=255), -1, "smaller"), (dict(xs=257), -1, "16-byte"), (dict(bs=264 - 4), -1, "16-byte"),
    (dict(ds=3), -1, "smaller"), (dict(cs=1 << 23), -2, "2^22"), (dict(H=1 << 17), -2, "2^22"), (dict(dtype=2), -2, "dtype"),
])
def test_scan_refuses(kw, rc, msg):
    p = [fake(i) for i in range(12)]
    args = (p[0], p[1], p[2], p[3], p[4], None, None, None, None, p[5], None, p[6], 1 << 40, None)
    assert layer._entry("gdr_ssm_scan_fwd")(ssm_shape(**kw), *args) == rc
    assert msg in last()
    assert layer._entry("gdr_ssm_scan_fwd_workspace_size")(ssm_shape(**kw)) == 0
    step = dict(kw, T=1)
    assert layer._entry("gdr_ssm_step")(ssm_shape(**step), p[0], p[1], p[2], p[3], p[4], None, None, p[5], 4, None, p[6], None) == rc


def test_scan_refuses_pointers_and_workspace():
    f, s = layer._entry("gdr_ssm_scan_fwd"), layer._entry("gdr_ssm_step")
    p = [fake(i) for i in range(12)]
    ok = [p[0], p[1], p[2], p[3], p[4], None, None, None, None, p[5], None, p[6], 1 << 40, None]

    def swap(i, v):
        return ok[:i] + [v] + ok[i + 1:]

    assert f(ssm_shape(), *swap(0, None)) == -1 and "non-NULL" in last()
    assert f(ssm_shape(), *swap(0, p[0] + 8)) == -1 and "16-byte" in last()
    assert f(ssm_shape(), *swap(9, p[5] + 8)) == -1 and "16-byte" in last()
    assert f(ssm_shape(), *swap(1, p[1] + 1)) == -1 and "elements" in last()
    assert f(ssm_shape(T=100000), *swap(12, 64)) == -3 and "workspace too small" in last()
    assert f(ssm_shape(B=2), *swap(8, p[7])) == -1 and "B == 1" in last()
    assert s(ssm_shape(T=1), *p[:5], None, None, p[5] + 4, 4, None, p[6], None) == -1 and "16-byte" in last()
    assert s(ssm_shape(B=5, T=1), *p[:5], None, None, p[5], 4, None, p[6], None) == -1 and "num_slots" in last()


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(T=2), -1, "T == 1"), (dict(Hq=3), -1, "multiple of Hq"), (dict(V=64), -2, "K must equal V"),
    (dict(K=96, V=96), -2, "32, 64 or 128"), (dict(dtype=5), -2, "dtype"), (dict(B=9), -1, "num_slots"),
])
def test_rule_step_refuses(kw, rc, msg):
    d = dict(B=1, T=1, Hq=2, Hv=4, K=128, V=128, dtype=0) | kw
    sh = gdr._Shape(d["B"], d["T"], d["Hq"], d["Hv"], d["K"], d["V"], 0, d["dtype"])
    p = [fake(i) for i in range(9)]
    f = layer._entry("gdr_step")
    assert f(sh, p[0], 0, p[1], 0, p[2], 0, p[3], p[4], 1.0, p[5], 8, None, p[6], None) == rc
    assert msg in last()


def test_rule_step_refuses_scale_strides_and_pointers():
    f = layer._entry("gdr_step")
    sh = gdr._Shape(1, 1, 2, 4, 128, 128, 0, 0)
    p = [fake(i) for i in range(9)]
    assert f(sh, p[0], 0, p[1], 0, p[2], 0, p[3], p[4], float("inf"), p[5], 8, None, p[6], None) == -1 and "scale" in last()
    assert f(sh, p[0], 255, p[1], 0, p[2], 0, p[3], p[4], 1.0, p[5], 8, None, p[6], None) == -1 and "smaller" in last()
    assert f(sh, p[0], 260, p[1], 0, p[2], 0, p[3], p[4], 1.0, p[5], 8, None, p[6], None) == -1 and "16-byte" in last()
    assert f(sh, p[0], -8, p[1], 0, p[2], 0, p[3], p[4], 1.0, p[5], 8, None, p[6], None) == -1
    assert f(sh, p[0], 0, p[1], 0, p[2], 0, p[3] + 2, p[4], 1.0, p[5], 8, None, p[6], None) == -1 and "elements" in last()
    assert f(sh, p[0], 0, p[1], 0, p[2], 0, p[3], p[4], 1.0, None, 8, None, p[6], None) == -1 and "non-NULL" in last()


def norm_shape(rows=4, inner=1, dim=64, dtype=0, eps=1e-6, quant=0, xo=0, xi=0):
    return layer._NormShape(rows, inner, dim, dtype, eps, quant, xo, xi, 0, 0, 0, 0)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(rows=-1), -1, "rows"), (dict(inner=3), -1, "multiple of inner"), (dict(dim=0), -1, "positive"),
    (dict(dim=16385), -2, "at most 16384"), (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"),
    (dict(quant=2), -1, "quant"), (dict(xo=-64), -1, "negative"), (dict(rows=1 << 40), -2, "too many rows"), (dict(dtype=9), -2, "dtype"),
])
def test_norm_refuses(kw, rc, msg):
    p = [fake(i) for i in range(9)]
    assert layer._entry("gdr_rms_norm_fwd")(norm_shape(**kw), p[0], None, None, p[1], p[2], p[3], None, None) == rc
    assert msg in last()
    assert layer._entry("gdr_rms_norm_bwd_workspace_size")(norm_shape(**kw)) == 0


def test_norm_refuses_pointers_and_workspace():
    f, b = layer._entry("gdr_rms_norm_fwd"), layer._entry("gdr_rms_norm_bwd")
    p = [fake(i) for i in range(9)]
    assert f(norm_shape(quant=1), p[0], None, None, p[1], p[2], None, None, None) == -1 and "scales" in last()
    assert f(norm_shape(), p[0], p[4] + 1, None, p[1], p[2], None, None, None) == -1 and "aligned" in last()
    assert b(norm_shape(), p[0], p[1], p[2], p[3], None, p[4], p[5], None, p[6], 1 << 30, None) == -1 and "dgate" in last()
    assert b(norm_shape(), p[0], None, p[2], p[3], None, p[4], p[5], None, p[6], 8, None) == -3


def raises(msg, f, *a, **kw):
    with pytest.raises(gdr.GdrError, match=msg):
        f(*a, **kw)


def test_python_checks_run_before_the_library():
    t = torch.zeros
    raises("B, T, D", gdr.gdr_causal_conv_fwd, t(4, 8), t(8, 4))
    raises("device tensor", gdr.gdr_causal_conv_fwd, t(1, 4, 8), t(8, 4))
    raises("unsupported dtype", gdr.gdr_causal_conv_fwd, t(1, 4, 8, dtype=torch.float16), t(8, 4))
    raises("unknown activation", gdr.gdr_causal_conv_fwd, t(1, 4, 8), t(8, 4), activation="gelu")
    raises("rows, D", gdr.gdr_causal_conv_step, t(1, 4, 8), t(1, 3, 8), t(8, 4))
    raises("3-D", gdr.gdr_step, t(1, 1, 2, 32), t(1, 1, 2, 32), t(1, 1, 2, 32), t(1, 2), t(1, 2), t(1, 2, 32, 32))
    raises("4-D", gdr.gdr_ssm_scan_fwd, t(4, 2, 32), t(4, 2), t(2), t(4, 1, 32), t(4, 1, 32))
    raises("at least two", gdr.gdr_rms_norm_fwd, t(8), t(8))
    leaf = torch.zeros(1, 4, 2, 32, requires_grad=True)
    raises("no gradient", gdr.gdr_ssm_scan_fwd, leaf, t(1, 4, 2), t(2), t(1, 4, 1, 32), t(1, 4, 1, 32))
    raises("no gradient", gdr.gdr_causal_conv_step, torch.zeros(1, 8, requires_grad=True), t(1, 3, 8), t(8, 4))


def test_python_offsets_are_checked_on_the_host():
    dev = torch.device("cpu")
    raises("B == 1", layer._offsets, torch.tensor([0, 4], dtype=torch.int32), 2, 4, dev)
    raises("non-decreasing", layer._offsets, [0, 3, 2], 1, 4, dev)
    raises("non-decreasing", layer._offsets, [0, 5], 1, 4, dev)
    raises("at least two", layer._offsets, [0], 1, 4, dev)
    raises("int32 or int64", layer._offsets, torch.tensor([0.0, 4.0]), 1, 4, dev)
    cu, n = layer._offsets([0, 2, 2, 4], 1, 4, dev)
    assert n == 3 and cu.dtype == torch.int32


def test_outputs_in_an_inputs_place_are_refused():
    p = [fake(i) for i in range(12)]
    f, b, s = (layer._entry(n) for n in ("gdr_causal_conv_fwd", "gdr_causal_conv_bwd", "gdr_ssm_scan_fwd"))
    assert f(conv_shape(), p[0], p[1], None, None, None, p[0], None, None) == -1 and "overlap" in last()
    assert f(conv_shape(), p[0], p[1], None, p[2], None, p[3], p[2], None) == -1 and "overlap" in last()
    for dx, dh0 in ((p[0], p[7]), (p[3], p[7]), (p[5], p[2]), (p[5], p[4])):
        assert b(conv_shape(), p[0], p[1], None, p[2], None, p[3], p[4], dx, p[6], None, dh0, p[8], 1 << 30, None) == -1 and "overlap" in last()
    assert s(ssm_shape(), p[0], p[1], p[2], p[3], p[4], None, None, None, None, p[0], None, p[6], 1 << 40, None) == -1 and "overlap" in last()
    assert s(ssm_shape(), p[0], p[1], p[2], p[3], p[4], None, None, p[7], None, p[5], p[7], p[6], 1 << 40, None) == -1 and "overlap" in last()

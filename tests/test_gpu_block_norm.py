"""The norms around a block on the GPU against their plain 64-bit form
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

NORMS = [
    # rows, dim, type, gate, scale, dres
    (1, 1, F32, True, True, True),
    (3, 7, BF, True, True, True),
    (17, 100, F32, False, True, False),
    (40, 128, BF, True, False, True),
    (700, 129, BF, True, True, True),
    (9, 256, F32, False, False, True),
    (33, 500, BF, True, True, False),
    (5, 1000, F32, True, True, True),
    (130, 1024, BF, False, True, True),
    (600, 2048, BF, True, True, True),
    (7, 2500, F32, True, True, True),
    (1100, 4096, BF, True, True, True),
    (3, 4099, F32, True, False, True),
    (11, 8192, BF, True, True, True),
    (5, 8191, F32, True, True, True),
    (3, 16384, F32, True, True, True),
    (300, 16381, BF, True, True, True),
    (1300, 2049, BF, False, True, True),
    (530, 4097, BF, True, False, True),
    (600, 5120, BF, True, True, True),
    (4, 6145, F32, False, False, False),
    (270, 8193, BF, False, False, True),
    (9, 12000, F32, True, False, False),
    (520, 9000, BF, False, True, False),
]


def norm_case(k, rows, dim, dtype, gate, scale, dres):
    g = gen(900 + k)
    c = dict(x=randn(g, rows, dim, dtype=dtype), residual=randn(g, rows, dim, dtype=dtype, std=2.0),
             post=(1 + randn(g, dim, std=0.1)).to(dtype), pre=(1 + randn(g, dim, std=0.1)).to(dtype),
             gate=randn(g, rows, dim, dtype=dtype, std=2.0) if gate else None,
             scale=randn(g, dim, std=0.5).to(dtype) if scale else None,
             dy=randn(g, rows, dim, dtype=dtype), dres=randn(g, rows, dim, dtype=dtype) if dres else None)
    c["h"] = ref.block_norm(*(c[n] for n in ("x", "post", "residual", "pre", "gate", "scale")))[2].to(dtype)
    return c


def wide(t):
    """On the device, as a slice of a wider row (a copy of a slice would be dense)."""
    return t if t is None else sliced(cuda(t), 3 if t.shape[-1] % 2 else 8, 1 if t.shape[-1] % 2 else 4)


@pytest.mark.parametrize("k", range(len(NORMS)))
def test_block_norm_fwd(k):
    c = norm_case(k, *NORMS[k])
    args = [c[n] for n in ("x", "post", "residual", "pre", "gate", "scale")]
    x, post, residual, pre, gate, scale = args
    y, h = gdr.gdr_block_norm_fwd(wide(x), cuda(post), wide(residual), cuda(pre), wide(gate), cuda(scale), eps=ref.EPS)
    ry, rye, rh, rhe = ref.block_norm(*args)
    check(y, ry, rye, "y")
    check(h, rh, rhe, "h")


@pytest.mark.parametrize("k", range(len(NORMS)))
def test_block_norm_bwd(k):
    c = norm_case(k, *NORMS[k])
    args = [c[n] for n in ("x", "post", "h", "pre", "dy", "gate", "scale", "dres")]
    x, post, h, pre, dy, gate, scale, dres = args
    got = gdr.gdr_block_norm_bwd(wide(x), cuda(post), wide(h), cuda(pre), cuda(dy), wide(gate), cuda(scale), cuda(dres), eps=ref.EPS)
    for name, t, (v, b) in zip(("dx", "dh", "dpost", "dpre", "dgate", "dscale"), got, ref.block_norm_bwd(*args)):
        if v is None:
            assert t is None
        else:
            check(t, v, b, name)


def test_zero_rows_and_no_rows():
    z = torch.zeros(4, 300, device="cuda", dtype=BF)
    w = torch.ones(300, device="cuda", dtype=BF)
    y, h = gdr.gdr_block_norm_fwd(z, w, z, w, z, w)
    assert not y.any() and not h.any()
    grads = gdr.gdr_block_norm_bwd(z, w, h, w, torch.ones_like(z), z, w)
    assert all(bool(torch.isfinite(t.float()).all()) for t in grads)
    e = z[:0]
    y, h = gdr.gdr_block_norm_fwd(e, w, e, w)
    assert y.shape == h.shape == (0, 300)
    dx, dh, dpost, dpre, dgate, dscale = gdr.gdr_block_norm_bwd(e, w, e, w, e, scale=w)
    assert dx.shape == dh.shape == (0, 300) and dgate is None
    assert not dpost.any() and not dpre.any() and not dscale.any()


def test_rows_keep_their_values_beside_rows_that_are_not_finite():
    c = norm_case(50, 40, 96, BF, True, True, True)
    dev = {n: cuda(t) for n, t in c.items()}
    args = lambda d: [d[n] for n in ("x", "post", "residual", "pre", "gate", "scale")]  # noqa: E731
    back = lambda d: [d[n] for n in ("x", "post", "h", "pre", "dy", "gate", "scale", "dres")]  # noqa: E731
    y, h = gdr.gdr_block_norm_fwd(*args(dev))
    grads = gdr.gdr_block_norm_bwd(*back(dev))
    bad = {n: t.clone() if t.dim() == 2 else t for n, t in dev.items()}
    bad["x"][7, 3], bad["residual"][9, 0], bad["gate"][11, 5] = float("nan"), float("inf"), float("nan")
    bad["h"][9, 0], bad["dy"][13, 1] = float("inf"), float("nan")
    y2, h2 = gdr.gdr_block_norm_fwd(*args(bad))
    g2 = gdr.gdr_block_norm_bwd(*back(bad))
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[7, 9, 11, 13]] = False
    for a, b in ((y, y2), (h, h2), (grads[0], g2[0]), (grads[1], g2[1]), (grads[4], g2[4])):
        assert torch.equal(a[keep], b[keep])


def test_three_dimensions_are_rows():
    c = norm_case(51, 30, 64, F32, True, True, True)
    dev = {n: cuda(t) for n, t in c.items()}
    flat = gdr.gdr_block_norm_fwd(*(dev[n] for n in ("x", "post", "residual", "pre", "gate", "scale")))
    cube = lambda t: t.unflatten(0, (5, 6)) if t.dim() == 2 else t  # noqa: E731
    got = gdr.gdr_block_norm_fwd(*(cube(dev[n]) for n in ("x", "post", "residual", "pre", "gate", "scale")))
    assert all(torch.equal(a.flatten(0, 1), b) for a, b in zip(got, flat))


def test_autograd_matches_the_plain_calls_and_refuses_dropped_gradients():
    c = norm_case(52, 60, 320, BF, True, True, True)
    leaves = [cuda(c[n]).detach().clone().requires_grad_(True) for n in ("x", "post", "residual", "pre", "gate", "scale")]
    y, h = gdr.block_norm(*leaves)
    dy, dres = cuda(c["dy"]), cuda(c["dres"])
    grads = torch.autograd.grad([y, h], leaves, [dy, dres])
    x, post, residual, pre, gate, scale = (t.detach() for t in leaves)
    dx, dh, dpost, dpre, dgate, dscale = gdr.gdr_block_norm_bwd(x, post, h.detach(), pre, dy, gate, scale, dres)
    for a, b in zip(grads, (dx, dpost, dh, dpre, dgate, dscale)):
        assert torch.equal(a, b)
    with pytest.raises(gdr.GdrError, match="block_norm"):
        gdr.gdr_block_norm_fwd(*leaves)
    only_h = torch.autograd.grad(gdr.block_norm(*leaves)[1].float().sum(), [leaves[0], leaves[2]])
    assert bool((only_h[1] == 1).all()) and bool(torch.isfinite(only_h[0].float()).all())


def test_captured_training_step_replays():
    c = norm_case(53, 200, 512, BF, True, True, True)
    names = ("x", "post", "residual", "pre", "gate", "scale")
    leaves = [cuda(c[n]).detach().clone().requires_grad_(True) for n in names]
    dy, dres = cuda(c["dy"]), cuda(c["dres"])

    def step():
        y, h = gdr.block_norm(*leaves)
        return y, h, *torch.autograd.grad([y, h], leaves, [dy, dres])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in range(3):
        with torch.no_grad():
            leaves[0].copy_(cuda(randn(gen(60 + n), 200, 512, dtype=BF)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        with torch.no_grad():
            y, h = gdr.gdr_block_norm_fwd(*leaves)
            x, post, residual, pre, gate, scale = leaves
            dx, dh, dpost, dpre, dgate, dscale = gdr.gdr_block_norm_bwd(x, post, h, pre, dy, gate, scale, dres)
        for a, b in zip(got, (y, h, dx, dpost, dh, dpre, dgate, dscale)):
            assert torch.equal(a, b)

"""The operators of a recurrent block at sizes drawn over their ranges (ones, odd
numbers, powers of two and their neighbours, slices of wider rows), through the C
entry points, with guard bytes around every output and workspace."""
import math
import random

import pytest
import torch

import block_reference as ref
from block_reference import check
from gated_deltanet_chunked_rule_amd import layer
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 4096


class Draw:
    def __init__(self, seed):
        self.rng, self.gen, self.buffers = random.Random(seed), gen(seed), []
        self.type = self.rng.choice([BF, F32])
        self.code = 0 if self.type is BF else 1

    def often(self):
        return self.rng.random() < 0.6

    def size(self, most):
        kind, v = self.rng.random(), int(2 ** self.rng.uniform(0, math.log2(most)))
        if kind < 0.3:
            v = self.rng.randint(1, 20)
        elif kind < 0.6:
            v = 2 ** round(math.log2(v)) + self.rng.choice([-1, 0, 1])
        return max(1, min(most, v))

    def values(self, *shape, std=1.0, dtype=None):
        return randn(self.gen, *shape, std=std, dtype=dtype or self.type)

    def rows(self, t):
        """On the device, dense or a slice of wider rows; and the stride to hand over (0: dense)."""
        more = self.rng.choice([0, 0, 1, 3, 8])
        if not more:
            return cuda(t), 0
        at = self.rng.randint(0, more)
        wide = torch.full((*t.shape[:-1], t.shape[-1] + more), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., at:at + t.shape[-1]] = cuda(t)
        return wide[..., at:at + t.shape[-1]], t.shape[-1] + more

    def out(self, *shape, dtype=None):
        dtype = dtype or self.type
        width = torch.empty(0, dtype=dtype).element_size()
        n, at = math.prod(shape) * width, GUARD + width * self.rng.randint(0, 7)
        buf = torch.full((n + at + GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
        self.buffers.append((buf, at, n))
        return buf[at:at + n].view(dtype).view(shape)

    def workspace(self, name, shape):
        n = layer._bytes(name, shape)
        buf = torch.full((n + 2 * GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
        self.buffers.append((buf, GUARD, n))
        return buf[GUARD:GUARD + n]

    def call(self, name, shape, *args):
        layer._call(0, layer._entry(name), shape, *(t.data_ptr() if isinstance(t, torch.Tensor) else t for t in args))

    def guards(self):
        for buf, at, n in self.buffers:
            assert bool((buf[:at] == 0x5a).all() and (buf[at + n:] == 0x5a).all())


@pytest.mark.parametrize("seed", range(40))
def test_linear_scan(seed):
    d = Draw(2000 + seed)
    T = d.size(6000)
    B = 1 if d.often() or T > 800 else d.size(6)
    D = min(d.size(600), max(1, 300000 // (B * T)))
    cu, N = None, B
    if B == 1 and d.often():
        N = d.size(12)
        cu = sorted(d.rng.randint(0, T) for _ in range(N + 1))
    carried, ends, most = d.often(), d.often(), d.rng.choice([1e-3, 0.1, 1.0, 8.0])
    print(f"B {B} T {T} D {D} {d.type} {cu} {carried} {ends} {most}", flush=True)
    x, r, i, dy = (d.values(B, T, D) for _ in range(4))
    A = -most * torch.rand(D, generator=d.gen)
    h0, dht = d.values(N, D, dtype=F32) if carried else None, d.values(N, D, dtype=F32) if ends else None
    table = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    (X, xs), (R, rs), (I, ist) = d.rows(x), d.rows(r), d.rows(i)
    shape = layer._LinearScanShape(B, T, D, N, d.code, xs, rs, ist)
    dev = [X, R, I, cuda(A), cuda(h0), table]
    y, ht = d.out(B, T, D), d.out(N, D, dtype=F32)
    w = d.workspace("gdr_linear_scan_fwd_workspace_size", shape)
    d.call("gdr_linear_scan_fwd", shape, *dev, y, ht, w, w.numel())
    ry, rye, rh, rhe, _, _ = ref.linear_scan(x, r, i, A, h0, cu)
    check(y, ry, rye, "y")
    check(ht, rh, rhe, "final state")
    grads = [d.out(B, T, D), d.out(B, T, D), d.out(B, T, D), d.out(D, dtype=F32), d.out(N, D, dtype=F32) if carried else None]
    w, DY, DHT = d.workspace("gdr_linear_scan_bwd_workspace_size", shape), cuda(dy), cuda(dht)
    d.call("gdr_linear_scan_bwd", shape, *dev, DY, DHT, *grads, w, w.numel())
    for name, t, (v, b) in zip(("dx", "dr", "di", "dA", "dh0"), grads, ref.linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)):
        if t is not None:
            check(t, v, b, name)
    d.guards()


@pytest.mark.parametrize("seed", range(15))
def test_linear_scan_step(seed):
    d = Draw(3000 + seed)
    rows, D = d.size(300), d.size(3000)
    print(f"rows {rows} D {D} {d.type}", flush=True)
    x, r, i = (d.values(rows, D) for _ in range(3))
    A, state = -torch.rand(D, generator=d.gen), d.values(rows + 2, D, dtype=F32)
    slots = torch.randperm(rows + 2, generator=d.gen)[:rows].to(torch.int32)
    pool, y = d.out(rows + 2, D, dtype=F32), d.out(rows, D)
    pool.copy_(state)
    (X, xs), (R, rs), (I, ist) = d.rows(x), d.rows(r), d.rows(i)
    rates, where = cuda(A), cuda(slots)
    d.call("gdr_linear_scan_step", layer._LinearScanShape(rows, 1, D, 0, d.code, xs, rs, ist), X, R, I, rates, pool, rows + 2, where, y)
    at = slots.long()
    ry, rye, rh, rhe, _, _ = ref.linear_scan(x[:, None], r[:, None], i[:, None], A, state[at])
    check(y, ry[:, 0], rye[:, 0], "y")
    check(pool.cpu()[at], rh, rhe, "state")
    others = torch.ones(rows + 2, dtype=torch.bool)
    others[at] = False
    assert torch.equal(pool.cpu()[others], state[others])
    d.guards()


@pytest.mark.parametrize("seed", range(30))
def test_block_norm(seed):
    d = Draw(4000 + seed)
    dim = d.size(16384)
    rows = min(d.size(3000), max(1, 400000 // dim))
    gated, scaled, more = d.often(), d.often(), d.often()
    print(f"rows {rows} dim {dim} {d.type} {gated} {scaled} {more}", flush=True)
    x, residual, dy = d.values(rows, dim), d.values(rows, dim, std=2.0), d.values(rows, dim)
    post, pre = ((1 + d.values(dim, std=0.1, dtype=F32)).to(d.type) for _ in range(2))
    gate, scale, dres = d.values(rows, dim, std=2.0) if gated else None, d.values(dim, std=0.5) if scaled else None, d.values(rows, dim) if more else None
    ry, rye, rh, rhe = ref.block_norm(x, post, residual, pre, gate, scale)
    h = rh.to(d.type)
    (X, xs), (RES, rs), (H, hs), (Z, zs) = d.rows(x), d.rows(residual), d.rows(h), d.rows(gate) if gated else (None, 0)
    vectors = [cuda(post), cuda(pre), cuda(scale)]
    y, ho = d.out(rows, dim), d.out(rows, dim)
    d.call("gdr_block_norm_fwd", layer._BlockNormShape(rows, dim, d.code, ref.EPS, xs, rs, zs), X, RES, Z, *vectors, y, ho)
    check(y, ry, rye, "y")
    check(ho, rh, rhe, "h")
    shape = layer._BlockNormShape(rows, dim, d.code, ref.EPS, xs, hs, zs)
    grads = [d.out(rows, dim), d.out(rows, dim), d.out(rows, dim) if gated else None, d.out(dim), d.out(dim), d.out(dim) if scaled else None]
    w, DY, DRES = d.workspace("gdr_block_norm_bwd_workspace_size", shape), cuda(dy), cuda(dres)
    d.call("gdr_block_norm_bwd", shape, X, H, Z, *vectors, DY, DRES, *grads, w, w.numel())
    dx, dh, dpost, dpre, dgate, dscale = ref.block_norm_bwd(x, post, h, pre, dy, gate, scale, dres)
    # sums of rows: 90 roundings at most (steps, a workgroup's rows, strands), 2^-17 of the magnitudes beside the reference's 2^-18
    for name, t, (v, b) in zip(("dx", "dh", "dgate", "dpost", "dpre", "dscale"), grads, (dx, dh, dgate, dpost, dpre, dscale)):
        if t is not None:
            check(t, v, 3 * b if t.dim() == 1 else b, name)
    d.guards()


@pytest.mark.parametrize("seed", range(20))
def test_quantize_rows(seed):
    d = Draw(5000 + seed)
    K = d.size(32768)
    rows = min(d.size(2000), max(1, 400000 // K))
    print(f"rows {rows} K {K} {d.type}", flush=True)
    x, pad, more = d.values(rows, K, std=3.0), -(-K // 16) * 16, 16 * d.rng.randint(0, 2)
    X, xs = d.rows(x)
    buf = torch.full((rows * (pad + more) + 2 * GUARD,), 0x5a, dtype=torch.int8, device="cuda")
    scales = d.out(rows, dtype=F32)
    d.call("gdr_quantize_rows", layer._QuantizeShape(rows, K, d.code, xs, pad + more), X, buf.data_ptr() + GUARD, scales)
    q = buf[GUARD:-GUARD].view(rows, pad + more)
    rq, rs = ref.quantize(x)
    assert torch.equal(q[:, :K].cpu(), rq) and torch.equal(scales.cpu(), rs) and not q[:, K:pad].any()
    assert all(bool((t == 0x5a).all()) for t in (q[:, pad:], buf[:GUARD], buf[-GUARD:]))
    d.guards()


@pytest.mark.parametrize("seed", range(40))
def test_matmul_i8(seed):
    d = Draw(6000 + seed)
    M, N = d.size(2500), d.size(9000)
    K = min(d.size(5000), max(1, int(4e9) // (M * N)))
    print(f"M {M} N {N} K {K} {d.type}", flush=True)
    # anything behind K, up to the next rows
    wide = lambda n: torch.randint(-128, 128, (n, -(-K // 16) * 16 + 16 * d.rng.randint(0, 3)), generator=d.gen, dtype=torch.int8).cuda()  # noqa: E731
    q, w = wide(M), wide(N)
    s, ws = (cuda(torch.rand(n, generator=d.gen) + 0.1) for n in (M, N))
    bias = cuda(d.values(N, std=50.0, dtype=F32)) if d.often() else None
    y = d.out(M, N)
    d.call("gdr_matmul_i8", layer._MatmulI8Shape(M, N, K, d.code, q.stride(0), w.stride(0)), q, s, w, ws, bias, y)
    check(y, *ref.matmul_i8(q[:, :K], s, w[:, :K], ws, bias))
    d.guards()

"""Plain 64-bit forms of the linear recurrence, the norms around a block and the
products in 8 bits (torch, on the CPU), and the bounds that their tests use.

Each reference returns its value and, beside it, a bound of a kernel's error
before the output's own rounding.  u = 2^-24 is half a step of fp32.

Linear recurrence.  sigmoid(v) is off by (|v| + 5) u (the argument's rounding,
exp2, 1 + q, reciprocal), s = A sigmoid(r) by (|r| + 7) u, a = exp(s) by
|s| (|r| + 7) u + 2 u, and sqrt(1 - a^2) by half of s's relative error plus 20 u
(its series, or the difference from 1/4 on, where it is at most 3.5 of a's
error), b by 2^-18 in all for |r|, |i| up to 10.  The state's error then runs
through the same recurrence: E_t = a E_{t-1} + a |h_{t-1}| (error of a + 2 u) +
|b| 2^-18 + 2 u |h_t|, whether runs of tokens are joined one by one or as
products of decays (a product of n of them is off by the sum of their errors
and n u)."""
import torch

from layer_reference import HALF, dbl, runs

U = 2.0 ** -24
SLACK = 2.0 ** -18


def check(got, ref, bound, label=""):
    """|got - ref| <= half a step of got's type * |ref| + bound (and a step of the smallest values)."""
    got = got.detach().cpu()
    assert tuple(got.shape) == tuple(ref.shape), (label, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    most = HALF[got.dtype] * ref.abs() + (1 + HALF[got.dtype]) * bound + 1e-37
    worst = float((err / most).max()) if err.numel() else 0.0
    print(f"[{label}] worst error / bound {worst:.3f}", flush=True)
    assert bool((err <= most).all()), (label, worst)


# --------------------------------------------------------- linear recurrence --
def gates(x, r, i, A):
    e, j = torch.sigmoid(r), torch.sigmoid(i)
    s = A * e
    a, m = torch.exp(s), torch.sqrt(-torch.expm1(2 * s))
    err_a = s.abs() * (r.abs() + 7) * U + 2 * U
    return e, j, s, a, m, m * j * x, err_a


def linear_scan(x, r, i, A, h0=None, cu=None):
    """(y, bound, final states, bound, state before each token, its bound); tokens of no sequence are zero."""
    x, r, i, A, h0 = map(dbl, (x, r, i, A, h0))
    B, T, D = x.shape
    _, _, _, a, _, b, ea = gates(*(t.reshape(B * T, D) for t in (x, r, i)), A)
    N = B if cu is None else len(cu) - 1
    zeros = lambda n: torch.zeros(n, D, dtype=torch.float64)  # noqa: E731
    y, ye, old, olde, last, laste = (zeros(B * T), zeros(B * T), zeros(B * T), zeros(B * T), zeros(N), zeros(N))
    for n, s, e in runs(B, T, cu):
        h = zeros(1)[0] if h0 is None else h0[n].clone()
        E = zeros(1)[0]
        for t in range(s, e):
            old[t], olde[t] = h, E
            E = a[t] * E + a[t] * h.abs() * (ea[t] + 2 * U) + b[t].abs() * SLACK
            h = a[t] * h + b[t]
            E = E + 2 * U * h.abs()
            y[t], ye[t] = h, E
        last[n], laste[n] = h, E
    return y.view(B, T, D), ye.view(B, T, D), last, laste, old, olde


def linear_scan_bwd(x, r, i, A, dy, h0=None, dht=None, cu=None):
    """[(value, bound)] of dx, dr, di, dA, dh0.

    The gradient of the state has the same recurrence backwards: G_t = a_{t+1} (G_{t+1} + |g_{t+1}| (error of a + 2 u)) +
    2 u |g_t|.  a^2 / m is off by 2 (error of a) + 2^-18; dA's sums (a lane's, the waves', then the tiles' in 64 strands)
    by at most 2^-17 of their terms' magnitudes."""
    _, _, _, _, old, olde = linear_scan(x, r, i, A, h0, cu)
    x, r, i, A, dy, dht = map(dbl, (x, r, i, A, dy, dht))
    B, T, D = x.shape
    x, r, i, dy = (t.reshape(B * T, D) for t in (x, r, i, dy))
    e, j, s, a, m, b, ea = gates(x, r, i, A)
    N = B if cu is None else len(cu) - 1
    g, ge = torch.zeros(B * T, D, dtype=torch.float64), torch.zeros(B * T, D, dtype=torch.float64)
    inside = torch.zeros(B * T, 1, dtype=torch.float64)
    dh0, dh0e = torch.zeros(N, D, dtype=torch.float64), torch.zeros(N, D, dtype=torch.float64)
    for n, first, end in runs(B, T, cu):
        c = torch.zeros(D, dtype=torch.float64) if dht is None else dht[n].clone()
        ce = torch.zeros(D, dtype=torch.float64)
        inside[first:end] = 1
        for t in range(end - 1, first - 1, -1):
            g[t] = dy[t] + c
            ge[t] = ce + 2 * U * g[t].abs()
            c = a[t] * g[t]
            ce = a[t] * (ge[t] + g[t].abs() * (ea[t] + 2 * U))
        dh0[n], dh0e[n] = c, ce
    dm = torch.where(m > 0, a * a / m, 0)
    part = a * old - dm * j * x
    ds = g * part * inside
    dse = ge * part.abs() + g.abs() * (a * olde + (a * old).abs() * (ea + 4 * U) + (dm * j * x).abs() * (2 * ea + 2 * SLACK))
    dx, dr, di = g * m * j, ds * A * e * (1 - e), g * b * (1 - j)
    v = lambda t: t.view(B, T, D)  # noqa: E731
    return [(v(dx), v(ge * m * j + dx.abs() * SLACK)),
            (v(dr), v(dse * (A * e * (1 - e)).abs() + dr.abs() * SLACK)),
            (v(di), v(ge * (b * (1 - j)).abs() + di.abs() * 2 * SLACK)),
            ((ds * e).sum(0), (dse * e * inside).sum(0) + (ds * e).abs().sum(0) * 2 * SLACK),
            (dh0, dh0e)]


# ------------------------------------------------------- norms around a block --
EPS = 1e-6


def silu_of(z):
    e = torch.sigmoid(z)
    return z * e, e * (1 + z * (1 - e))


def block_norm(x, post, residual, pre, gate=None, scale=None, eps=EPS):
    """(y, bound, h, bound): p is off by 2^-18 of itself, h by that and a rounding, and y by its h's error, and by that of
    the mean over the row."""
    x, post, residual, pre, gate, scale = map(dbl, (x, post, residual, pre, gate, scale))
    p = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * post
    p = p if gate is None else p * silu_of(gate)[0]
    p = p if scale is None else p * scale
    h = residual + p
    off = SLACK * p.abs() + U * h.abs()
    mean = h.square().mean(-1, keepdim=True) + eps
    y = h * mean.rsqrt() * pre
    moved = (h.abs() * off).mean(-1, keepdim=True) / mean      # of the reciprocal root, relatively
    return y, off * mean.rsqrt() * pre.abs() + y.abs() * (moved + SLACK), h, off


def block_norm_bwd(x, post, h, pre, dy, gate=None, scale=None, dres=None, eps=EPS):
    """[(value, bound)] of dx, dh, dpost, dpre, dgate, dscale: 2^-18 of the magnitudes that each is added from."""
    x, post, h, pre, dy, gate, scale, dres = map(dbl, (x, post, h, pre, dy, gate, scale, dres))
    rx, rh = ((t.square().mean(-1, keepdim=True) + eps).rsqrt() for t in (x, h))
    n, q, u = h * rh, x * rx, dy * pre
    dh = rh * (u - n * (u * n).mean(-1, keepdim=True))
    mh = rh * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True))
    if dres is not None:
        dh, mh = dh + dres, mh + dres.abs()
    k = 1.0 if scale is None else scale
    act, slope = (torch.ones_like(x), None) if gate is None else silu_of(gate)
    dp, mp = dh * k * act, mh * (k * act).abs()
    dq, mq = dp * post, mp * post.abs()
    dx = rx * (dq - q * (dq * q).mean(-1, keepdim=True))
    mx = rx * (mq + q.abs() * (mq * q.abs()).mean(-1, keepdim=True))
    cols = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    out = [(dx, mx), (dh, mh), (cols(dp * q), cols(mp * q.abs())), (cols(dy * n), cols((dy * n).abs()))]
    # silu' is off by a few u of (1 + |gate|)
    out.append((None, None) if gate is None else (dh * k * q * post * slope, mh * (k * q * post).abs() * (slope.abs() + 1 + 0.1 * gate.abs())))
    out.append((None, None) if scale is None else (cols(dh * q * post * act), cols(mh * (q * post * act).abs())))
    return [(v, None if m is None else SLACK * m) for v, m in out]


# ------------------------------------------------------------ products in 8 bits --
def quantize(x):
    """(q, scales): scale = max |x| / 127 in fp32, the quotient rounded to fp32 and then to an integer, ties to even."""
    x = dbl(x)
    most = x.abs().amax(-1)
    sound = torch.isfinite(most)
    scale = (most.clamp(min=2.0 ** -100) / 127.0).float()
    q = torch.round((x / scale.double()[..., None]).float())
    q = torch.where(sound[..., None], q, 0.0).nan_to_num(0.0)
    return q.to(torch.int8), torch.where(sound, scale, float("nan"))


def matmul_i8(q, scales, weight, weight_scales, bias=None):
    """(y, bound): the sum is exact; its conversion, two products and an addition round."""
    q, weight, scales, weight_scales, bias = (None if t is None else t.detach().cpu().double() for t in (q, weight, scales, weight_scales, bias))
    y = (q @ weight.t()) * scales[..., None] * weight_scales
    mag = y.abs()
    if bias is not None:
        y, mag = y + bias, mag + bias.abs()
    return y, 4 * U * mag

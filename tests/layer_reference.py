"""Plain 64-bit forms of the operators around the rule (torch, on the CPU), and
the bounds that their tests use.

Each reference returns its value and, beside it, the sum of the magnitudes of
the terms that the value is added from; a kernel's error is bounded by

    half a step of the output's type * |value|  +  slack * sum of magnitudes

where slack covers the roundings inside: 2^-18 for chains of fp32 operations
(a few dozen roundings of 2^-24, exponentials and reciprocals of an ulp each),
and where matrix products take bf16 operands one more half step, 2^-8."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(got, ref, mag, slack=2.0 ** -18, label=""):
    got = got.detach().cpu()
    assert tuple(got.shape) == tuple(ref.shape), (label, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    bound = HALF[got.dtype] * ref.abs() + slack * mag + 1e-37
    worst = float((err / bound).max()) if err.numel() else 0.0
    print(f"[{label}] worst error / bound {worst:.3f}", flush=True)
    assert bool((err <= bound).all()), (label, worst)


def dbl(t):
    return None if t is None else t.detach().cpu().double()


def runs(B, T, cu):
    """(sequence, first token, end) in b * T + t numbering."""
    if cu is None:
        return [(b, b * T, b * T + T) for b in range(B)]
    c = [int(v) for v in cu]
    return [(n, c[n], c[n + 1]) for n in range(len(c) - 1)]


def conv_parts(x, weight, bias, h0, cu):
    """Per sequence: (n, start, end, extended rows, z, magnitude of z)."""
    B, T, D = x.shape
    W = weight.shape[1]
    flat, w = x.reshape(B * T, D), weight
    for n, s, e in runs(B, T, cu):
        before = torch.zeros(W - 1, D, dtype=torch.float64) if h0 is None else h0[n]
        ext = torch.cat([before, flat[s:e]])
        z = torch.zeros(e - s, D, dtype=torch.float64) if bias is None else bias.expand(e - s, D)
        m = z.abs()
        for j in range(W):
            z = z + ext[j:j + e - s] * w[:, j]
            m = m + (ext[j:j + e - s] * w[:, j]).abs()
        yield n, s, e, ext, z, m


def conv(x, weight, bias=None, h0=None, cu=None, act=True):
    """(y, magnitude, final_state); tokens of no sequence are zero."""
    x, weight, bias, h0 = map(dbl, (x, weight, bias, h0))
    B, T, D = x.shape
    W = weight.shape[1]
    y, mag = torch.zeros(B * T, D, dtype=torch.float64), torch.zeros(B * T, D, dtype=torch.float64)
    last = []
    for n, s, e, ext, z, m in conv_parts(x, weight, bias, h0, cu):
        y[s:e] = z * torch.sigmoid(z) if act else z
        mag[s:e] = m            # |silu'| < 1.1; sigmoid adds a relative error of a few ulps
        last.append(ext[ext.shape[0] - (W - 1):])
    return y.view(B, T, D), 1.2 * mag.view(B, T, D), torch.stack(last)


def conv_bwd(x, weight, bias, dy, h0=None, dht=None, cu=None, act=True):
    """[(value, magnitude)] of dx, dw, db, dh0."""
    x, weight, bias, dy, h0, dht = map(dbl, (x, weight, bias, dy, h0, dht))
    B, T, D = x.shape
    W = weight.shape[1]
    z64 = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    N = B if cu is None else len(cu) - 1
    dx, dxm, dw, dwm, db, dbm = z64(B * T, D), z64(B * T, D), z64(D, W), z64(D, W), z64(D), z64(D)
    dh, dhm = z64(N, W - 1, D), z64(N, W - 1, D)
    g = dy.reshape(B * T, D)
    for n, s, e, ext, z, m in conv_parts(x, weight, bias, h0, cu):
        sig = torch.sigmoid(z)
        dz = g[s:e] * (sig * (1 + z * (1 - sig))) if act else g[s:e]
        # an error of z moves dz by |silu''| <= 0.5 of it
        dzm = g[s:e].abs() * (1.2 + 0.5 * m) if act else g[s:e].abs()
        de, dem = z64(*ext.shape), z64(*ext.shape)
        for j in range(W):
            de[j:j + e - s] += dz * weight[:, j]
            dem[j:j + e - s] += dzm * weight[:, j].abs()
            dw[:, j] += (dz * ext[j:j + e - s]).sum(0)
            dwm[:, j] += (dzm * ext[j:j + e - s].abs()).sum(0)
        db += dz.sum(0)
        dbm += dzm.sum(0)
        if dht is not None:
            de[ext.shape[0] - (W - 1):] += dht[n]
            dem[ext.shape[0] - (W - 1):] += dht[n].abs()
        dx[s:e], dxm[s:e], dh[n], dhm[n] = de[W - 1:], dem[W - 1:], de[:W - 1], dem[:W - 1]
    return [(dx.view(B, T, D), dxm.view(B, T, D)), (dw, dwm), (db, dbm), (dh, dhm)]


def softplus(u):
    return torch.where(u > 30, u, torch.log1p(torch.exp(u.clamp(max=30))))


def scan(x, dt, A, B, C, D=None, bias=None, h0=None, cu=None, use_softplus=True):
    """Token by token: (y, magnitude, final states, their magnitude)."""
    x, dt, A, B, C, D, bias, h0 = map(dbl, (x, dt, A, B, C, D, bias, h0))
    b, T, H, P = x.shape
    G, N = B.shape[2:]
    xs, Bs, Cs = x.reshape(b * T, H, P), B.reshape(b * T, G, N), C.reshape(b * T, G, N)
    d = dt.reshape(b * T, H) + (0 if bias is None else bias)
    d = softplus(d) if use_softplus else d
    y, mag = torch.zeros_like(xs), torch.zeros_like(xs)
    S = b if cu is None else len(cu) - 1
    last, lastm = torch.zeros(S, H, N, P, dtype=torch.float64), torch.zeros(S, H, N, P, dtype=torch.float64)
    r = H // G
    for n, s, e in runs(b, T, cu):
        h = torch.zeros(H, N, P, dtype=torch.float64) if h0 is None else h0[n].clone()
        hm = h.abs()
        for t in range(s, e):
            a = torch.exp(d[t] * A)[:, None, None]
            Bt, Ct = Bs[t].repeat_interleave(r, 0), Cs[t].repeat_interleave(r, 0)
            u = Bt[:, :, None] * (d[t][:, None] * xs[t])[:, None, :]
            h, hm = a * h + u, a * hm + u.abs()
            y[t] = (Ct[:, :, None] * h).sum(1)
            mag[t] = (Ct[:, :, None].abs() * hm).sum(1)
            if D is not None:
                y[t] += D[:, None] * xs[t]
                mag[t] += (D[:, None] * xs[t]).abs()
        last[n], lastm[n] = h, hm
    return y.view(b, T, H, P), mag.view(b, T, H, P), last, lastm


def rule_step(q, k, v, g, beta, state, scale):
    """(o, magnitude, new state, its magnitude); row r on state[r]."""
    q, k, v, g, beta, state = map(dbl, (q, k, v, g, beta, state))
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    s = torch.exp(g)[..., None, None] * state
    p = (k[..., None] * s).sum(-2)
    pm = (k[..., None] * s).abs().sum(-2)
    delta, dm = beta[..., None] * (v - p), beta[..., None] * (v.abs() + pm)
    new, nm = s + k[..., None] * delta[..., None, :], s.abs() + k.abs()[..., None] * dm[..., None, :]
    return scale * (q[..., None] * new).sum(-2), scale * (q.abs()[..., None] * nm).sum(-2), new, nm


def norm(x, weight, residual=None, gate=None, eps=1e-6):
    """(y, magnitude, h); in 64 bits, so h is unrounded."""
    x, weight, residual, gate = map(dbl, (x, weight, residual, gate))
    h = x if residual is None else x + residual
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight
    if gate is not None:
        y = y * gate * torch.sigmoid(gate)
    return y, y.abs(), h


def norm_bwd(h, weight, dy, gate=None, dres=None, eps=1e-6):
    """[(value, magnitude)] of dh, dw and dgate (None without a gate)."""
    h, weight, dy, gate, dres = map(dbl, (h, weight, dy, gate, dres))
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = h * r
    s = None if gate is None else torch.sigmoid(gate)
    a = dy if gate is None else dy * gate * s
    u = a * weight
    dh, dhm = r * (u - n * (u * n).mean(-1, keepdim=True)), r * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True))
    if dres is not None:
        dh, dhm = dh + dres, dhm + dres.abs()
    D = h.shape[-1]
    dw, dwm = (a * n).reshape(-1, D).sum(0), (a * n).abs().reshape(-1, D).sum(0)
    if gate is None:
        return [(dh, dhm), (dw, dwm), None]
    e = dy * n * weight
    return [(dh, dhm), (dw, dwm), (e * (s * (1 + gate * (1 - s))), e.abs() * 1.2)]


def e4m3_parts(y):
    """Per-128 groups of y [..., dim]: the scale max(|y|, 2^-100) / 448 and the bound on |q scale - y|: half a step
    of e4m3 (2^-4 of the value, 2^-10 scales below its normal range) and the fp32 chain's slack."""
    dim = y.shape[-1]
    scales, bound = [], []
    for a in range(0, dim, 128):
        m = y[..., a:a + 128]
        scales.append(m.abs().amax(-1).clamp(min=2.0 ** -100) / 448)
        bound.append((2.0 ** -4 + 2.0 ** -18) * m.abs() + 2.0 ** -10 * 1.001 * scales[-1][..., None])
    return torch.stack(scales, -1), torch.cat(bound, -1)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def scan_inputs(g, b, T, H, G, P, N, dtype, seqs=None):
    """CPU inputs with the usual step sizes and decays; x, B, C are slices of one wider row."""
    row = torch.nn.functional.silu(torch.randn(b, T, H * P + 2 * G * N, generator=g)).to(dtype)
    x = row[..., :H * P].unflatten(-1, (H, P))
    B = row[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    C = row[..., H * P + G * N:].unflatten(-1, (G, N))
    dt = randn(g, b, T, H, dtype=dtype, std=0.5)
    first = torch.exp(torch.rand(H, generator=g) * math.log(100) + math.log(1e-3))
    return dict(x=x, dt=dt, A=-(1 + 15 * torch.rand(H, generator=g)), B=B, C=C, D=1 + randn(g, H, std=0.1),
                bias=first + torch.log(-torch.expm1(-first)), h0=randn(g, seqs or b, H, N, P, std=0.1), row=row)

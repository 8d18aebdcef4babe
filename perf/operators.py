"""Cases, inputs and plain forms of the operators around the gated delta rule in a linear-attention layer:

* ``conv``       short causal convolution with SiLU, of prompts (packed sequences, with carried states),
* ``conv_bwd``   its gradient,
* ``conv_step``  its form for one new token of each sequence, on a pool of states,
* ``scan``       selective state space scan of prompts (scalar decay per head, grouped B and C),
* ``scan_step``  its form for one new token of each sequence,
* ``rule_step``  the gated delta rule for one new token of each sequence,
* ``norm``       root-mean-square norm with the residual's addition, a gate, and an output in 8 bits with scales,
* ``norm_bwd``   its gradient.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, with the framework's
kernels.  Tokens are rows; the scan's x, B and C are slices of the convolution's output row, and the norm's gate is a
slice of the input projection's row, as a layer leaves them.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
TINY = 2.0 ** -100     # an all-zero group gets the scale TINY / 448
W_TAPS = 4             # taps of the convolution


def listed():
    return [
        # the q, k, v channels of the edge prefill layer (Hq = 16, Hv = 32, K = V = 128: 2 * 2048 + 4096), a batch of
        # prompts of ragged lengths that go on from earlier states
        {"name": "conv prompts", "op": "conv", "type": "bf16", "tokens": 8192, "seqs": 13, "channels": 8192, "carried": True},
        # the training layer of the repository's backward workload: B = 2, T = 16384, Hq = 16, Hv = 32
        {"name": "conv training", "op": "conv_bwd", "type": "bf16", "tokens": 32768, "seqs": 2, "channels": 8192},
        # a serving batch: one new token of each of 128 sequences
        {"name": "conv token", "op": "conv_step", "type": "bf16", "rows": 128, "channels": 8192},
        # one long prompt through a state space layer of 64 heads that share one group of B and C
        {"name": "scan prompt", "op": "scan", "type": "bf16", "tokens": 8192, "seqs": 1, "heads": 64, "groups": 1, "P": 64, "N": 128, "carried": False},
        # a batch of prompts of ragged lengths, B and C in 8 groups, with carried states
        {"name": "scan prompts", "op": "scan", "type": "bf16", "tokens": 20000, "seqs": 16, "heads": 64, "groups": 8, "P": 64, "N": 128, "carried": True},
        # a small layer in 32 bits, one prompt of an odd length
        {"name": "scan small", "op": "scan", "type": "f32", "tokens": 301, "seqs": 1, "heads": 8, "groups": 1, "P": 32, "N": 64, "carried": False},
        # one new token of each of 64 sequences through the state space layer
        {"name": "scan token", "op": "scan_step", "type": "bf16", "rows": 64, "heads": 64, "groups": 8, "P": 64, "N": 128},
        # the smallest call of serving: one new token of one sequence through the edge prefill layer's rule
        {"name": "rule one token", "op": "rule_step", "type": "bf16", "rows": 1, "Hq": 16, "Hv": 32, "K": 128},
        # one new token of each of 100 sequences through the same layer
        {"name": "rule tokens", "op": "rule_step", "type": "bf16", "rows": 100, "Hq": 16, "Hv": 32, "K": 128},
        # before a layer's 8-bit input projection in serving: 64 rows of the residual stream
        {"name": "norm rows to 8 bits", "op": "norm", "type": "bf16", "rows": 64, "heads": 1, "dim": 4096, "residual": True, "gate": False, "bits": 8},
        # after the rule of the edge prefill layer: a norm of each head's 128 values with the layer's gate, for an
        # 8-bit output projection
        {"name": "norm heads to 8 bits", "op": "norm", "type": "bf16", "rows": 8192, "heads": 32, "dim": 128, "residual": False, "gate": True, "bits": 8},
        # the residual stream's norm in training
        {"name": "norm training", "op": "norm_bwd", "type": "bf16", "rows": 16384, "heads": 1, "dim": 4096, "gate": False},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "conv_step", "scan", "scan", "scan_step", "rule_step", "rule_step", "norm", "norm", "norm_bwd"])
    kind = "f32" if rng.random() < 0.25 else "bf16"
    if op in ("conv", "conv_bwd"):
        channels = _spread(rng, 96, 8192)
        channels = channels if rng.random() < 0.3 else -(-channels // 64) * 64
        tokens = _spread(rng, 1, 8192)
        case = {"op": op, "type": kind, "tokens": tokens, "seqs": min(tokens, _spread(rng, 1, 24)), "channels": channels}
        return case | ({"carried": rng.random() < 0.5} if op == "conv" else {})
    if op == "conv_step":
        channels = _spread(rng, 96, 8192)
        return {"op": op, "type": kind, "rows": _spread(rng, 1, 256), "channels": channels if rng.random() < 0.3 else -(-channels // 64) * 64}
    if op in ("scan", "scan_step"):
        groups = rng.choice([1, 1, 2, 4, 8])
        heads = groups * rng.randint(1, 64 // groups)
        shape = {"heads": heads, "groups": groups, "P": rng.choice([32, 64, 64, 128]), "N": rng.choice([32, 64, 128, 128])}
        if op == "scan_step":
            return {"op": op, "type": kind, "rows": _spread(rng, 1, 64)} | shape
        tokens = _spread(rng, 1, 8192)
        if kind == "f32":
            tokens = -(-tokens // 4)
        return {"op": op, "type": kind, "tokens": tokens, "seqs": min(tokens, _spread(rng, 1, 12)), "carried": rng.random() < 0.5} | shape
    if op == "rule_step":
        Hq = rng.choice([1, 2, 4, 8, 16])
        return {"op": op, "type": kind, "rows": _spread(rng, 1, 128), "Hq": Hq, "Hv": Hq * rng.choice([1, 2, 4]), "K": rng.choice([32, 64, 128, 128])}
    heads = rng.choice([1, 1, 8, 32])
    dim = rng.choice([64, 128, 256]) if heads > 1 else _spread(rng, 100, 8192)
    dim = dim if heads > 1 or rng.random() < 0.3 else -(-dim // 128) * 128
    case = {"op": op, "type": kind, "rows": _spread(rng, 1, 8192), "heads": heads, "dim": dim, "gate": rng.random() < 0.4}
    return case | ({"residual": rng.random() < 0.5, "bits": rng.choice([8, 16])} if op == "norm" else {})


# ---------------------------------------------------------------- inputs --
def lengths(seqs, tokens):
    """Ragged lengths (up to 8 : 1) of `seqs` sequences that sum to `tokens`."""
    share = [8.0 ** ((i * 0.618) % 1.0) for i in range(seqs)]
    got = [max(1, int(tokens * s / sum(share))) for s in share]
    got[-1] += tokens - sum(got)
    over = max(0, 1 - got[-1])
    got[-1] += over
    got[got.index(max(got))] -= over
    return got


def prepare(case, seed):
    op, kind = case["op"], TYPES[case["type"]]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *shape, std=1.0: torch.randn(*shape, generator=gen, device="cuda") * std  # noqa: E731
    uniform = lambda *shape, lo=0.0, hi=1.0: torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo  # noqa: E731
    s = {"op": op}
    if op in ("conv", "conv_bwd", "conv_step"):
        D = case["channels"]
        s["weight"] = uniform(D, W_TAPS, lo=-0.5, hi=0.5).to(kind)      # the usual initial range, 1 / sqrt(taps)
        s["bias"] = uniform(D, lo=-0.5, hi=0.5).to(kind)
        if op == "conv_step":
            rows = case["rows"]
            s["x"] = normal(rows, D).to(kind)
            s["state"] = normal(rows + 3, W_TAPS - 1, D).to(kind)        # the pool has free slots too
            s["slots"] = torch.randperm(rows + 3, generator=gen, device="cuda")[:rows].to(torch.int32)
            return s
        T = case["tokens"]
        s["cu"] = _offsets(case)
        s["x"] = normal(1, T, D).to(kind)
        if op == "conv":
            s["initial"] = normal(case["seqs"], W_TAPS - 1, D).to(kind) if case["carried"] else None
        else:
            s["dy"] = normal(1, T, D).to(kind)
        return s
    if op in ("scan", "scan_step"):
        H, G, P, N = case["heads"], case["groups"], case["P"], case["N"]
        T = case["rows"] if op == "scan_step" else case["tokens"]
        # x, B and C are slices of the convolution's output row, dt one of the projection's
        row = (torch.nn.functional.silu(normal(T, H * P + 2 * G * N))).to(kind)
        s["x"] = row[:, :H * P].view(T, H, P)
        s["B"] = row[:, H * P:H * P + G * N].view(T, G, N)
        s["C"] = row[:, H * P + G * N:].view(T, G, N)
        s["dt"] = normal(T, H, std=0.5).to(kind)
        s["A"] = -uniform(H, lo=1.0, hi=16.0)
        first = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))   # the usual initial step sizes
        s["dt_bias"] = first + torch.log(-torch.expm1(-first))
        s["D"] = 1.0 + normal(H, std=0.1)
        if op == "scan_step":
            s["state"] = normal(T + 3, H, N, P, std=0.1)
            s["slots"] = torch.randperm(T + 3, generator=gen, device="cuda")[:T].to(torch.int32)
            return s
        s["x"], s["B"], s["C"], s["dt"] = (s[n][None] for n in ("x", "B", "C", "dt"))
        s["cu"], s["longest"] = _offsets(case), max(lengths(case["seqs"], case["tokens"]))
        s["initial"] = normal(case["seqs"], H, N, P, std=0.1) if case["carried"] else None
        return s
    if op == "rule_step":
        rows, Hq, Hv, K = case["rows"], case["Hq"], case["Hv"], case["K"]
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
        s["q"], s["k"] = unit(normal(rows, Hq, K)).to(kind), unit(normal(rows, Hq, K)).to(kind)
        s["v"] = normal(rows, Hv, K).to(kind)
        s["g"] = torch.log(uniform(rows, Hv, lo=0.85, hi=1.0))
        s["beta"] = torch.sigmoid(normal(rows, Hv))
        s["state"] = normal(rows + 3, Hv, K, K, std=0.1)
        s["slots"] = torch.randperm(rows + 3, generator=gen, device="cuda")[:rows].to(torch.int32)
        return s
    rows, heads, dim = case["rows"], case["heads"], case["dim"]
    shape = (rows, heads, dim) if heads > 1 else (rows, dim)
    s["x"] = normal(*shape).to(kind)
    s["weight"] = (1.0 + normal(dim, std=0.1)).to(kind)
    s["gate"] = normal(rows, heads * dim + 64).to(kind)[:, :heads * dim].view(shape) if case["gate"] else None
    if op == "norm_bwd":
        s["dy"] = normal(*shape).to(kind)
        s["dres"] = normal(*shape).to(kind)     # the gradient of the residual stream behind the layer
        return s
    s["residual"] = normal(*shape, std=2.0).to(kind) if case["residual"] else None
    s["bits"] = case["bits"]
    return s


def _offsets(case):
    at = [0]
    for n in lengths(case["seqs"], case["tokens"]):
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ plain forms --
def _places(cu, T):
    """Sequence, first token and end of the sequence of every token."""
    t = torch.arange(T, device=cu.device)
    n = torch.searchsorted(cu.long(), t, right=True) - 1
    return t, n, cu.long()[n], cu.long()[n + 1]


def _taps(x, initial, cu):
    """For each tap, the input rows [T, D] that it meets (earlier states, or zeros, before a sequence's first token)."""
    T, D = x.shape[1:]
    t, n, start, _ = _places(cu, T)
    N = cu.numel() - 1
    before = x.new_zeros(N * (W_TAPS - 1), D) if initial is None else initial.reshape(-1, D)
    rows = torch.cat([x[0], before]).float()
    return [rows[torch.where(t - (W_TAPS - 1) + j >= start, t - (W_TAPS - 1) + j, T + n * (W_TAPS - 1) + t - start + j)] for j in range(W_TAPS)]


def plain_conv(x, weight, bias, initial, cu):
    w = weight.float()
    z = bias.float() + sum(r * w[:, j] for j, r in enumerate(_taps(x, initial, cu)))
    # the last three inputs of every sequence, or of its earlier state where it is shorter
    T, D = x.shape[1:]
    N = cu.numel() - 1
    before = x.new_zeros(N, W_TAPS - 1, D) if initial is None else initial
    at = cu[1:].long()[:, None] - (W_TAPS - 1) + torch.arange(W_TAPS - 1, device=x.device)
    back = (at - cu[:-1].long()[:, None] + W_TAPS - 1).clamp(0, W_TAPS - 2)
    old = before[torch.arange(N, device=x.device)[:, None], back]
    last = torch.where((at >= cu[:-1].long()[:, None])[..., None], x[0][at.clamp(min=0)], old)
    return (z * torch.sigmoid(z)).to(x.dtype)[None], last


def plain_conv_bwd(x, weight, bias, dy, cu):
    T = x.shape[1]
    w, taps = weight.float(), _taps(x, None, cu)
    z = bias.float() + sum(r * w[:, j] for j, r in enumerate(taps))
    e = torch.sigmoid(z)
    dz = dy[0].float() * (e * (1 + z * (1 - e)))
    t, _, _, end = _places(cu, T)
    rows = torch.cat([dz, dz.new_zeros(1, dz.shape[1])])
    dx = sum(rows[torch.where(t + W_TAPS - 1 - j < end, t + W_TAPS - 1 - j, T)] * w[:, j] for j in range(W_TAPS))
    dw = torch.stack([(dz * r).sum(0) for r in taps], 1)
    return dx.to(x.dtype)[None], dw.to(x.dtype), dz.sum(0).to(x.dtype)


def plain_conv_step(x, state, weight, bias, slots):
    window = torch.cat([state[slots], x[:, None]], 1)
    z = bias.float() + (window.float() * weight.float().t()).sum(1)
    state[slots] = window[:, 1:]
    return (z * torch.sigmoid(z)).to(x.dtype), state


def _step_size(dt, dt_bias):
    u = dt.float() + dt_bias
    return torch.where(u > 20, u, torch.log1p(torch.exp(u.clamp(max=20))))


def plain_scan(x, dt, A, B, C, D, dt_bias, initial, cu, longest):
    """The scan in chunks of 64 tokens: masked products within a chunk, and the chunks' states joined by one product with their decays."""
    Q = 64
    T, H, P = x.shape[1:]
    G, N = B.shape[2:]
    S = cu.numel() - 1
    t, n, start, _ = _places(cu, T)
    nc = -(-longest // Q)
    longest = nc * Q
    spot = n * longest + t - start                       # its place on the padded grid
    pad = lambda v: v.new_zeros(S * longest, *v.shape[1:]).index_copy(0, spot, v)  # noqa: E731
    step = _step_size(dt[0], dt_bias)
    xs = pad(x[0].float() * step[..., None]).view(S, nc, Q, H, P).permute(0, 3, 1, 2, 4)        # S H nc Q P
    Bs = pad(B[0].float()).view(S, nc, Q, G, N).permute(0, 3, 1, 2, 4)                          # S G nc Q N
    Cs = pad(C[0].float()).view(S, nc, Q, G, N).permute(0, 3, 1, 2, 4)
    a = pad((step * A).double()).view(S, nc, Q, H).permute(0, 3, 1, 2).cumsum(-1)               # S H nc Q
    total = a[..., -1].cumsum(-1)                                                               # S H nc
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp(torch.where(low, a[..., :, None] - a[..., None, :], -math.inf)).float()
    scores = (Cs @ Bs.transpose(-1, -2)).repeat_interleave(H // G, 1) * decay
    y = scores @ xs
    left = torch.exp(a[..., -1:] - a).float()[..., None]
    states = (Bs.repeat_interleave(H // G, 1) * left).transpose(-1, -2) @ xs                    # S H nc N P
    # the state behind each chunk: sums over the chunks up to it, weighted with the decays between them
    low = torch.ones(nc, nc, dtype=torch.bool, device=x.device).tril()
    between = torch.exp(torch.where(low, total[..., :, None] - total[..., None, :], -math.inf)).float()
    behind = (between @ states.reshape(S, H, nc, N * P)).view(S, H, nc, N, P)
    first = x.new_zeros(S, H, N, P, dtype=torch.float32) if initial is None else initial
    behind = behind + torch.exp(total).float()[..., None, None] * first[:, :, None]
    entry = torch.cat([first[:, :, None], behind[:, :, :-1]], 2)
    y = y + torch.exp(a).float()[..., None] * (Cs.repeat_interleave(H // G, 1) @ entry)
    y = y.permute(0, 2, 3, 1, 4).reshape(S * longest, H, P)[spot] + D[:, None] * x[0].float()
    return y.to(x.dtype)[None], behind[:, :, -1]


def plain_scan_step(x, dt, A, B, C, state, D, dt_bias, slots):
    H, G = x.shape[1], B.shape[1]
    step = _step_size(dt, dt_bias)
    Bh, Ch = (v.float().repeat_interleave(H // G, 1) for v in (B, C))
    new = torch.exp(step * A)[..., None, None] * state[slots] + Bh[..., None] * (step[..., None] * x.float())[..., None, :]
    state[slots] = new
    return ((Ch[..., None] * new).sum(-2) + D[:, None] * x.float()).to(x.dtype), state


def plain_rule_step(q, k, v, g, beta, state, slots):
    r = v.shape[1] // q.shape[1]
    qh, kh = (t.float().repeat_interleave(r, 1) for t in (q, k))
    new = torch.exp(g)[..., None, None] * state[slots]
    delta = beta[..., None] * (v.float() - (kh[..., None] * new).sum(-2))
    new = new + kh[..., None] * delta[..., None, :]
    state[slots] = new
    return (q.shape[-1] ** -0.5 * (qh[..., None] * new).sum(-2)).to(q.dtype), state


EPS = 1e-6


def plain_norm(x, weight, residual, gate, bits):
    # to 8 bits in 64: a value next to a border goes to the side that it lies on
    wide = torch.float64 if bits == 8 else torch.float32
    h = x.to(wide) if residual is None else x.to(wide) + residual.to(wide)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * weight.to(wide)
    if gate is not None:
        z = gate.to(wide)
        y = y * z * torch.sigmoid(z)
    out = [] if residual is None else [h.to(x.dtype)]
    if bits == 16:
        return [y.to(x.dtype)] + out
    # one scale for each 128 values of a row, the last group as long as it is
    dim = y.shape[-1]
    groups = -(-dim // 128)
    v = torch.nn.functional.pad(y, (0, groups * 128 - dim)).view(*y.shape[:-1], groups, 128)
    scale = (v.abs().amax(-1).clamp(min=TINY) / E4M3_MAX).float()
    q = (v / scale.to(wide)[..., None]).float().clamp(-E4M3_MAX, E4M3_MAX)
    return [q.view(*y.shape[:-1], groups * 128)[..., :dim].contiguous().to(torch.float8_e4m3fn), scale] + out


def plain_norm_bwd(h, weight, gate, dy, dres):
    hf, w, d = h.float(), weight.float(), dy.float()
    r = torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS)
    n = hf * r
    out = []
    if gate is not None:
        z = gate.float()
        e = torch.sigmoid(z)
        out = [(d * n * w * (e * (1 + z * (1 - e)))).to(h.dtype)]
        d = d * z * e
    u = d * w
    dh = r * (u - n * (u * n).mean(-1, keepdim=True)) + dres.float()
    dw = (d * n).reshape(-1, h.shape[-1]).sum(0)
    return [dh.to(h.dtype), dw.to(h.dtype)] + out


def run(s):
    op = s["op"]
    if own:
        import gated_deltanet_chunked_rule_amd as gdr
        if op == "conv":
            return gdr.gdr_causal_conv_fwd(s["x"], s["weight"], s["bias"], s["initial"], s["cu"], output_final_state=True)
        if op == "conv_bwd":
            return gdr.gdr_causal_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], cu_seqlens=s["cu"])[:3]
        if op == "conv_step":
            return gdr.gdr_causal_conv_step(s["x"], s["state"], s["weight"], s["bias"], slots=s["slots"]), s["state"]
        if op == "scan":
            return gdr.gdr_ssm_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"], s["initial"], s["cu"], output_final_state=True)
        if op == "scan_step":
            return gdr.gdr_ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["dt_bias"], slots=s["slots"]), s["state"]
        if op == "rule_step":
            return gdr.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"]), s["state"]
        if op == "norm":
            y, scale, h = gdr.gdr_rms_norm_fwd(s["x"], s["weight"], s["residual"], s["gate"], eps=EPS, quant=s["bits"] == 8)
            return [t for t in (y, scale, h) if t is not None]
        dh, dw, dgate = gdr.gdr_rms_norm_bwd(s["x"], s["weight"], s["dy"], s["gate"], s["dres"], eps=EPS)
        return [t for t in (dh, dw, dgate) if t is not None]
    if op == "conv":
        return plain_conv(s["x"], s["weight"], s["bias"], s["initial"], s["cu"])
    if op == "conv_bwd":
        return plain_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["cu"])
    if op == "conv_step":
        return plain_conv_step(s["x"], s["state"], s["weight"], s["bias"], s["slots"])
    if op == "scan":
        return plain_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"], s["initial"], s["cu"], s["longest"])
    if op == "scan_step":
        return plain_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["dt_bias"], s["slots"])
    if op == "rule_step":
        return plain_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots"])
    if op == "norm":
        return plain_norm(s["x"], s["weight"], s["residual"], s["gate"], s["bits"])
    return plain_norm_bwd(s["x"], s["weight"], s["gate"], s["dy"], s["dres"])


def work(case):
    """Every input read once, every output written once; the operations of the recurrences themselves."""
    op, e = case["op"], 2 if case["type"] == "bf16" else 4
    if op in ("conv", "conv_bwd", "conv_step"):
        D = case["channels"]
        weights = D * (W_TAPS + 1) * e
        if op == "conv_step":
            return {"bytes": case["rows"] * D * e * (2 + 2 * (W_TAPS - 1)) + weights, "flops": case["rows"] * D * (2 * W_TAPS + 5)}
        n = case["tokens"] * D
        states = case["seqs"] * (W_TAPS - 1) * D * e
        if op == "conv":
            return {"bytes": 2 * n * e + weights + states * (2 if case["carried"] else 1), "flops": n * (2 * W_TAPS + 5)}
        return {"bytes": 3 * n * e + 2 * weights, "flops": n * (6 * W_TAPS + 12)}
    if op in ("scan", "scan_step"):
        H, G, P, N = case["heads"], case["groups"], case["P"], case["N"]
        T = case["rows"] if op == "scan_step" else case["tokens"]
        row = (2 * H * P + 2 * G * N + H) * e
        state = H * N * P * 4
        if op == "scan_step":
            return {"bytes": T * (row + 2 * state) + 12 * H, "flops": T * H * N * P * 5}
        # a chunk of 64 tokens: the scores' lower half, their product with x, the state's reading and its update
        chunked = T * H * (65 * N + 65 * P + 4 * N * P)
        return {"bytes": T * row + 12 * H + case["seqs"] * state * (2 if case["carried"] else 1), "flops": chunked}
    if op == "rule_step":
        rows, Hq, Hv, K = case["rows"], case["Hq"], case["Hv"], case["K"]
        return {"bytes": rows * (2 * Hq * K * e + 2 * Hv * K * e + 8 * Hv + 2 * Hv * K * K * 4), "flops": rows * Hv * K * K * 7}
    n = case["rows"] * case["heads"] * case["dim"]
    if op == "norm_bwd":
        return {"bytes": n * e * (6 if case["gate"] else 4) + 2 * case["dim"] * e, "flops": n * 14}
    groups = case["rows"] * case["heads"] * -(-case["dim"] // 128)
    reads = 1 + (1 if case["residual"] else 0) + (1 if case["gate"] else 0)
    writes = (e if case["bits"] == 16 else 1) + (e if case["residual"] else 0)
    return {"bytes": n * (reads * e + writes) + case["dim"] * e + (groups * 4 if case["bits"] == 8 else 0), "flops": n * 8}


# ------------------------------------------------------- exact, in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if op in ("conv", "conv_bwd"):
        return _exact_conv(op, f, s["cu"].tolist())
    if op == "conv_step":
        at = f["slots"].long()
        y = torch.nn.functional.silu(f["bias"] + f["x"] * f["weight"][:, 3] + sum(f["state"][at, j] * f["weight"][:, j] for j in range(3)))
        f["state"][at] = torch.stack([f["state"][at, 1], f["state"][at, 2], f["x"]], 1)
        return y, f["state"]
    if op in ("scan", "scan_step"):
        return _exact_scan(op, f, s["cu"].tolist() if op == "scan" else None)
    if op == "rule_step":
        at, r = f["slots"].long(), f["v"].shape[1] // f["q"].shape[1]
        k, q = f["k"].repeat_interleave(r, 1), f["q"].repeat_interleave(r, 1)
        old = f["state"][at] * f["g"].exp()[..., None, None]
        # (I - beta k k^T) S + beta k v^T, the rule as it is written
        kk = torch.eye(k.shape[-1], device=k.device, dtype=torch.float64) - f["beta"][..., None, None] * k[..., :, None] * k[..., None, :]
        new = kk @ old + f["beta"][..., None, None] * k[..., :, None] * f["v"][..., None, :]
        f["state"][at] = new
        return (q[..., None, :] @ new)[..., 0, :] * k.shape[-1] ** -0.5, f["state"]
    if op == "norm_bwd":
        h, w, z = (f[n].clone().requires_grad_(True) if f[n] is not None else None for n in ("x", "weight", "gate"))
        y = h / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
        y = y if z is None else y * torch.nn.functional.silu(z)
        got = torch.autograd.grad((y * f["dy"]).sum() + (h * f["dres"]).sum(), [t for t in (h, w, z) if t is not None])
        return list(got)
    h = f["x"] if f["residual"] is None else f["x"] + f["residual"]
    y = h / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * f["weight"]
    y = y if f["gate"] is None else y * torch.nn.functional.silu(f["gate"])
    out = [] if f["residual"] is None else [h]
    if case["bits"] == 16:
        return [y] + out
    dim = y.shape[-1]
    parts, scales = [], []
    for a in range(0, dim, 128):
        part = y[..., a:a + 128]
        scale = (part.abs().amax(-1, keepdim=True).clamp(min=TINY) / E4M3_MAX).float().double()
        v = part / scale
        # 3 bits behind the leading one, down to steps of 2^-9
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        parts.append((torch.round(v / unit) * unit).clamp(-E4M3_MAX, E4M3_MAX))
        scales.append(scale)
    return [torch.cat(parts, -1), torch.cat(scales, -1)] + out


def _exact_conv(op, f, cu):
    x = f["x"][0]
    if op == "conv":
        ys, last = [], []
        for n in range(len(cu) - 1):
            before = f["initial"][n] if f["initial"] is not None else x.new_zeros(3, x.shape[1])
            rows = torch.cat([before, x[cu[n]:cu[n + 1]]])
            z = torch.nn.functional.conv1d(rows.t()[None], f["weight"][:, None], f["bias"], groups=x.shape[1])[0].t()
            ys.append(torch.nn.functional.silu(z))
            last.append(rows[-3:])
        return torch.cat(ys)[None], torch.stack(last)
    e = [torch.zeros_like(x), torch.zeros_like(f["weight"]), torch.zeros_like(f["bias"])]
    for n in range(len(cu) - 1):
        rows = torch.nn.functional.pad(x[cu[n]:cu[n + 1]], (0, 0, 3, 0))
        L = cu[n + 1] - cu[n]
        z = f["bias"] + sum(f["weight"][:, j] * rows[j:j + L] for j in range(4))
        sig = torch.sigmoid(z)
        dz = f["dy"][0, cu[n]:cu[n + 1]] * (sig + z * sig * (1 - sig))
        for j in range(4):
            e[0][cu[n]:cu[n + 1] - (3 - j)] += (f["weight"][:, j] * dz)[3 - j:] if L > 3 - j else 0
            e[1][:, j] += (dz * rows[j:j + L]).sum(0)
        e[2] += dz.sum(0)
    return e[0][None], e[1], e[2]


def _exact_scan(op, f, cu):
    """The recurrence, token by token, all sequences side by side."""
    step = torch.nn.functional.softplus(f["dt"] + f["dt_bias"], threshold=1e9)
    r = f["x"].shape[-2] // f["B"].shape[-2]

    def token(h, x, d, B, C):
        h = h * (d * f["A"]).exp()[..., None, None] + B.repeat_interleave(r, 1)[..., None] * (d[..., None] * x)[..., None, :]
        return h, (C.repeat_interleave(r, 1)[..., None, :] @ h)[..., 0, :] + f["D"][:, None] * x

    if op == "scan_step":
        at = f["slots"].long()
        f["state"][at], y = token(f["state"][at], f["x"], step, f["B"], f["C"])
        return y, f["state"]
    x, B, C, step = f["x"][0], f["B"][0], f["C"][0], step[0]
    N = len(cu) - 1
    order = sorted(range(N), key=lambda n: cu[n] - cu[n + 1])     # the longest first: those that go on are the first ones
    h = x.new_zeros(N, x.shape[1], B.shape[2], x.shape[2]) if f["initial"] is None else f["initial"][torch.tensor(order, device=x.device)]
    first = torch.tensor([cu[n] for n in order], device=x.device)
    y = torch.zeros_like(x)
    live = N
    for i in range(cu[order[0] + 1] - cu[order[0]]):
        while cu[order[live - 1] + 1] - cu[order[live - 1]] <= i:
            live -= 1
        at = first[:live] + i
        h[:live], y[at] = token(h[:live], x[at], step[at], B[at], C[at])
    back = torch.empty_like(h)
    back[torch.tensor(order, device=x.device)] = h
    return y[None], back

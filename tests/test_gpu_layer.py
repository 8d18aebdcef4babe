"""The operators around the rule on the GPU against their plain 64-bit forms
(layer_reference.py, which states how the bounds come about)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
import gdr_inputs as gi
import layer_reference as ref
from layer_reference import check, gen, randn
from parity import TOL, dev, f64, oracle_fwd, rel_err

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
cuda = lambda t: None if t is None else t.to("cuda")  # noqa: E731  (keeps strides)


def sliced(t, extra=8, at=4):
    """The same values as a slice of a wider row (offset and width in elements of the last dimension)."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., at:at + t.shape[-1]] = t
    return wide[..., at:at + t.shape[-1]]


# ------------------------------------------------------------ convolution --
CONV = [
    # B, T, D, W, type, cu, carried
    (1, 1, 8, 4, BF, None, False),
    (1, 1, 1, 2, F32, None, True),
    (2, 7, 67, 4, BF, None, True),          # odd rows: no element group is aligned
    (3, 33, 13, 3, F32, None, False),
    (2, 100, 256, 2, BF, None, True),
    (1, 41, 96, 4, BF, [0, 1, 1, 3, 6, 40, 41], True),       # shorter than the taps, empty, long
    (1, 41, 30, 4, F32, [0, 1, 1, 3, 6, 40, 41], True),
    (1, 50, 72, 3, BF, [5, 5, 17, 44], True),                # tokens before the first and behind the last sequence
    (1, 700, 520, 4, BF, [0, 333, 600, 700], False),
    (1, 4, 24, 4, BF, [0, 0, 0], True),                      # no sequence has a token
]


def conv_case(i, B, T, D, W, dtype, cu, carried):
    g = gen(100 + i)
    N = B if cu is None else len(cu) - 1
    x = sliced(randn(g, B, T, D, dtype=dtype), 3 if D % 2 else 8, 1 if D % 2 else 4)
    return dict(x=x, weight=randn(g, D, W, dtype=dtype, std=0.5), bias=randn(g, D, dtype=dtype) if i % 3 else None,
                h0=randn(g, N, W - 1, D, dtype=dtype) if carried else None,
                cu=None if cu is None else torch.tensor(cu, dtype=torch.int32),
                dy=randn(g, B, T, D, dtype=dtype), dht=randn(g, N, W - 1, D, dtype=dtype))


@pytest.mark.parametrize("i", range(len(CONV)))
def test_conv_fwd(i):
    c = conv_case(i, *CONV[i])
    act = i % 4 != 3
    y, ht = gdr.gdr_causal_conv_fwd(cuda(c["x"]), cuda(c["weight"]), cuda(c["bias"]), cuda(c["h0"]), cuda(c["cu"]),
                                    activation="silu" if act else None, output_final_state=True)
    ry, rm, rht = ref.conv(c["x"], c["weight"], c["bias"], c["h0"], c["cu"], act)
    check(y, ry, rm, label="y")
    assert torch.equal(ht.cpu().double(), rht)      # inputs, moved


@pytest.mark.parametrize("i", range(len(CONV)))
def test_conv_bwd(i):
    c = conv_case(i, *CONV[i])
    act = i % 4 != 3
    got = gdr.gdr_causal_conv_bwd(cuda(c["x"]), cuda(c["weight"]), cuda(c["bias"]), cuda(c["dy"]), cuda(c["h0"]), cuda(c["dht"]),
                                  cuda(c["cu"]), activation="silu" if act else None)
    want = ref.conv_bwd(c["x"], c["weight"], c["bias"], c["dy"], c["h0"], c["dht"], c["cu"], act)
    for name, t, r, given in zip(("dx", "dw", "db", "dh0"), got, want, (1, 1, c["bias"] is not None, c["h0"] is not None)):
        if not given:
            assert t is None
        else:
            check(t, *r, label=name)


def test_conv_with_more_sequences_than_the_staged_table():
    g = gen(5)
    lens = [(7 * i) % 4 for i in range(1500)]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    T = int(cu[-1])
    x, w, dy = randn(g, 1, T, 16, dtype=F32), randn(g, 16, 4), randn(g, 1, T, 16)
    y, ht = gdr.gdr_causal_conv_fwd(cuda(x), cuda(w), None, None, cuda(cu), output_final_state=True)
    ry, rm, rht = ref.conv(x, w, None, None, cu)
    check(y, ry, rm)
    assert torch.equal(ht.cpu().double(), rht)
    dx, dw, _, _ = gdr.gdr_causal_conv_bwd(cuda(x), cuda(w), None, cuda(dy), cu_seqlens=cuda(cu))
    want = ref.conv_bwd(x, w, None, dy, None, None, cu)
    check(dx, *want[0], label="dx")
    check(dw, *want[1], label="dw")


def test_conv_gradient_agrees_with_differences():
    # central differences of the kernel's own fp32 forward along random directions: the loss is a sum of about
    # T D = 2000 terms of size 1 with fp32 errors 2^-20 each, so a step of 2^-6 leaves about
    # sqrt(2000) 2^-20 / 2^-6 = 3e-3 and the third-order term about 2^-12 sum |f'''| / 6 = 0.05
    g = gen(6)
    x, w, b, h0 = randn(g, 2, 40, 24), randn(g, 24, 4, std=0.5), randn(g, 24), randn(g, 2, 3, 24)
    dy, dht = randn(g, 2, 40, 24), randn(g, 2, 3, 24)
    got = gdr.gdr_causal_conv_bwd(cuda(x), cuda(w), cuda(b), cuda(dy), cuda(h0), cuda(dht))

    def loss(*a):
        y, ht = gdr.gdr_causal_conv_fwd(*map(cuda, a), output_final_state=True)
        return float((y.cpu().double() * dy).sum() + (ht.cpu().double() * dht).sum())

    args, eps = [x, w, b, h0], 2.0 ** -6
    for k, grad in enumerate(got):
        d = randn(g, *args[k].shape)
        d = d / d.norm()
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + eps * d, args[k] - eps * d
        num, ana = (loss(*up) - loss(*dn)) / (2 * eps), float((grad.cpu().double() * d).sum())
        print(k, num, ana, flush=True)
        assert abs(num - ana) <= 0.06


@pytest.mark.parametrize("rows,D,W,dtype", [(1, 5, 4, BF), (3, 600, 2, F32), (70, 96, 4, BF), (9, 1025, 3, BF)])
def test_conv_step_padding_and_pool(rows, D, W, dtype):
    g = gen(rows)
    x = sliced(randn(g, rows, D, dtype=dtype), 1, 1)
    w, b, pool = randn(g, D, W, dtype=dtype), randn(g, D, dtype=dtype), randn(g, rows + 2, W - 1, D, dtype=dtype)
    slots = torch.randperm(rows + 2, generator=g)[:rows].to(torch.int32)
    pad = torch.zeros(rows, dtype=torch.bool)
    if rows >= 3:
        slots[0], slots[2] = -1, slots[1]        # out of the pool; named before
        pad[0] = pad[2] = True
    if rows > 60:
        slots[-1] = rows + 2
        slots[-2] = slots[1]
        pad[-1] = pad[-2] = True
    state = cuda(pool)
    y = gdr.gdr_causal_conv_step(cuda(x), state, cuda(w), cuda(b), slots=cuda(slots))
    new = pool.clone()
    for r in range(rows):
        if pad[r]:
            assert not y[r].any()
            continue
        s = int(slots[r])
        ry, rm, rht = ref.conv(x[r][None, None], w, b, pool[s][None])
        check(y[r], ry[0, 0], rm[0, 0], label=f"row {r}")
        new[s] = rht[0].to(dtype)
    assert torch.equal(state.cpu(), new)


# ------------------------------------------------------ gated delta rule --
def rule_case(g, rows, Hq, Hv, K, dtype):
    unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(dtype)  # noqa: E731
    return dict(q=unit(randn(g, rows, Hq, K)), k=unit(randn(g, rows, Hq, K)), v=randn(g, rows, Hv, K, dtype=dtype),
                g=torch.log(0.85 + 0.15 * torch.rand(rows, Hv, generator=g)), beta=torch.sigmoid(randn(g, rows, Hv)))


@pytest.mark.parametrize("rows,Hq,Hv,K,dtype", [(1, 1, 1, 32, F32), (1, 2, 4, 128, BF), (5, 1, 3, 64, BF), (7, 4, 4, 128, F32),
                                                (70, 2, 8, 64, BF), (66, 16, 32, 32, BF)])
def test_rule_step(rows, Hq, Hv, K, dtype):
    g = gen(rows + K)
    c = rule_case(g, rows, Hq, Hv, K, dtype)
    wide = torch.full((rows, (2 * Hq + Hv) * K + 16), float("nan"), dtype=dtype)    # q, k, v as slices of one row
    at = 8
    for n in ("q", "k", "v"):
        part = wide[:, at:at + c[n][0].numel()].unflatten(-1, tuple(c[n].shape[1:]))
        part.copy_(c[n])
        c[n], at = part, at + c[n][0].numel()
    pool = randn(g, rows + 2, Hv, K, K, std=0.1)
    slots = torch.randperm(rows + 2, generator=g)[:rows].to(torch.int32)
    live = torch.ones(rows, dtype=torch.bool)
    if rows > 4:
        slots[1], slots[3], slots[4] = 2 ** 31 - 1, -5, slots[0]
        live[1] = live[3] = live[4] = False
    wide_d = wide.to("cuda")
    view = lambda t, o: wide_d[:, o:o + t[0].numel()].unflatten(-1, tuple(t.shape[1:]))  # noqa: E731
    state = cuda(pool)
    o = gdr.gdr_step(view(c["q"], 8), view(c["k"], 8 + Hq * K), view(c["v"], 8 + 2 * Hq * K), cuda(c["g"]), cuda(c["beta"]), state,
                     slots=cuda(slots))
    at = slots[live].long()
    ro, rm, rs, rsm = ref.rule_step(*(c[n][live] for n in ("q", "k", "v", "g", "beta")), pool[at], K ** -0.5)
    check(o.cpu()[live], ro, rm, label="o")
    check(state.cpu()[at], rs, rsm, label="state")
    assert not o.cpu()[~live].any()
    others = torch.ones(rows + 2, dtype=torch.bool)
    others[at] = False
    assert torch.equal(state.cpu()[others], pool[others])


def test_rule_steps_agree_with_the_oracle():
    w = gi.custom(B=3, T=9, Hq=2, Hv=4, K=64, V=64, dtype="bf16", seed=5, initial_state=True)
    inp = gi.make_inputs(w)
    ro, rht = oracle_fwd(inp)
    state = dev(inp["initial_state"]).clone()
    o = [gdr.gdr_step(*(dev(inp[n][:, t]) for n in ("q", "k", "v", "g", "beta")), state, inp["scale"]) for t in range(9)]
    assert rel_err(torch.stack(o, 1), ro) <= 2.0 ** -8 + 1e-5
    assert rel_err(state, rht) <= 1e-5


# -------------------------------------------------------------------- scan --
def scan_check(c, y, ht, cu=None, use_softplus=True, skip=True):
    ry, rm, rh, rhm = ref.scan(c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"] if skip else None, c["bias"], c["h0"], cu, use_softplus)
    # bf16: the scores times decays, and the state, each take one rounding as operands of their products with x and C
    check(y, ry, rm, slack=2.0 ** -8 if y.dtype == BF else 2.0 ** -17, label="y")
    check(ht, rh, rhm, slack=2.0 ** -17, label="state")


def run_scan(c, cu=None, **kw):
    P, H = c["x"].shape[3], c["x"].shape[2]
    G, N = c["B"].shape[2:]
    row = c["row"].to("cuda")
    x, B, C = (t.unflatten(-1, s) for t, s in zip(row.split([H * P, G * N, G * N], -1), ((H, P), (G, N), (G, N))))
    return gdr.gdr_ssm_scan_fwd(x, cuda(c["dt"]), cuda(c["A"]), B, C, cuda(c["D"]), cuda(c["bias"]), cuda(c["h0"]), cuda(cu),
                                output_final_state=True, **kw)


@pytest.mark.parametrize("b,T,H,G,P,N,dtype", [
    (1, 1, 1, 1, 32, 32, BF), (1, 1, 2, 1, 64, 128, F32), (2, 63, 3, 1, 64, 64, BF), (1, 64, 4, 2, 32, 128, BF),
    (1, 65, 5, 5, 128, 32, F32), (2, 130, 2, 1, 128, 128, BF), (1, 129, 2, 2, 64, 128, F32), (1, 300, 9, 3, 32, 64, F32),
    (1, 600, 4, 1, 64, 128, BF),       # three segments
    (2, 1100, 2, 1, 32, 32, F32),      # segments that end inside a batch row
    (1, 1000, 2, 2, 128, 64, BF),
])
def test_scan(b, T, H, G, P, N, dtype):
    c = ref.scan_inputs(gen(T + H), b, T, H, G, P, N, dtype)
    scan_check(c, *run_scan(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cu", [[0, 1, 1, 2, 66, 130, 600, 600, 640], [3, 200, 256, 512, 513, 620], [0, 0, 0], [0, 64, 128, 256, 640],
                                list(range(0, 641, 1))])
def test_scan_packed(cu, dtype):
    c = ref.scan_inputs(gen(len(cu)), 1, 640, 4, 2, 32, 32, dtype, seqs=len(cu) - 1)
    cu = torch.tensor(cu, dtype=torch.int32)
    scan_check(c, *run_scan(c, cu), cu=cu)


@pytest.mark.parametrize("H,G,P,N", [(10, 2, 64, 128), (6, 1, 128, 64), (7, 1, 64, 32)])
def test_scan_packed_with_a_part_of_a_workgroups_channels(H, G, P, N):
    cu = torch.tensor([2, 2, 70, 71, 199, 460, 460, 600], dtype=torch.int32)
    c = ref.scan_inputs(gen(H), 1, 640, H, G, P, N, BF, seqs=len(cu) - 1)
    scan_check(c, *run_scan(c, cu), cu=cu)


def test_scan_without_options_and_initial_state():
    c = ref.scan_inputs(gen(3), 2, 90, 2, 1, 64, 64, F32)
    c["dt"] = torch.nn.functional.softplus(c["dt"] - 3)
    y, ht = gdr.gdr_ssm_scan_fwd(*(cuda(c[n].contiguous()) for n in ("x", "dt", "A", "B", "C")), dt_softplus=False)
    assert ht is None
    c.update(bias=None, h0=None)
    ry, rm, _, _ = ref.scan(c["x"], c["dt"], c["A"], c["B"], c["C"], use_softplus=False)
    check(y, ry, rm, slack=2.0 ** -17)


def test_scan_strong_decay_and_none():
    # decays that underflow within a chunk, and A = 0: a plain sum over 700 tokens
    c = ref.scan_inputs(gen(4), 1, 700, 4, 1, 32, 64, BF)
    c["A"] = torch.tensor([-1000.0, -100.0, 0.0, -1e-3])
    scan_check(c, *run_scan(c))


def test_scan_keeps_what_is_not_finite_to_its_sequence():
    # NaN and infinities in one sequence, and in rows of no sequence, reach no other one
    c = ref.scan_inputs(gen(5), 1, 400, 2, 1, 64, 64, BF)
    cu = torch.tensor([0, 100, 130, 390], dtype=torch.int32)
    c["h0"] = randn(gen(6), 3, 2, 64, 64)
    clean_y, clean_h = run_scan(c, cu)
    c["row"][:, 100:130] = float("nan")
    c["row"][:, 390:] = float("inf")
    c["dt"][:, 100:130] = float("nan")
    y, ht = run_scan(c, cu)
    for s in (slice(0, 100), slice(130, 390)):
        assert torch.equal(y[:, s], clean_y[:, s])
    assert not y[:, 390:].any()
    assert torch.equal(ht[0], clean_h[0]) and torch.equal(ht[2], clean_h[2]) and ht[1].isnan().any()


@pytest.mark.parametrize("what", ["x", "dt", "B", "C", "all"])
@pytest.mark.parametrize("H,P,N,dtype", [(4, 64, 128, BF), (8, 32, 32, BF), (2, 64, 64, F32)])
def test_scan_keeps_what_is_not_finite_from_earlier_tokens(H, P, N, dtype, what):
    # a padded batch whose rows end anywhere in a chunk and hold anything behind that
    c = ref.scan_inputs(gen(P + N), 4, 400, H, 1, P, N, dtype)
    clean, _ = run_scan(c)
    widths = {"x": slice(0, H * P), "B": slice(H * P, H * P + N), "C": slice(H * P + N, H * P + 2 * N), "all": slice(0, H * P + 2 * N)}
    ends = (1, 77, 207, 399)
    for b, end in enumerate(ends):
        bad = float("nan") if b % 2 else float("-inf")
        if what in widths:
            c["row"][b, end:, widths[what]] = bad
        if what in ("dt", "all"):
            c["dt"][b, end:] = bad
    y, _ = run_scan(c)
    for b, end in enumerate(ends):
        assert torch.equal(y[b, :end], clean[b, :end])
        if what in ("x", "all"):
            assert not torch.isfinite(y[b, end:]).any()


def test_scan_keeps_what_is_not_finite_to_its_channel():
    # one value of x: its channel's outputs from there on, its column of the state, and nothing else
    c = ref.scan_inputs(gen(8), 1, 300, 8, 2, 64, 64, BF)
    clean_y, clean_h = run_scan(c)
    c["row"][0, 170, 3 * 64 + 37] = float("inf")
    y, ht = run_scan(c)
    assert not torch.isfinite(y[0, 170:, 3, 37]).any() and not torch.isfinite(ht[0, 3, :, 37]).any()
    for got, want in ((y[0], clean_y[0]), (ht, clean_h)):
        got, want = got.clone(), want.clone()
        where = (slice(170, None), 3, 37) if got.dim() == 3 else (0, 3, slice(None), 37)
        got[where] = want[where] = 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("rows,H,G,P,N,dtype", [(1, 1, 1, 32, 32, BF), (3, 4, 2, 64, 128, F32), (70, 6, 1, 128, 64, BF), (64, 8, 8, 64, 128, BF)])
def test_ssm_step(rows, H, G, P, N, dtype):
    g = gen(rows + N)
    c = ref.scan_inputs(g, rows, 1, H, G, P, N, dtype, seqs=rows + 2)
    slots = torch.randperm(rows + 2, generator=g)[:rows].to(torch.int32)
    live = torch.ones(rows, dtype=torch.bool)
    if rows > 2:
        slots[0], slots[2] = rows + 2, slots[1]
        live[0] = live[2] = False
    row = c["row"].to("cuda")[:, 0]
    x, B, C = (t.unflatten(-1, s) for t, s in zip(row.split([H * P, G * N, G * N], -1), ((H, P), (G, N), (G, N))))
    state = cuda(c["h0"])
    y = gdr.gdr_ssm_step(x, cuda(c["dt"][:, 0]), cuda(c["A"]), B, C, state, cuda(c["D"]), cuda(c["bias"]), slots=cuda(slots))
    at = slots[live].long()
    ry, rm, rh, rhm = ref.scan(*(c[n][live] for n in ("x", "dt")), c["A"], c["B"][live], c["C"][live], c["D"], c["bias"], c["h0"][at])
    check(y.cpu()[live], ry[:, 0], rm[:, 0], label="y")
    check(state.cpu()[at], rh, rhm, label="state")
    assert not y.cpu()[~live].any()
    others = torch.ones(rows + 2, dtype=torch.bool)
    others[at] = False
    assert torch.equal(state.cpu()[others], c["h0"][others])


# -------------------------------------------------------------------- norm --
NORM = [
    # shape, type, residual, gate
    ((1, 1), F32, False, False), ((3, 7), BF, True, True), ((2, 5, 128), BF, False, True), ((5, 129), F32, True, False),
    ((4, 3, 200), BF, True, True), ((9, 512), BF, True, False), ((3, 700), F32, False, True), ((2, 1023), BF, True, False),
    ((5, 2048), BF, False, False), ((2, 4096), F32, True, True), ((3, 4100), BF, True, False), ((2, 8192), BF, False, True),
    ((2, 9000), F32, True, False), ((1, 16384), BF, True, True), ((1100, 64), BF, False, False), ((2, 40, 16, 64), BF, False, True),
]


def norm_case(i, shape, dtype, residual, gate):
    g = gen(300 + i)
    return dict(x=sliced(randn(g, *shape, dtype=dtype)), weight=(1 + randn(g, shape[-1], std=0.2)).to(dtype),
                residual=sliced(randn(g, *shape, dtype=dtype, std=3), 5, 1) if residual else None,
                gate=sliced(randn(g, *shape, dtype=dtype, std=2)) if gate else None,
                dy=randn(g, *shape, dtype=dtype), dres=randn(g, *shape, dtype=dtype) if residual else None)


def wide_cuda(t):
    """A slice moved to the GPU as a slice (with its whole base)."""
    if t is None:
        return None
    base = t._base.to("cuda")
    return base.as_strided(t.shape, t.stride(), t.storage_offset())


@pytest.mark.parametrize("i", range(len(NORM)))
def test_norm_fwd(i):
    c = norm_case(i, *NORM[i])
    args = [wide_cuda(c["x"]), cuda(c["weight"]), wide_cuda(c["residual"]), wide_cuda(c["gate"])]
    y, scales, h = gdr.gdr_rms_norm_fwd(*args, eps=1e-5)
    ry, rm, rh = ref.norm(c["x"], c["weight"], c["residual"], c["gate"], 1e-5)
    check(y, ry, rm, label="y")
    assert scales is None and (h is None) == (c["residual"] is None)
    if h is not None:
        assert torch.equal(h.cpu(), (c["x"].float() + c["residual"].float()).to(c["x"].dtype))
    q, scales, _ = gdr.gdr_rms_norm_fwd(*args, eps=1e-5, quant=True)
    rs, bound = ref.e4m3_parts(ry)
    check(scales, rs, rs, label="scales")
    full = scales.cpu().double().repeat_interleave(128, -1)[..., :ry.shape[-1]]
    assert bool(((q.cpu().float().double() * full - ry).abs() <= bound).all())


@pytest.mark.parametrize("i", range(len(NORM)))
def test_norm_bwd(i):
    c = norm_case(i, *NORM[i])
    got = gdr.gdr_rms_norm_bwd(wide_cuda(c["x"]), cuda(c["weight"]), cuda(c["dy"]), wide_cuda(c["gate"]), cuda(c["dres"]), eps=1e-5)
    want = ref.norm_bwd(c["x"], c["weight"], c["dy"], c["gate"], c["dres"], 1e-5)
    for name, t, r in zip(("dh", "dw", "dgate"), got, want):
        if r is None:
            assert t is None
        else:
            check(t, *r, label=name)


def test_norm_edge_values():
    # zero rows, rows whose squares underflow, NaN and infinity keep to their rows; a NaN's group is NaN
    x = torch.zeros(5, 256)
    x[1] = 1e-30
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    x[4] = torch.linspace(-3, 3, 256)
    w = torch.ones(256)
    y, _, _ = gdr.gdr_rms_norm_fwd(cuda(x), cuda(w), eps=0.0)
    assert y[0].isnan().all() and y[2].isnan().all()          # 0 / 0, as the formula says
    y, _, _ = gdr.gdr_rms_norm_fwd(cuda(x), cuda(w))
    assert not y[0].any() and torch.isfinite(y[1]).all() and y[2].isnan().all() and y[3, 200].isnan()
    ry, rm, _ = ref.norm(x[4:5], w)
    check(y[4:5], ry, rm)
    q, s, _ = gdr.gdr_rms_norm_fwd(cuda(x), cuda(w), quant=True)
    assert not q[0].float().any() and bool((s[0] > 0).all()) and bool(torch.isfinite(s[0]).all())
    assert q[2].float().isnan().all() and s[2].isnan().all()
    assert q[3, 200].float().isnan() and not q[3, :128].float().any()


def test_norm_of_no_rows():
    w = torch.ones(64, device="cuda", dtype=BF)
    y, s, h = gdr.gdr_rms_norm_fwd(torch.empty(0, 64, device="cuda", dtype=BF), w, quant=True)
    assert y.shape == (0, 64) and s.shape == (0, 1)
    dh, dw, _ = gdr.gdr_rms_norm_bwd(torch.empty(0, 64, device="cuda", dtype=BF), w, torch.empty(0, 64, device="cuda", dtype=BF))
    assert not dw.any()


def test_norm_gradient_agrees_with_differences():
    # as for the convolution: 2000 terms of size 1, a step of 2^-6 along a unit direction
    g = gen(8)
    x, w, z, dy = randn(g, 8, 2, 128), 1 + randn(g, 128, std=0.1), randn(g, 8, 2, 128), randn(g, 8, 2, 128)
    got = gdr.gdr_rms_norm_bwd(cuda(x), cuda(w), cuda(dy), cuda(z))

    def loss(x, w, z):
        return float((gdr.gdr_rms_norm_fwd(cuda(x), cuda(w), None, cuda(z))[0].cpu().double() * dy).sum())

    args, eps = [x, w, z], 2.0 ** -6
    for k, grad in enumerate(got):
        d = randn(g, *args[k].shape)
        d = d / d.norm()
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + eps * d, args[k] - eps * d
        num, ana = (loss(*up) - loss(*dn)) / (2 * eps), float((grad.cpu().double() * d).sum())
        assert abs(num - ana) <= 0.06, (k, num, ana)


# ------------------------------------------------------------ as a user has them --
def test_autograd_of_conv_and_norm():
    g = gen(9)
    x, w, b = (cuda(t).requires_grad_(True) for t in (randn(g, 1, 50, 32), randn(g, 32, 4), randn(g, 32)))
    h0 = cuda(randn(g, 2, 3, 32)).requires_grad_(True)
    y, ht = gdr.causal_conv(x, w, b, h0, True, [0, 20, 50])
    n, wn, z = cuda(randn(g, 1, 50, 32)).requires_grad_(True), cuda(randn(g, 32)).requires_grad_(True), cuda(randn(g, 1, 50, 32)).requires_grad_(True)
    o, h = gdr.rms_norm(y, wn, n, z)
    do, dh, dht = randn(g, 1, 50, 32), randn(g, 1, 50, 32), randn(g, 2, 3, 32)
    grads = torch.autograd.grad((o, h, ht), (x, w, b, h0, n, wn, z), (cuda(do), cuda(dh), cuda(dht)))
    cu = [0, 20, 50]
    yd = y.detach().cpu()
    (gn, _), (gw, gwm), (gz, gzm) = ref.norm_bwd(yd + n.detach().cpu(), wn, do, z, dh)
    want = ref.conv_bwd(x, w, b, gn.float(), h0, dht, cu)
    # a gradient that went through two operators carries the first one's fp32 error into the second: 2^-15 of the magnitudes
    for t, r in zip(grads[:4], want):
        check(t, *r, slack=2.0 ** -15)
    check(grads[4], gn, gn.abs() + dh.abs().double() + 1, slack=2.0 ** -15)
    check(grads[5], gw, gwm, slack=2.0 ** -15)
    check(grads[6], gz, gzm, slack=2.0 ** -15)
    # only one of the outputs is used
    y, ht = gdr.causal_conv(x, w, b, h0, True, [0, 20, 50])
    gx, gh = torch.autograd.grad(ht.sum(), (x, h0))
    assert float(gx.sum()) == 2 * 3 * 32 and not gh.any()
    o, h = gdr.rms_norm(x, wn, n)
    assert torch.equal(torch.autograd.grad(h.sum(), n)[0], torch.ones_like(n))


def layer_parts(g, T, Hq, Hv, K, B=1):
    D = (2 * Hq + Hv) * K
    return dict(row=randn(g, B, T, D + Hv * K, dtype=BF), w=randn(g, D, 4, dtype=BF, std=0.5), b=randn(g, D, dtype=BF, std=0.2),
                g=torch.log(0.85 + 0.15 * torch.rand(B, T, Hv, generator=g)), beta=torch.sigmoid(randn(g, B, T, Hv)),
                wn=(1 + randn(g, K, std=0.1)).to(BF))


def mixer_prompt(p, Hq, Hv, K, cu):
    """Convolution, the rule and the gated norm, as a layer runs a packed batch of prompts."""
    D = (2 * Hq + Hv) * K
    x, z = p["row"][..., :D], p["row"][..., D:].unflatten(-1, (Hv, K))
    y, conv_state = gdr.gdr_causal_conv_fwd(x, p["w"], p["b"], None, cu, output_final_state=True)
    q, k, v = (t.unflatten(-1, (-1, K)) for t in y.split([Hq * K, Hq * K, Hv * K], -1))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF) for t in (q, k))
    o, state, _, _ = gdr.gdr_chunk_fwd(q, k, v.contiguous(), p["g"], p["beta"], None, None, cu)
    y8, scales, _ = gdr.gdr_rms_norm_fwd(o, p["wn"], None, z, quant=True)
    return o, y8, scales, conv_state, state


def test_layer_prompts_then_tokens():
    """Prompts through convolution, rule and gated norm, then one token of each sequence on the carried states, against
    the prompts with that token at once."""
    Hq, Hv, K, lens = 2, 4, 64, [70, 1, 129]
    D = (2 * Hq + Hv) * K
    p = layer_parts(gen(11), sum(lens) + 3, Hq, Hv, K)
    p = {n: cuda(t) for n, t in p.items()}
    ends = torch.tensor([0] + [n + 1 for n in lens]).cumsum(0)
    full = mixer_prompt(p, Hq, Hv, K, cuda(ends.to(torch.int32)))
    keep = torch.tensor([i for n in range(3) for i in range(int(ends[n]), int(ends[n + 1]) - 1)], device="cuda")
    new = (ends[1:] - 1).to("cuda")
    part = {n: (t[:, keep].contiguous() if n in ("row", "g", "beta") else t) for n, t in p.items()}
    cu = cuda(torch.tensor([0] + lens).cumsum(0).to(torch.int32))
    _, _, _, conv_state, state = mixer_prompt(part, Hq, Hv, K, cu)
    # the pools hold the sequences in another order, with a free slot
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    conv_pool, pool = conv_state.new_zeros(4, 3, D), state.new_zeros(4, Hv, K, K)
    conv_pool[slots.long()], pool[slots.long()] = conv_state, state
    row = p["row"][0, new]
    y = gdr.gdr_causal_conv_step(row[:, :D], conv_pool, p["w"], p["b"], slots=slots)
    q, k, v = (t.unflatten(-1, (-1, K)) for t in y.split([Hq * K, Hq * K, Hv * K], -1))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF) for t in (q, k))
    o = gdr.gdr_step(q, k, v, p["g"][0, new], p["beta"][0, new], pool, slots=slots)
    y8, scales, _ = gdr.gdr_rms_norm_fwd(o, p["wn"], None, row[:, D:].unflatten(-1, (Hv, K)), quant=True)
    fo, fy, fs, fc, fst = full
    assert torch.equal(conv_pool[slots.long()], fc)
    assert rel_err(o, f64(fo[0, new])) <= TOL["bf16"]["o"]
    assert rel_err(pool[slots.long()], f64(fst)) <= TOL["bf16"]["final_state"]
    a, b = y8.float() * scales, fy[0, new].float() * fs[0, new]
    assert rel_err(a, f64(b)) <= TOL["bf16"]["o"] + 2.0 ** -3
    assert not conv_pool[1].any() and not pool[1].any()


def test_scan_prompt_then_tokens():
    H, G, P, N = 4, 2, 64, 128
    c = ref.scan_inputs(gen(12), 2, 203, H, G, P, N, F32)
    t = {n: cuda(v.contiguous()) for n, v in c.items()}
    y, last = gdr.gdr_ssm_scan_fwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["bias"], t["h0"], output_final_state=True)
    cut = 200
    s = lambda n: t[n][:, :cut].contiguous()  # noqa: E731
    _, state = gdr.gdr_ssm_scan_fwd(s("x"), s("dt"), t["A"], s("B"), s("C"), t["D"], t["bias"], t["h0"], output_final_state=True)
    for i in range(cut, 203):
        yi = gdr.gdr_ssm_step(t["x"][:, i], t["dt"][:, i], t["A"], t["B"][:, i], t["C"][:, i], state, t["D"], t["bias"])
        assert rel_err(yi, f64(y[:, i])) <= 1e-5
    assert rel_err(state, f64(last)) <= 1e-5


def test_deterministic_and_on_another_stream():
    c = ref.scan_inputs(gen(13), 1, 900, 4, 1, 64, 64, BF)
    k = conv_case(2, 2, 300, 256, 4, BF, None, True)
    h, w, dy = (cuda(randn(gen(1), *s, dtype=BF)) for s in ((500, 256), (256,), (500, 256)))

    def all_of_it():
        return [*run_scan(c), *gdr.gdr_causal_conv_bwd(cuda(k["x"]), cuda(k["weight"]), None, cuda(k["dy"]), cuda(k["h0"]))[:2],
                *gdr.gdr_rms_norm_bwd(h, w, dy)[:2]]

    first = all_of_it()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        second = all_of_it()
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_captured_serving_step_replays():
    """Convolution, rule and norm steps, a packed prompt scan and a packed convolution captured into one graph, replayed on
    new inputs, slots and offsets."""
    Hq, Hv, K, rows = 2, 4, 64, 6
    D = (2 * Hq + Hv) * K
    p = {n: cuda(t) for n, t in layer_parts(gen(14), rows, Hq, Hv, K).items()}
    c = ref.scan_inputs(gen(15), 1, 600, 4, 1, 64, 64, BF, seqs=3)
    s = {n: cuda(v.contiguous()) for n, v in c.items()}
    cu = torch.tensor([0, 100, 420, 600], dtype=torch.int32, device="cuda")
    slots = torch.arange(rows, dtype=torch.int32, device="cuda")
    conv_pool = cuda(randn(gen(16), rows + 2, 3, D, dtype=BF))
    pool = cuda(randn(gen(17), rows + 2, Hv, K, K, std=0.1))

    def work():
        y = gdr.gdr_causal_conv_step(p["row"][0, :, :D], conv_pool, p["w"], p["b"], slots=slots)
        q, k, v = (t.unflatten(-1, (-1, K)) for t in y.split([Hq * K, Hq * K, Hv * K], -1))
        o = gdr.gdr_step(q, k, v, p["g"][0], p["beta"][0], pool, slots=slots)
        n, sc, _ = gdr.gdr_rms_norm_fwd(o, p["wn"], None, p["row"][0, :, D:].unflatten(-1, (Hv, K)), quant=True)
        z, zl = gdr.gdr_ssm_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["bias"], s["h0"], cu, output_final_state=True)
        f, fl = gdr.gdr_causal_conv_fwd(s["row"], cvw, None, None, cu, output_final_state=True)
        return [y, o, n.view(torch.uint8), sc, z, zl, f, fl]

    cvw = cuda(randn(gen(18), s["row"].shape[-1], 4, dtype=BF))
    start = (conv_pool.clone(), pool.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for r in range(4):
        g = gen(50 + r)
        p["row"].copy_(randn(g, *p["row"].shape))
        s["x"].copy_(randn(g, *s["x"].shape))
        slots.copy_(torch.randperm(rows + 2, generator=g)[:rows])
        cu.copy_(torch.tensor([0, 1 + r, 300 + 70 * r, 600 - 13 * r]))
        conv_pool.copy_(start[0])
        pool.copy_(start[1])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [conv_pool.clone(), pool.clone()]
        conv_pool.copy_(start[0])
        pool.copy_(start[1])
        want = work() + [conv_pool, pool]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), r


def test_python_refuses_on_the_device():
    def raises(msg, f, *a, **kw):
        with pytest.raises(gdr.GdrError, match=msg):
            f(*a, **kw)

    t = lambda *s, dtype=BF: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    raises("expanded", gdr.gdr_causal_conv_fwd, t(1, 1, 16).expand(1, 5, 16), t(16, 4))
    raises("one stride", gdr.gdr_causal_conv_fwd, t(4, 2, 16).transpose(0, 1), t(16, 4))
    raises("contiguous", gdr.gdr_causal_conv_fwd, t(1, 16, 5).transpose(1, 2), t(16, 4))
    raises("shape mismatch", gdr.gdr_causal_conv_fwd, t(1, 5, 16), t(15, 4))
    raises("must be torch.bfloat16", gdr.gdr_causal_conv_fwd, t(1, 5, 16), t(16, 4, dtype=F32))
    raises("W must be", gdr.gdr_causal_conv_fwd, t(1, 5, 16), t(16, 5))
    raises("holds 2 slots", gdr.gdr_causal_conv_step, t(3, 16), t(2, 3, 16), t(16, 4))
    raises("torch.int32", gdr.gdr_causal_conv_step, t(3, 16), t(5, 3, 16), t(16, 4), slots=torch.arange(3, device="cuda"))
    raises("16-byte", gdr.gdr_step, *(t(2, 100)[:, 1:65].unflatten(-1, (2, 32)) for _ in range(2)), t(2, 2, 32), t(2, 2, dtype=F32),
           t(2, 2, dtype=F32), t(2, 2, 32, 32, dtype=F32))
    raises("leading dimensions", gdr.gdr_rms_norm_fwd, t(4, 3, 2, 64)[:, :2], t(64))
    raises("workspace", gdr.gdr_rms_norm_bwd, t(4, 64), t(64), t(4, 64), workspace=t(8, dtype=torch.uint8))
    raises("device tensor", gdr.gdr_rms_norm_fwd, t(4, 64), torch.zeros(64, dtype=BF))


def test_steps_of_many_rows_and_far_slots():
    # a state pool of over 4 GiB: the last slots lie behind 32-bit offsets
    rows, Hv, K, n = 4, 32, 128, 2060
    pool = torch.empty(n, Hv, K, K, device="cuda", dtype=F32)
    g = gen(20)
    c = rule_case(g, rows, 16, Hv, K, BF)
    slots = torch.tensor([n - 1, 0, n - 2, 1024], dtype=torch.int32)
    first = randn(g, rows, Hv, K, K, std=0.1)
    pool[slots.long().to("cuda")] = cuda(first)
    o = gdr.gdr_step(*(cuda(c[m]) for m in ("q", "k", "v", "g", "beta")), pool, slots=cuda(slots))
    ro, rm, rs, rsm = ref.rule_step(*(c[m] for m in ("q", "k", "v", "g", "beta")), first, K ** -0.5)
    check(o, ro, rm, label="o")
    check(pool[slots.long().to("cuda")], rs, rsm, label="state")


def test_timing_hooks_name_the_kernels():
    gdr.timing.enable(True)
    gdr.timing.reset()
    h, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    gdr.gdr_rms_norm_bwd(h, w, h)
    got = gdr.timing.collect()
    gdr.timing.enable(False)
    gdr.timing.reset()
    assert set(got) == {"norm_bwd", "norm_dw"}


def test_norm_to_8_bits_at_borders_beside_what_is_not_finite():
    # 17 lies between 16 and 18 where the largest value is 448: such rows are looked at again in 64 bits, with the other
    # rows of their wave, among them one with an infinity (whose scale is NaN) and one of zeros
    x = torch.zeros(4, 128)
    x[0, 3] = float("inf")
    x[1, 5], x[1, 6], x[1, 7] = 448.0, 17.0, -19.0
    x[2] = torch.linspace(-448, 448, 128)
    w = torch.ones(128)
    q, s, _ = gdr.gdr_rms_norm_fwd(cuda(x), cuda(w), quant=True)
    assert s[0].isnan().all() and q[0].float().isnan().all()
    y, _, _ = ref.norm(x, w)
    want = torch.zeros(128, dtype=torch.float64)
    unit = y[1, 5] / 448
    check(s[1], unit[None], unit[None])
    want[5], want[6], want[7] = 448, 16, -20              # ties go to the even value
    assert torch.equal(q[1].cpu().double(), want)
    assert not q[3].float().any()
    rs, bound = ref.e4m3_parts(y[2:3])
    assert bool(((q[2].cpu().double() * float(s[2, 0]) - y[2]).abs() <= bound[0]).all())


def test_norm_to_8_bits_is_the_rounding_of_the_exact_value():
    # 2^20 values: fp32 would put about ten of them on the wrong side of a border
    g = gen(21)
    x, w, z = randn(g, 2048, 4, 128, dtype=BF), (1 + randn(g, 128, std=0.2)).to(BF), randn(g, 2048, 4, 128, dtype=BF)
    q, s, _ = gdr.gdr_rms_norm_fwd(cuda(x), cuda(w), None, cuda(z), quant=True)
    y, _, _ = ref.norm(x, w, None, z)
    v = y / (y.abs().amax(-1, keepdim=True) / 448).float().double()
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    want = torch.round(v / unit) * unit
    # a value whose 64-bit sum was added in another order may still differ where it ties to 2^-50
    assert int((q.cpu().double() != want).sum()) <= 1


def test_no_tokens():
    w, b = cuda(randn(gen(30), 16, 4)), cuda(randn(gen(31), 16))
    for x, cu, N in ((torch.empty(2, 0, 16), None, 2), (torch.empty(1, 0, 16), torch.zeros(4, dtype=torch.int32), 3)):
        h0 = cuda(randn(gen(32), N, 3, 16))
        y, ht = gdr.gdr_causal_conv_fwd(cuda(x), w, b, h0, cuda(cu), output_final_state=True)
        assert y.shape == x.shape and torch.equal(ht, h0)
        dht = cuda(randn(gen(33), N, 3, 16))
        dx, dw, db, dh0 = gdr.gdr_causal_conv_bwd(cuda(x), w, b, cuda(x), h0, dht, cuda(cu))
        assert dx.shape == x.shape and not dw.any() and not db.any() and torch.equal(dh0, dht)
        c = ref.scan_inputs(gen(34), x.shape[0], 0, 4, 2, 32, 64, F32, seqs=N)
        y, ht = run_scan(c, cu)
        assert y.shape == (x.shape[0], 0, 4, 32) and torch.equal(ht.cpu(), c["h0"])
    state = torch.zeros(2, 3, 16, device="cuda")
    assert gdr.gdr_causal_conv_step(torch.empty(0, 16, device="cuda"), state, w).shape == (0, 16)


def test_differentiable_calls_with_their_defaults():
    g = gen(35)
    x, w = cuda(randn(g, 2, 9, 16)).requires_grad_(True), cuda(randn(g, 16, 3)).requires_grad_(True)
    y, ht = gdr.causal_conv(x, w)
    assert ht is None
    dy = randn(g, 2, 9, 16)
    want = ref.conv_bwd(x, w, None, dy)
    for t, r in zip(torch.autograd.grad(y, (x, w), cuda(dy)), want):
        check(t, *r)
    n = cuda(randn(g, 16)).requires_grad_(True)
    y, h = gdr.rms_norm(x, n)
    assert h is None
    want = ref.norm_bwd(x, n, dy)
    for t, r in zip(torch.autograd.grad(y, (x, n), cuda(dy)), want):
        check(t, *r)


def test_offsets_beyond_32_bits():
    # the last rows of tensors of over 2^31 elements, against calls on those rows alone
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    T, D = 270000, 8192
    x, w = rnd(1, T, D), rnd(D, 4)
    y, _ = gdr.gdr_causal_conv_fwd(x, w)
    assert torch.equal(y[:, -50:], gdr.gdr_causal_conv_fwd(x[:, -53:].contiguous(), w)[0][:, 3:])
    dx, _, _, _ = gdr.gdr_causal_conv_bwd(x, w, None, y)
    assert torch.equal(dx[:, -50:], gdr.gdr_causal_conv_bwd(x[:, -53:].contiguous(), w, None, y[:, -53:].contiguous())[0][:, 3:])
    del dx
    rows = x.view(-1, 4096)
    n = rnd(4096)
    assert torch.equal(gdr.gdr_rms_norm_fwd(rows, n)[0][-3:], gdr.gdr_rms_norm_fwd(rows[-3:].contiguous(), n)[0])
    assert torch.equal(gdr.gdr_rms_norm_bwd(rows, n, y.view(-1, 4096))[0][-3:],
                       gdr.gdr_rms_norm_bwd(rows[-3:].contiguous(), n, y.view(-1, 4096)[-3:].contiguous())[0])
    del y
    H, P, N = 64, 128, 32
    xs, dt, A = x.view(1, T, H, P), rnd(1, T, H), -torch.rand(H, generator=g, device="cuda")
    B, C = rnd(1, T, 1, N), rnd(1, T, 1, N)
    cut = T - 70
    y, last = gdr.gdr_ssm_scan_fwd(xs, dt, A, B, C, output_final_state=True)
    _, mid = gdr.gdr_ssm_scan_fwd(xs[:, :cut], dt[:, :cut], A, B[:, :cut], C[:, :cut], output_final_state=True)
    ye, end = gdr.gdr_ssm_scan_fwd(xs[:, cut:].contiguous(), dt[:, cut:], A, B[:, cut:].contiguous(), C[:, cut:].contiguous(),
                                   initial_state=mid, output_final_state=True)
    # the chunks fall elsewhere: bf16 roundings of the operands, and fp32 sums in another order
    assert float((y[:, cut:].float() - ye.float()).norm() / ye.float().norm()) <= 2.0 ** -7
    assert float((last - end).norm() / end.norm()) <= 1e-5


def test_in_place_residual_through_the_c_entry():
    from gated_deltanet_chunked_rule_amd import layer
    g = gen(36)
    x, r, w = cuda(randn(g, 40, 4100, dtype=BF)), cuda(randn(g, 40, 4100, dtype=BF)), cuda(randn(g, 4100, dtype=BF))
    y, _, h = gdr.gdr_rms_norm_fwd(x, w, r)
    out = torch.empty_like(x)
    sh = layer._NormShape(40, 1, 4100, 0, 1e-6, 0, 0, 0, 0, 0, 0, 0)
    stream = torch.cuda.current_stream().cuda_stream
    assert layer._entry("gdr_rms_norm_fwd")(sh, x.data_ptr(), r.data_ptr(), None, w.data_ptr(), out.data_ptr(), None, r.data_ptr(), stream) == 0
    assert torch.equal(out, y) and torch.equal(r, h)


def test_two_streams_at_once():
    # calls on two streams, each with workspaces of its own, against the same calls one after another
    c = [ref.scan_inputs(gen(40 + i), 1, 3000, 16, 2, 64, 128, BF) for i in range(2)]
    k = [dict(x=cuda(randn(gen(50 + i), 2, 3000, 512, dtype=BF)), w=cuda(randn(gen(60 + i), 512, 4, dtype=BF))) for i in range(2)]
    want = [[*run_scan(c[i]), *gdr.gdr_causal_conv_bwd(k[i]["x"], k[i]["w"], None, k[i]["x"])[:2]] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for r in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [*run_scan(c[i]), *gdr.gdr_causal_conv_bwd(k[i]["x"], k[i]["w"], None, k[i]["x"])[:2]]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_captured_training_step_replays():
    """Convolution and gated norm, forward and backward, captured into one graph and replayed on new inputs and offsets.  The
    captured leaves are used by no eager graph: torch binds a leaf's gradient to the stream it was first needed on."""
    def leaves(g):
        return [cuda(t).requires_grad_(True) for t in (randn(g, 1, 600, 64, dtype=BF), randn(g, 64, 4, dtype=BF), randn(g, 64, dtype=BF),
                                                       randn(g, 1, 600, 64, dtype=BF), randn(g, 64, dtype=BF), randn(g, 1, 600, 64, dtype=BF))]

    def work(x, w, b, res, wn, z, cu, do, dh):
        y, _ = gdr.causal_conv(x, w, b, cu_seqlens=cu)
        o, h = gdr.rms_norm(y, wn, res, z)
        return [o, h, *torch.autograd.grad((o, h), (x, w, b, res, wn, z), (do, dh))]

    cu = torch.tensor([0, 100, 420, 600], dtype=torch.int32, device="cuda")
    do, dh = cuda(randn(gen(21), 1, 600, 64, dtype=BF)), cuda(randn(gen(22), 1, 600, 64, dtype=BF))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(*leaves(gen(20)), cu, do, dh)
    torch.cuda.current_stream().wait_stream(side)
    static = leaves(gen(20))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(*static, cu, do, dh)
    for r in range(4):
        fresh = leaves(gen(70 + r))
        with torch.no_grad():
            for a, b in zip(static, fresh):
                a.copy_(b)
        do.copy_(randn(gen(80 + r), 1, 600, 64))
        cu.copy_(torch.tensor([0, 1 + r, 300 + 70 * r, 600 - 13 * r]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        want = work(*fresh, cu, do, dh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), r

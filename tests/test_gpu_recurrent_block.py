"""The operators together, as a recurrent layer uses them: a training step with
its gradients, and a prompt and the tokens behind it through 8-bit projections."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
import layer_reference
from block_reference import check
from layer_reference import gen, randn
from test_gpu_layer import cuda

pytestmark = pytest.mark.gpu
F32 = torch.float32


def test_training_step_of_a_block():
    """conv -> gates' projection -> recurrence -> norms with gate and scale, fp32, against autograd of the plain forms in
    64 bits.  Every operator is off by at most 2^-18 of the magnitudes that it adds (torch's two products with 40 terms
    by 40 u); with the norms' gains around one, sums over 90 tokens and eleven operators there and back, 2^-12 of each
    tensor's largest value leaves a factor of four."""
    g = gen(1)
    T, D, cu = 90, 40, [0, 33, 34, 90]
    names = ("x", "w", "b", "proj", "A", "post", "residual", "pre", "gate", "scale")
    values = [randn(g, 1, T, D), randn(g, D, 4, std=0.5), randn(g, D), randn(g, D, 2 * D, std=D ** -0.5), -torch.rand(D, generator=g) - 0.1,
              1 + randn(g, D, std=0.1), randn(g, 1, T, D), 1 + randn(g, D, std=0.1), randn(g, 1, T, D), randn(g, D, std=0.5)]
    dy, dh = randn(g, 1, T, D), randn(g, 1, T, D)

    def plain(x, w, b, proj, A, post, residual, pre, gate, scale):
        rows = []
        for s, e in zip(cu, cu[1:]):
            ext = torch.cat([x.new_zeros(3, D), x[0, s:e]])
            z = b + sum(w[:, j] * ext[j:j + e - s] for j in range(4))
            c = z * torch.sigmoid(z)
            r, i = (c @ proj).split(D, 1)
            a = torch.exp(A * torch.sigmoid(r))
            u = torch.sqrt(1 - a * a) * torch.sigmoid(i) * c
            h = x.new_zeros(D)
            for t in range(e - s):
                h = a[t] * h + u[t]
                rows.append(h)
        v = torch.stack(rows)[None]
        norm = lambda t, k: t / (t.square().mean(-1, keepdim=True) + ref.EPS).sqrt() * k  # noqa: E731
        h = residual + scale * norm(v, post) * gate * torch.sigmoid(gate)
        return norm(h, pre), h

    leaves = [t.double().requires_grad_(True) for t in values]
    y, h = plain(*leaves)
    want = [y, h, *torch.autograd.grad([y, h], leaves, [dy.double(), dh.double()])]

    dev = {n: cuda(t).requires_grad_(True) for n, t in zip(names, values)}
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    c, _ = gdr.causal_conv(dev["x"], dev["w"], dev["b"], cu_seqlens=table)
    row = c @ dev["proj"]
    v, _ = gdr.linear_scan(c, row[..., :D], row[..., D:], dev["A"], cu_seqlens=table)
    y, h = gdr.block_norm(v, dev["post"], dev["residual"], dev["pre"], dev["gate"], dev["scale"])
    got = [y, h, *torch.autograd.grad([y, h], list(dev.values()), [cuda(dy), cuda(dh)])]
    for n, a, b in zip(("y", "h", *names), got, want):
        off = float((a.detach().cpu().double() - b.detach()).abs().max()) / float(b.detach().abs().max())
        print(f"[{n}] {off:.2e}")
        assert off <= 2.0 ** -12, n


def test_prompt_and_tokens_through_8_bit_projections():
    """Each stage against its own 64-bit form, on the inputs that the stage before left it."""
    g = gen(2)
    T, n, D, E, seqs = 70, 3, 64, 96, 2
    w_in, w_in_s = gdr.gdr_quantize_rows(cuda(randn(g, 3 * E, D, std=D ** -0.5)))
    w_out, w_out_s = gdr.gdr_quantize_rows(cuda(randn(g, D, E, std=E ** -0.5)))
    taps, bias = cuda(randn(g, E, 4, std=0.5)), cuda(randn(g, E))
    A, post, pre, scale = (cuda(t) for t in (-torch.rand(E, generator=g), 1 + randn(g, D, std=0.1), 1 + randn(g, D, std=0.1), randn(g, D, std=0.5)))

    def project(x, w, ws, name):
        q, s = gdr.gdr_quantize_rows(x)
        rq, rs = ref.quantize(x)
        assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
        y = gdr.gdr_matmul_i8(q, s, w, ws, dtype=F32)
        check(y, *ref.matmul_i8(q, s, w, ws), label=name)
        return y

    def behind(v, residual):
        o = project(v, w_out, w_out_s, "out")
        y, h = gdr.gdr_block_norm_fwd(o, post, residual, pre, scale=scale)
        ry, rye, rh, rhe = ref.block_norm(o, post, residual, pre, None, scale)
        check(y, ry, rye, "y")
        check(h, rh, rhe, "h")
        return h

    x = cuda(randn(g, seqs, T, D))
    row = project(x, w_in, w_in_s, "in")
    c, taps_state = gdr.gdr_causal_conv_fwd(row[..., :E], taps, bias, output_final_state=True)
    layer_reference.check(c, *layer_reference.conv(row[..., :E], taps, bias)[:2], label="conv")
    v, state = gdr.gdr_linear_scan_fwd(c, row[..., E:2 * E], row[..., 2 * E:], A, output_final_state=True)
    rv, rve, rs, rse, _, _ = ref.linear_scan(c, row[..., E:2 * E], row[..., 2 * E:], A)
    check(v, rv, rve, "recurrence")
    check(state, rs, rse, "state")
    behind(v, x)
    for k in range(n):
        x = cuda(randn(g, seqs, D))
        row = project(x, w_in, w_in_s, f"in {k}")
        old, window = state.clone(), torch.cat([taps_state, row[:, None, :E]], 1)
        c = gdr.gdr_causal_conv_step(row[:, :E], taps_state, taps, bias)
        wide = layer_reference.conv(window, taps, bias)
        layer_reference.check(c, wide[0][:, -1], wide[1][:, -1], label=f"conv {k}")
        v = gdr.gdr_linear_scan_step(c, row[:, E:2 * E], row[:, 2 * E:], A, state)
        rv, rve, rs, rse, _, _ = ref.linear_scan(c[:, None], row[:, None, E:2 * E], row[:, None, 2 * E:], A, old)
        check(v, rv[:, 0], rve[:, 0], f"recurrence {k}")
        check(state, rs, rse, f"state {k}")
        behind(v, x)

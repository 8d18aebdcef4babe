"""The gradients that the GPU tests compare with, against differences of their
forward forms (64 bits, on the CPU)."""
import pytest
import torch

import block_reference as ref


def differences(f, t, step=1e-6):
    """Central differences of the number f() by every value of t."""
    g = torch.zeros_like(t)
    flat, gf = t.view(-1), g.view(-1)
    for k in range(flat.numel()):
        old = float(flat[k])
        flat[k] = old + step
        up = f()
        flat[k] = old - step
        down = f()
        flat[k] = old
        gf[k] = (up - down) / (2 * step)
    return g


def rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def near(got, want):
    assert float((got - want).abs().max()) <= 2e-7 * (1 + float(want.abs().max()))


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7], [1, 2, 6]])
def test_linear_scan_gradient(cu):
    g = torch.Generator().manual_seed(3)
    x, r, i, dy = (rand(g, 1, 7, 3) for _ in range(4))
    A = -torch.rand(3, generator=g, dtype=torch.float64) - 0.05
    N = 1 if cu is None else len(cu) - 1
    h0, dht = rand(g, N, 3), rand(g, N, 3)

    def loss():
        y, _, last, _, _, _ = ref.linear_scan(x, r, i, A, h0, cu)
        return float((y * dy).sum() + (last * dht).sum())

    got = ref.linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)
    for (value, _), t in zip(got, (x, r, i, A, h0)):
        near(value, differences(loss, t))


@pytest.mark.parametrize("gate,scale", [(True, True), (False, False), (True, False)])
def test_block_norm_gradient(gate, scale):
    g = torch.Generator().manual_seed(4)
    x, residual, dy, dres = (rand(g, 3, 6) for _ in range(4))
    post, pre = 1 + 0.3 * rand(g, 6), 1 + 0.3 * rand(g, 6)
    z = rand(g, 3, 6) if gate else None
    k = rand(g, 6) if scale else None

    def loss():
        y, _, h, _ = ref.block_norm(x, post, residual, pre, z, k)
        return float((y * dy).sum() + (h * dres).sum())

    got = ref.block_norm_bwd(x, post, ref.block_norm(x, post, residual, pre, z, k)[2], pre, dy, z, k, dres)
    for (value, _), t in zip(got, (x, residual, post, pre, z, k)):
        if t is None:
            assert value is None
        else:
            near(value, differences(loss, t))

"""The linear recurrence over few channels and several tiles of tokens (one
channel has a column's lanes share it), with guard bytes around its workspaces."""
import pytest
import torch

import block_reference as ref
import gated_deltanet_chunked_rule_amd as gdr
from block_reference import check
from gated_deltanet_chunked_rule_amd import layer
from layer_reference import gen, randn
from test_gpu_layer import cuda, sliced

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

CASES = [
    # T, type, cu: tiles are 128 tokens in bf16, 64 in fp32, and a group of them 16
    (129, BF, None),
    (300, F32, [0, 100, 100, 290]),
    (700, BF, [0, 333, 600, 700]),
    (1500, F32, None),
    (4500, BF, None),
    (4500, BF, [3, 1000, 1001, 4400]),
]


@pytest.mark.parametrize("D", [1, 2, 3])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_few_channels(k, D):
    T, dtype, cu = CASES[k]
    g = gen(1200 + 10 * k + D)
    N = 1 if cu is None else len(cu) - 1
    x, r, i, dy = (randn(g, 1, T, D, dtype=dtype) for _ in range(4))
    A, h0, dht = -0.3 * torch.rand(D, generator=g), randn(g, N, D), randn(g, N, D)
    table, guard = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"), 1 << 16
    spaces = []
    for name in ("gdr_linear_scan_fwd_workspace_size", "gdr_linear_scan_bwd_workspace_size"):
        n = layer._bytes(name, layer._LinearScanShape(1, T, D, N, 0 if dtype == BF else 1, 0, 0, 0))
        spaces.append(torch.full((n + 2 * guard,), 0x5a, dtype=torch.uint8, device="cuda"))
    args = [sliced(cuda(x), 3, 1), cuda(r), sliced(cuda(i), 2, 1), cuda(A)]
    print(f"forward T={T} D={D} {dtype}", flush=True)
    y, ht = gdr.gdr_linear_scan_fwd(*args, cuda(h0), table, output_final_state=True, workspace=spaces[0][guard:-guard])
    ry, rye, rh, rhe, _, _ = ref.linear_scan(x, r, i, A, h0, cu)
    check(y, ry, rye, "y")
    check(ht, rh, rhe, "final state")
    for _ in range(5):
        again, _ = gdr.gdr_linear_scan_fwd(*args, cuda(h0), table, workspace=spaces[0][guard:-guard])
        assert torch.equal(again, y)
    print("backward", flush=True)
    grads = gdr.gdr_linear_scan_bwd(*args, cuda(dy), cuda(h0), cuda(dht), table, workspace=spaces[1][guard:-guard])
    for name, t, (v, b) in zip(("dx", "dr", "di", "dA", "dh0"), grads, ref.linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)):
        check(t, v, b, name)
    for w in spaces:
        assert bool((w[:guard] == 0x5a).all() and (w[-guard:] == 0x5a).all())

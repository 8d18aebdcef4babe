"""What the layer operators tell torch.autograd."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr
from layer_reference import gen, randn

pytestmark = pytest.mark.gpu


def steps(g, rows):
    """(state, call) of each step that works on a pool in place."""
    d = lambda *s: randn(g, *s).to("cuda")  # noqa: E731
    x, w, conv = d(rows, 16), d(16, 4), d(rows, 3, 16)
    q, k, v, gates, beta, pool = d(rows, 2, 32), d(rows, 2, 32), d(rows, 2, 32), -d(rows, 2).abs(), d(rows, 2).sigmoid(), d(rows, 2, 32, 32)
    dt, A, B, C, state = d(rows, 2), -d(2).abs(), d(rows, 1, 32), d(rows, 1, 32), d(rows, 2, 32, 32)
    return [(conv, lambda: gdr.gdr_causal_conv_step(x, conv, w)), (pool, lambda: gdr.gdr_step(q, k, v, gates, beta, pool)),
            (state, lambda: gdr.gdr_ssm_step(v, dt, A, B, C, state))]


@pytest.mark.parametrize("which", range(3))
def test_a_state_saved_for_a_backward_pass_is_known_to_have_changed(which):
    state, call = steps(gen(1), 3)[which]
    w = torch.ones_like(state, requires_grad=True)
    z = (w * state).sum()           # keeps the state for w's gradient
    call()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


@pytest.mark.parametrize("which", range(3))
def test_steps_on_inference_tensors(which):
    with torch.inference_mode():
        state, call = steps(gen(2), 3)[which]
        before = state.clone()
        call()
    call()                          # also outside, as before
    assert not torch.equal(state, before)

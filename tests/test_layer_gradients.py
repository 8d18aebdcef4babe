"""Entry points that record no gradient refuse inputs that require one (CPU only:
before anything else is looked at)."""
import pytest
import torch

import gated_deltanet_chunked_rule_amd as gdr


def raises(msg, f, *a, **kw):
    with pytest.raises(gdr.GdrError, match=msg):
        f(*a, **kw)


def test_forwards_name_the_differentiable_call():
    t = torch.zeros
    leaf = lambda *s: torch.zeros(*s, requires_grad=True)  # noqa: E731
    x, w, b, h0 = (1, 4, 8), (8, 4), (8,), (1, 3, 8)
    raises("call causal_conv", gdr.gdr_causal_conv_fwd, leaf(*x), t(*w))
    raises("call causal_conv", gdr.gdr_causal_conv_fwd, t(*x), leaf(*w))
    raises("call causal_conv", gdr.gdr_causal_conv_fwd, t(*x), t(*w), leaf(*b))
    raises("call causal_conv", gdr.gdr_causal_conv_fwd, t(*x), t(*w), None, leaf(*h0))
    raises("call rms_norm", gdr.gdr_rms_norm_fwd, leaf(4, 8), t(8))
    raises("call rms_norm", gdr.gdr_rms_norm_fwd, t(4, 8), leaf(8))
    raises("call rms_norm", gdr.gdr_rms_norm_fwd, t(4, 8), t(8), leaf(4, 8))
    raises("call rms_norm", gdr.gdr_rms_norm_fwd, t(4, 8), t(8), None, leaf(4, 8), quant=True)


def test_without_recording_they_go_on_to_the_other_checks():
    leaf = torch.zeros(1, 4, 8, requires_grad=True)
    with torch.no_grad():
        raises("device tensor", gdr.gdr_causal_conv_fwd, leaf, torch.zeros(8, 4))
        raises("device tensor", gdr.gdr_rms_norm_fwd, leaf, torch.zeros(8))
    raises("device tensor", gdr.causal_conv, leaf, torch.zeros(8, 4))     # nor inside the differentiable calls
    raises("device tensor", gdr.rms_norm, leaf, torch.zeros(8))

"""Inputs that require a gradient: the forward entries, which record none, refuse them while gradients are on."""

import pytest
import torch

from test_layer_cpu import L   # noqa: F401  (the fixture)


def test_forward_entries_refuse_what_they_would_detach(L):   # noqa: F811
    import causal_gqa_flashattention_attn_gb300 as attn
    q, k, w = torch.zeros(2, 4, 128).bfloat16(), torch.zeros(2, 2, 128).bfloat16(), torch.ones(128)
    at = torch.tensor([0, 2], dtype=torch.int32)
    calls = {"q": lambda q, k, w: attn.attn_varlen_fwd(q, k, k, at, at), "k": lambda q, k, w: attn.attn_cross_decode(q, k, k, at),
             "q_weight": lambda q, k, w: attn.attn_qk_norm_rope(q, k, w, w), "k_weight": lambda q, k, w: attn.attn_qk_norm_rope(None, k, None, w)}
    for name, call in calls.items():
        mine = [t.clone() for t in (q, k, w)]
        mine[{"q": 0, "k": 1}.get(name, 2)].requires_grad_()
        with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
            call(*mine)
        # no gradients asked for: the call goes on, to the check of devices here
        with torch.no_grad(), pytest.raises(ValueError, match="current CUDA device"):
            call(*mine)
        with pytest.raises(ValueError, match="current CUDA device"):
            call(*(t.detach() for t in mine))

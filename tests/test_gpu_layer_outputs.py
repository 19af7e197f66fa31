"""Outputs given by the caller: those that are an input or one another are refused where the results would be wrong."""

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu


def test_outputs_apart():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [40, 60], [40, 60], 4, 4, 128, seed=61)   # queries and keys of one shape
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())
    given = dict(d_o=x.do, q=x.q, k=x.k, v=x.v, o=o)
    for name in ("q", "k", "v"):
        with pytest.raises(ValueError, match=f"o must not be the same memory as {name}"):
            attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args(), o=given[name])
    for out in ("d_q", "d_k", "d_v"):
        for name, t in given.items():
            with pytest.raises(ValueError, match=f"{out} must not be the same memory as {name}"):
                attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), **{out: t})
    one = torch.empty_like(x.q)
    for a, b in (("d_q", "d_k"), ("d_q", "d_v"), ("d_k", "d_v")):
        with pytest.raises(ValueError, match=f"{a} must not be the same memory as {b}"):
            attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), **{a: one, b: one})
    token = x.q[:2].contiguous()
    with pytest.raises(ValueError, match="o must not be the same memory as q"):
        attn.attn_cross_decode(token, x.k, x.v, x.kvp, o=token)
    for more, text in ((dict(q_out=one, k_out=one), "q_out must not be the same memory as k_out"),
                       (dict(q_out=x.k), "q_out must not be the same memory as k"), (dict(k_out=x.q), "k_out must not be the same memory as q")):
        with pytest.raises(ValueError, match=text):
            attn.attn_qk_norm_rope(x.q, x.k, **more)
    for more, text in ((dict(d_q=one, d_k=one), "d_q must not be the same memory as d_k"),
                       (dict(d_q=x.k), "d_q must not be the same memory as k"), (dict(d_k=x.do), "d_k must not be the same memory as d_q_out")):
        with pytest.raises(ValueError, match=text):
            attn.attn_qk_norm_rope_bwd(x.do, x.v, x.q, x.k, **more)


def test_one_tensor_as_several_inputs():
    """Keys that are the values too, and queries that are the keys: nothing is written to them."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [40, 60], [40, 60], 4, 4, 128, seed=62)
    x.k = x.v = x.q
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    ragged.check("o", o, want_o, tol_o)
    ragged.check("lse", lse, want_l, tol_l)
    x.do = x.q
    want, tol = ragged.backward(x, o, lse)
    for label, got, w, t in zip(("dq", "dk", "dv"), attn.attn_varlen_bwd(x.q, x.q, x.q, x.q, o, lse, **x.args()), want, tol):
        ragged.check(label, got, w, t)


def test_no_tokens():
    """Empty tensors have no memory to share."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    none, at = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_varlen_fwd(none, none, none, at, at, o=none)
    assert o is none and lse.shape == (0, 4)
    grads = attn.attn_varlen_bwd(none, none, none, none, none, lse, at, at, d_q=none, d_k=none, d_v=none)
    assert all(g is none for g in grads[:3])
    assert attn.attn_qk_norm_rope(none, none, q_out=none, k_out=none)[0] is none

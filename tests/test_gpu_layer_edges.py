"""Calls of the layer's operators that other tests do not make: lengths under the causal mask, strided results of the forward
pass, one side of a norm over many tokens, token rows past 32 bits."""

import pytest
import torch

import ragged
from parity import gpu_or_skip
from test_gpu_qk_norm import _backward, _forward, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 128), (3, 3, 64), (10, 2, 128)])
def test_causal_with_lengths(hq, hkv, d):
    """The diagonal ends at the last key that counts; keys behind it, NaN here, are not used and get zeros."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    q, kv, room = [70, 200, 31, 5], [70, 333, 9, 0], [100, 400, 150, 64]
    x, y = (ragged.Batch(dev, q, kv, hq, hkv, d, room=room, causal=True, lead=3, tail=50, seed=81, padding=pad)
            for pad in (float("nan"), None))
    of_q, of_kv = x.sequence_rows()
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())
    want_o, want_l, tol_o, tol_l = ragged.forward(y)
    ragged.check("o", o, want_o, tol_o, of_q)
    ragged.check("lse", lse, want_l, tol_l, of_q)
    want, tol = ragged.backward(y, o, lse)
    for label, got, w, t, rows in zip(("dq", "dk", "dv"), attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args()), want, tol,
                                      (of_q, of_kv, of_kv)):
        ragged.check(label, got, w, t, rows)


def test_gradient_from_strided_results():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [60, 130], [300, 40], 6, 2, 64, seed=82)
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())
    plain = attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args())[:3]
    both = torch.cat([o, x.do, x.q], dim=1)
    got = attn.attn_varlen_bwd(both[:, 6:12], both[:, 12:], x.k, x.v, both[:, :6], lse, **x.args())[:3]
    assert all(torch.equal(a, b) for a, b in zip(got, plain))


@pytest.mark.parametrize("heads", [1, 2, 3, 5, 6, 8])
@pytest.mark.parametrize("side", [0, 1])
def test_one_side_of_a_norm_over_many_tokens(heads, side):
    """As cross attention calls it, where a lane takes chunks of several rows."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    for i, (d, rot, interleaved, wtype) in enumerate([(128, 0, False, torch.float32), (64, 32, True, torch.bfloat16), (128, 128, False, None)]):
        hq, hkv = (heads, 0) if side == 0 else (0, heads)
        x, dy, w, table, pos = _inputs(dev, 24000 // heads + 7, hq, hkv, d, rot, wtype, False, 83 + i)
        more = dict(eps=1e-5, cos_sin=table, positions=pos, interleaved=interleaved)
        out = attn.attn_qk_norm_rope(*x, *w, **more)
        grads = attn.attn_qk_norm_rope_bwd(*dy, *x, *w, **more)
        assert out[1 - side] is None and grads[1 - side] is None and grads[3 - side] is None
        y, tol = _forward(x[side], w[side], 1e-5, table, pos, interleaved)
        assert ((out[side].double() - y).abs() <= tol).all()
        dx, tol, dw, tol_w = _backward(dy[side], x[side], w[side], 1e-5, table, pos, interleaved)
        assert ((grads[side].double() - dx).abs() <= tol).all()
        if wtype is None:
            assert grads[2 + side] is None
        else:
            assert ((grads[2 + side].double() - dw).abs() <= tol_w).all()
        # into its own rows, and the gradient into the gradient it comes from
        mine, back = x[side].clone(), dy[side].clone()
        pair = (lambda t: (t, None) if side == 0 else (None, t))   # noqa: E731
        names = ("q", "k")[side]
        attn.attn_qk_norm_rope_bwd(*pair(back), *x, *w, **more, **{f"d_{names}": back})
        assert torch.equal(back, grads[side])
        attn.attn_qk_norm_rope(*pair(mine), *w, **more, **{f"{names}_out": mine})
        assert torch.equal(mine, out[side])


def test_token_rows_of_a_norm_past_32_bits():
    """Tokens 64 KB apart: the last ones lie more than 2^31 elements behind the first."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    t, stride = 33000, 1 << 16
    x, dy, w, table, pos = _inputs(dev, t, 3, 2, 128, 64, torch.float32, False, 91)
    far = [[torch.empty(t, stride, dtype=torch.bfloat16, device=dev)[:, :a.shape[1] * 128].view(t, a.shape[1], 128) for a in x]
           for _ in range(3)]
    for to, of in ((far[0], x), (far[1], dy)):
        for a, b in zip(to, of):
            a.copy_(b)
    more = dict(eps=1e-5, cos_sin=table, positions=pos)
    attn.attn_qk_norm_rope(*far[0], *w, **more, q_out=far[2][0], k_out=far[2][1])
    for i in range(2):
        y, tol = _forward(x[i], w[i], 1e-5, table, pos, False)
        assert ((far[2][i].double() - y).abs() <= tol).all()
    grads = attn.attn_qk_norm_rope_bwd(*far[1], *far[0], *w, **more, d_q=far[2][0], d_k=far[2][1])
    for i in range(2):
        dx, tol, dw, tol_w = _backward(dy[i], x[i], w[i], 1e-5, table, pos, False)
        assert ((far[2][i].double() - dx).abs() <= tol).all()
        assert ((grads[2 + i].double() - dw).abs() <= tol_w).all()

"""NaN and infinities in attention over contiguous keys and in its gradient: they show in the results that they concern,
whether a batch is cut into parts along its keys or not."""

import math

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

NAN = float("nan")
# few queries and long keys, which are cut into parts, and a batch that is not
SHAPES = {"parts": ([3, 20], [4000, 2500], 8, 2), "whole": ([300, 900], [400, 250], 32, 8)}


def _batches(dev, shape, d, **more):
    """The same batch twice."""
    import causal_gqa_flashattention_attn_gb300 as attn
    q, kv, hq, hkv = SHAPES[shape]
    x, y = (ragged.Batch(dev, q, kv, hq, hkv, d, seed=31, **more) for _ in range(2))
    cut = attn.attn_varlen_fwd_workspace_bytes(len(q), x.total_q, x.total_kv, hq, hkv, d) > 0
    assert cut == (shape == "parts")
    return x, y


def _forward(x):
    import causal_gqa_flashattention_attn_gb300 as attn
    return attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())[:2]


def _backward(x, o, lse):
    import causal_gqa_flashattention_attn_gb300 as attn
    return attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args())[:3]


def _same_but(got, clean, concerned):
    """NaN where `concerned`, bit for bit as from clean inputs elsewhere."""
    assert torch.isnan(got[concerned]).all()
    assert torch.equal(got[~concerned], clean[~concerned])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_nan_shows_in_o_and_lse(shape, d, what):
    dev = gpu_or_skip()
    x, y = _batches(dev, shape, d)
    group = x.hq // x.hkv
    concerned = torch.zeros(x.total_q, x.hq, dtype=torch.bool, device=dev)
    if what == "query":
        x.q[2, 5, 7] = NAN
        concerned[2, 5] = True
    else:   # the last key of the first sequence, KV head 1
        (x.k if what == "key" else x.v)[x.kv_at[1] - 1, 1] = NAN
        concerned[:x.q_at[1], group:2 * group] = True
    (o, lse), (clean_o, clean_l) = _forward(x), _forward(y)
    _same_but(o, clean_o, concerned)
    if what == "value":
        assert torch.equal(lse, clean_l)
    else:
        _same_but(lse, clean_l, concerned)


@pytest.mark.parametrize("shape", SHAPES)
def test_infinite_scores(shape):
    """A key of infinite size: queries along it have a score of +inf, for which the softmax has no value; those against it
    give it no weight."""
    dev = gpu_or_skip()
    x, y = _batches(dev, shape, 128)
    at, group = x.kv_at[1] - 1, x.hq // x.hkv
    x.k[at, 1] = 0
    x.k[at, 1, 0] = math.inf
    o, lse = _forward(x)
    mine = torch.zeros(x.total_q, x.hq, dtype=torch.bool, device=dev)
    mine[:x.q_at[1], group:2 * group] = True
    along, against = mine & (x.q[..., 0] > 0), mine & (x.q[..., 0] < 0)
    assert along.any() and against.any() and (along | against)[mine].all()
    assert torch.isnan(o[along]).all() and not torch.isfinite(lse[along]).any() and not (lse[along] == -math.inf).any()
    # those against it as if the key were not there: it is the last of its sequence
    y.kv_len[0] -= 1
    y.v[at] = 0
    want_o, want_l, tol_o, tol_l = ragged.forward(y)
    ragged.check("o", o, want_o, tol_o, against)
    ragged.check("lse", lse, want_l, tol_l, against)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("what", ["query", "key"])
def test_nan_shows_in_the_gradients_it_concerns(shape, d, what):
    """By the formula a row of NaN weights reaches dK and dV of every key that it sees."""
    dev = gpu_or_skip()
    x, y = _batches(dev, shape, d)
    group = x.hq // x.hkv
    rows = torch.zeros(x.total_q, x.hq, dtype=torch.bool, device=dev)
    keys = torch.zeros(x.total_kv, x.hkv, dtype=torch.bool, device=dev)
    keys[:x.kv_at[1], 1] = True
    if what == "query":
        x.q[2, group] = NAN   # the first query head of KV head 1
        rows[2, group] = True
    else:
        x.k[x.kv_at[1] - 1, 1] = NAN
        rows[:x.q_at[1], group:2 * group] = True
    got, clean = _backward(x, *_forward(x)), _backward(y, *_forward(y))
    for g, c, concerned in zip(got, clean, (rows, keys, keys)):
        _same_but(g, c, concerned)

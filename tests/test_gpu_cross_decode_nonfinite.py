"""NaN and infinities in single tokens' attention: they show in the rows that they concern, whole or cut into pieces."""

import math

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

NAN = float("nan")
# q_len, keys, Hq, Hkv, D: sequences cut into pieces, whole ones, 16 rows a KV head
SHAPES = [(1, [5000, 1500], 8, 2, 128), (3, [40, 60, 90], 6, 2, 64), (4, [3000], 8, 2, 64), (2, [80] * 40, 4, 4, 128)]


def _batch(dev, case):
    nq, kv, hq, hkv, d = SHAPES[case]
    x = ragged.Batch(dev, [nq] * len(kv), kv, hq, hkv, d, seed=101)
    return x, x.q.view(len(kv), nq, hq, d)


def _decode(x, q):
    import causal_gqa_flashattention_attn_gb300 as attn
    o, lse, _ = attn.attn_cross_decode(q, x.k, x.v, x.kvp)
    return o.view(x.total_q, x.hq, x.d), lse.view(x.total_q, x.hq)


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_nan(case, what):
    dev = gpu_or_skip()
    x, q = _batch(dev, case)
    clean_o, clean_l = _decode(x, q)
    group = x.hq // x.hkv
    for at in (0, x.kv_len[0] // 2, x.kv_len[0] - 1):
        x, q = _batch(dev, case)
        concerned = torch.zeros(x.total_q, x.hq, dtype=torch.bool, device=dev)
        if what == "query":
            q[0, -1, group, 3] = NAN
            concerned[x.q_len[0] - 1, group] = True
        else:
            (x.k if what == "key" else x.v)[at, 1] = NAN
            concerned[:x.q_len[0], group:2 * group] = True
        o, lse = _decode(x, q)
        assert torch.isnan(o[concerned]).all() and torch.equal(o[~concerned], clean_o[~concerned])
        if what == "value":
            assert torch.equal(lse, clean_l)
        else:
            assert torch.isnan(lse[concerned]).all() and torch.equal(lse[~concerned], clean_l[~concerned])


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_infinite_scores(case):
    """A key of infinite size: no softmax for queries along it, no weight from those against it."""
    dev = gpu_or_skip()
    x, q = _batch(dev, case)
    at, group = x.kv_len[0] - 1, x.hq // x.hkv
    x.k[at, 1] = 0
    x.k[at, 1, 0] = math.inf
    o, lse = _decode(x, q)
    mine = torch.zeros(x.total_q, x.hq, dtype=torch.bool, device=dev)
    mine[:x.q_len[0], group:2 * group] = True
    along, against = mine & (x.q[..., 0] > 0), mine & (x.q[..., 0] < 0)
    assert torch.isnan(o[along]).all() and not torch.isfinite(lse[along]).any() and not (lse[along] == -math.inf).any()
    x.kv_len[0] -= 1
    x.k[at] = 0
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    ragged.check("o", o, want_o, tol_o, against)
    ragged.check("lse", lse, want_l, tol_l, against)

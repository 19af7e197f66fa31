"""NaN and infinities in attention over contiguous keys and in its gradient: they show in the results that they concern,
whether a batch is cut into parts along its keys or not, and under the causal mask no further than the blocks and tiles
that hold them."""

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


# causal: queries, keys, Hq, Hkv, D
CAUSAL = [([256], [256], 2, 2, 128), ([300, 70], [300, 200], 3, 3, 64), ([200], [277], 8, 2, 128), ([130, 90], [130, 333], 10, 2, 64),
          ([400], [150], 4, 4, 128), ([40], [3000], 4, 2, 128), ([64], [1000], 2, 1, 64), ([500], [170], 8, 2, 64)]


def _reach(x, b, tiles):
    """For sequence b: whether a block of tiles * floor(128 / group) positions holds a query that sees a key of a tile of 128,
    as [queries, keys]; and whether a query sees a key."""
    n, m, per = x.q_len[b], x.kv_len[b], tiles * (128 // (x.hq // x.hkv))
    i, j = torch.arange(n, device=x.q.device)[:, None], torch.arange(m, device=x.q.device)
    last = torch.clamp(i // per * per + per, max=n) - 1
    return last + m - n >= j // 128 * 128, i + m - n >= j


@pytest.mark.parametrize("case", range(len(CAUSAL)))
def test_reach_of_a_nan_value_under_the_causal_mask(case):
    dev = gpu_or_skip()
    q, kv, hq, hkv, d = CAUSAL[case]
    x, y = (ragged.Batch(dev, q, kv, hq, hkv, d, causal=True, seed=41) for _ in range(2))
    clean_o, clean_l = _forward(y)
    b, group, n, m = len(q) - 1, hq // hkv, q[-1], kv[-1]
    meets, sees = _reach(x, b, 2)
    for key in sorted({0, m // 3, m // 2, m * 3 // 4, m - 70, m - 1}):
        x.v.copy_(y.v)
        x.v[x.kv_at[b] + key, hkv - 1] = NAN
        o, lse = _forward(x)
        assert torch.equal(lse, clean_l)
        rows = torch.zeros(x.total_q, hq, dtype=torch.bool, device=dev)
        rows[x.q_at[b]:x.q_at[b] + n, hq - group:] = sees[:, key, None]
        assert torch.isnan(o[rows]).all()
        nothing = ~sees.any(dim=1)   # rows that see no key at all stay empty
        rows[x.q_at[b]:x.q_at[b] + n, hq - group:] = (meets[:, key] & ~nothing)[:, None]
        assert torch.equal(o[~rows], clean_o[~rows])


@pytest.mark.parametrize("case", range(len(CAUSAL)))
@pytest.mark.parametrize("what", ["q", "do", "k", "v"])
def test_reach_of_a_nan_in_the_gradient_under_the_causal_mask(case, what):
    dev = gpu_or_skip()
    q, kv, hq, hkv, d = CAUSAL[case]
    x, y = (ragged.Batch(dev, q, kv, hq, hkv, d, causal=True, seed=43) for _ in range(2))
    o, lse = _forward(y)
    clean = _backward(y, o, lse)
    b, group, n, m = len(q) - 1, hq // hkv, q[-1], kv[-1]
    joined, sees = _reach(x, b, 1)
    of_q, of_k = slice(x.q_at[b], x.q_at[b] + n), slice(x.kv_at[b], x.kv_at[b] + m)
    size = n if what in ("q", "do") else m
    for at in sorted({0, size // 3, size // 2, size * 3 // 4, size - 1}):
        may = [torch.zeros(t.shape[:2], dtype=torch.bool, device=dev) for t in clean]   # results that it may show in
        has = [torch.zeros_like(t) for t in may]                                        # and has to
        if what in ("q", "do"):
            getattr(x, what).copy_(getattr(y, what))
            getattr(x, what)[x.q_at[b] + at, hq - 1] = NAN
            for which in (1, 2):
                may[which][of_k, hkv - 1] = joined[at]
                has[which][of_k, hkv - 1] = sees[at]
            may[0][x.q_at[b] + at, hq - 1] = has[0][x.q_at[b] + at, hq - 1] = bool(sees[at].any())
        else:
            getattr(x, what).copy_(getattr(y, what))
            getattr(x, what)[x.kv_at[b] + at, hkv - 1] = NAN
            may[0][of_q, hq - group:] = joined[:, at, None]
            has[0][of_q, hq - group:] = sees[:, at, None]
            seen = bool(sees[:, at].any())
            for which in (1, 2) if what == "k" else (1,):
                may[which][x.kv_at[b] + at, hkv - 1] = has[which][x.kv_at[b] + at, hkv - 1] = seen
        for got, c, m_, h_ in zip(_backward(x, o, lse), clean, may, has):
            assert torch.isnan(got[h_]).all()
            assert torch.equal(got[~m_], c[~m_])

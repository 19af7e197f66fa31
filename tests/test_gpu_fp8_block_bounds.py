"""Attention over the block-scaled cache against bounds that a wrong scale, page or head cannot meet.

The prefill rounds code * scale to bf16 once, in its copy of the cache: with K and V rounded the same way, scales of any size
are held to the bound of powers of two.  The decode's O over long sequences is held by its norm: the roundings of its weights
are independent of one another, so that over a whole output they add up as a sum of squares, where a bound for each element has
to take them as all of one sign."""

import numpy as np
import pytest
import torch

import block_cache as bc
from parity import gpu_or_skip
from test_gpu_fp8_block import Cache, decode

pytestmark = pytest.mark.gpu

D = 128


def as_copied(codes, scales, lists, block, b, n):
    """The rows [n, Hkv, D] that the prefill reads: code * scale in fp32, rounded to bf16."""
    t = np.arange(n)
    if n == 0:
        return np.zeros((0,) + codes.shape[2:])
    p = np.asarray(lists.rows[b])[t // lists.page]
    x = bc.E4M3.astype(np.float32)[codes[p, t % lists.page]] * scales[p, (t % lists.page) // block].astype(np.float32)[..., None]
    return bc.bf16(x).double().numpy()


def prefill_reference(q, ptr, cache, scales=None):
    """attend() of each sequence's rows; weights in bf16 (2^-8, fp32's exponents).  scales: others than the cache's."""
    parts = []
    for b, n in enumerate(cache.lens):
        kv = [as_copied(c, s, cache.lists, cache.block, b, n) for c, s in zip(cache.codes, scales or cache.scales)]
        parts.append(bc.attend(q[ptr[b]:ptr[b + 1]].double().numpy(), *kv, weight_step=2.0 ** -8, small=0.0))
    return [np.concatenate([p[i] for p in parts]) for i in range(4)]


def misses(o, lse, ref):
    """Whether check_attention refuses the outputs."""
    try:
        bc.check_attention(torch.from_numpy(o), torch.from_numpy(lse), ref)
    except AssertionError:
        return True
    return False


PREFILL = [
    ([90, 0, 333, 5], [40, 3, 333, 9], 15, 3, 48, 16, True),     # no cached token; more queries than tokens; 5 heads a group
    ([260, 31, 128, 127], [129, 31, 0, 127], 10, 2, 96, 32, False),
    ([700], [650], 12, 4, 256, 128, False),
]


@pytest.mark.parametrize("scales", ["any", "pow2"])
@pytest.mark.parametrize("lens,new,hq,hkv,page,block,csr", PREFILL)
def test_prefill_any_scales_tight(lens, new, hq, hkv, page, block, csr, scales):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(sum(lens) + 5)
    cache = Cache(lens, hkv, page, block, rng, csr, scales)
    q = bc.bf16(rng.standard_normal((sum(new), hq, D)))
    ptr = np.cumsum([0] + new)
    ref = prefill_reference(q, ptr, cache)
    # what a wrong result would be: zeros, V's scales from the next KV head, K's from the next block of the pool
    sees = ~np.isneginf(ref[1])
    assert np.mean(np.abs(ref[0][sees]) > ref[2][sees]) > 0.9
    assert misses(np.zeros_like(ref[0]), ref[1], ref)
    turned_v = prefill_reference(q, ptr, cache, [cache.scales[0], np.roll(cache.scales[1], 1, axis=2)])
    assert misses(turned_v[0], turned_v[1], ref)
    pages, indptr = cache.lists.tensors(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(q.to(dev), *cache.device(dev), torch.tensor(ptr, dtype=torch.int32, device=dev),
                                                  pages, torch.tensor(lens, dtype=torch.int32, device=dev), kv_indptr=indptr,
                                                  max_kv_rows=sum(lens), dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    bc.check_attention(o, lse, ref)


def attend_norm(q, k, v):
    """(O of q [n, Hq, D] in float64, the sum over its elements of the squares of w_t v_td / sum w, the largest error of a
    score)."""
    n, hq, _ = q.shape
    length, hkv = k.shape[:2]
    o, squares, off = np.zeros(q.shape), 0.0, 0.0
    for h in range(hq):
        kh, vh, qh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], q[:, h]
        s = qh @ kh.T * D ** -0.5
        s[np.arange(length)[None, :] > (length - n + np.arange(n))[:, None]] = -np.inf
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        o[:, h] = w @ vh
        squares += ((w ** 2) @ (vh ** 2)).sum()
        off = max(off, (2.0 ** -16 * (np.abs(qh) @ np.abs(kh).T) * D ** -0.5 + 2.0 ** -20 * np.abs(np.where(np.isinf(s), 0, s))).max())
    return o, squares, off


@pytest.mark.parametrize("lens,nq,hq,hkv,page,block,csr,scales", [
    ([6000, 2500, 900], 1, 16, 4, 64, 64, False, "pow2"),
    ([4000, 3000], 4, 12, 2, 48, 16, True, "any"),
    ([5000], 16, 8, 2, 256, 128, False, "any"),
])
def test_decode_norm_of_long_sequences(lens, nq, hq, hkv, page, block, csr, scales):
    """|O - O64| <= (2^-8 + part) |O64|, norms over a sequence's output: each element is rounded to bf16 (2^-8 of itself), and a
    weight to fp16 (2^-11 of itself, and 2^-11 more for its value scale's logarithm and the exponential, 2^-19 of fp32 each)
    after a score that is off by ``off``: errors of 2^-11 + 2^-18 + 2 off of w_t v_td / sum w, independent, 4 standard deviations
    of them at most (a rounding's is below its bound).  Weights below 2^-14 of the largest, which fp16 holds less well, are off
    by 2^-25 of it."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(sum(lens))
    cache = Cache(lens, hkv, page, block, rng, csr, scales)
    q = bc.bf16(rng.standard_normal((len(lens), nq, hq, D)))
    o, lse, status = decode(attn, q.to(dev), cache, dev)
    assert status == 0
    o = o.double().cpu().numpy()
    for b, n in enumerate(lens):
        k, v = cache.values(b)
        x = q[b].double().numpy()
        ref, squares, off = attend_norm(x, k, v)
        small = 2.0 ** -25 * np.sqrt(n * ref.size) * 448 * np.abs(v).max() / 100 / n   # weights of about 1 and more sum to n
        bound = 2.0 ** -8 * np.linalg.norm(ref) + 4 * (2.0 ** -11 + 2.0 ** -18 + 2 * off) * np.sqrt(squares) + small
        got = np.linalg.norm(o[b] - ref)
        assert got <= bound, f"sequence {b}: {got / np.linalg.norm(ref):.5f} of O's norm, bound {bound / np.linalg.norm(ref):.5f}"
        assert bound < 0.02 * np.linalg.norm(ref)
        # one block of values with eight times its scale is far outside
        p, at = cache.lists.rows[b][(n // 2) // page], (n // 2) % page // block
        keep = cache.scales[1][p, at].copy()
        cache.scales[1][p, at] *= 8
        wrong = attend_norm(x, k, cache.values(b)[1])[0]
        cache.scales[1][p, at] = keep
        assert np.linalg.norm(wrong - ref) > bound

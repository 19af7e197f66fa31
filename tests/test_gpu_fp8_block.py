"""Attention over the block-scaled e4m3 cache, decode and ragged prefill, against float64 (block_cache.attend, which derives
the bounds), and the cache's writers and readers used together as a serving loop uses them."""

import numpy as np
import pytest
import torch

import block_cache as bc
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

D = 128


class Cache:
    """A pool of random codes and scales for sequences of the given lengths.  What no sequence holds is NaN, in codes and
    scales, so that reading it shows."""

    def __init__(self, lens, hkv, page, block, rng, csr=False, scales="pow2"):
        self.lens, self.page, self.block = lens, page, block
        self.lists = bc.Lists(lens, page, rng, csr)
        n = self.lists.num_pages
        self.codes = [np.full((n, page, hkv, D), 0x7F, np.uint8) for _ in range(2)]
        self.scales = [np.full((n, page // block, hkv), np.nan, np.float32) for _ in range(2)]
        for b, length in enumerate(lens):
            t = np.arange(length)
            at = (self.lists.rows[b][t // page], t % page) if length else None
            for w in range(2):
                if length:
                    self.codes[w][at] = bc.e4m3_code(np.clip(rng.standard_normal((length, hkv, D)) * 100, -448, 448))
                    j = np.arange(-(-length // block))
                    where = (self.lists.rows[b][j * block // page], j * block % page // block)
                    self.scales[w][where] = self._scale(rng, (len(j), hkv), scales, w)

    @staticmethod
    def _scale(rng, shape, kind, w):
        if kind == "pow2":
            return 2.0 ** rng.integers(-9, -5, shape)
        if kind == "any":
            return rng.uniform(0.002, 0.02, shape)
        if kind == "far":      # values of very different sizes, some blocks of zeros
            e = rng.integers(-60, 40, shape) if w else rng.integers(-14, -6, shape)
            return np.where(rng.random(shape) < 0.2, 0.0, 2.0 ** e)
        raise ValueError(kind)

    def device(self, dev):
        c = [torch.from_numpy(x.copy()).to(dev) for x in self.codes]
        s = [torch.from_numpy(x.copy()).to(dev) for x in self.scales]
        return c + s

    def values(self, b, skip=()):
        return [bc.cached(c, s, self.lists, self.block, b, self.lens[b], skip) for c, s in zip(self.codes, self.scales)]


def reference(q, cache, scale=None, **kw):
    """attend() of q [B, n, Hq, D] over each sequence."""
    parts = [bc.attend(q[b], *cache.values(b), scale=scale, **kw) for b in range(len(cache.lens))]
    return tuple(np.stack([p[i] for p in parts]) for i in range(4))


def decode(attn, q, cache, dev, **kw):
    pages, indptr = cache.lists.tensors(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = torch.tensor(cache.lens, dtype=torch.int32, device=dev)
    o, lse, ws = attn.attn_decode_paged_fp8_block(q, *cache.device(dev), pages, lens, kv_indptr=indptr, dev_status=status, **kw)
    torch.cuda.synchronize()
    return o, lse, status.item()


#  (lens, q_len, Hq, Hkv, page, block, csr, scales)
DECODE = [
    ([1], 1, 4, 1, 16, 16, False, "pow2"),
    ([0], 1, 8, 8, 64, 64, False, "pow2"),
    ([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100], 1, 8, 8, 64, 64, False, "pow2"),
    ([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100], 1, 12, 4, 16, 16, True, "any"),
    ([700, 3, 0, 2049], 1, 32, 8, 256, 64, False, "pow2"),
    ([700, 3, 0, 2049], 2, 15, 3, 48, 16, True, "any"),
    ([7000], 1, 8, 1, 128, 128, False, "any"),               # one long sequence over all workers, merged
    ([5000, 40], 4, 16, 2, 32, 32, True, "pow2"),            # 32 rows a KV head: two groups of 16
    ([3, 4, 5, 200], 5, 14, 2, 32, 16, False, "pow2"),       # fewer tokens than queries: rows that see nothing
    ([300, 90], 16, 10, 10, 96, 32, False, "any"),           # G = 1, 16 queries
    ([260, 1], 3, 7, 7, 16, 16, True, "pow2"),               # 7 KV heads: shares across CTAs
    ([90, 33], 16, 64, 2, 32, 16, False, "pow2"),            # 512 rows a KV head: 32 groups
    ([50, 1000, 0], 1, 40, 5, 1024, 512, False, "far"),
    ([500, 333], 2, 4, 4, 64, 16, True, "far"),
    ([4] * 300, 1, 2, 2, 16, 16, False, "pow2"),
    ([0, 1, 96, 0, 33, 64, 0], 1, 8, 8, 64, 64, False, "pow2"),      # none long enough to be cut
    ([0, 5, 96] * 200, 1, 12, 12, 16, 16, True, "any"),              # and several sequences a share
    ([65, 129, 40], 1, 300, 300, 16, 16, False, "any"),      # 300 KV heads: a column each, fewer shares
    ([40, 70], 16, 80, 80, 16, 16, False, "any"),
]


@pytest.mark.parametrize("lens,nq,hq,hkv,page,block,csr,scales", DECODE)
def test_decode(lens, nq, hq, hkv, page, block, csr, scales):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(sum(lens) + nq)
    cache = Cache(lens, hkv, page, block, rng, csr, scales)
    q = bc.bf16(rng.standard_normal((len(lens), nq, hq, D)))
    o, lse, status = decode(attn, (q[:, 0] if nq == 1 else q).to(dev), cache, dev)
    assert status == 0
    if nq == 1:
        o, lse = o[:, None], lse[:, None]
    bc.check_attention(o, lse, reference(q.double().numpy(), cache))


#  more than 16 rows a KV head
MANY_ROWS = [
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300], 4, 16, 2, 16, 16, True, "any"),   # 32 rows, ends around a tile's
    ([500, 64], 3, 12, 2, 32, 32, False, "pow2"),             # 18 rows
    ([3000, 7], 9, 7, 1, 48, 16, False, "any"),               # 63 rows, cut over many CTAs
    ([2000, 0, 1, 70], 16, 8, 1, 64, 64, True, "pow2"),       # 128 rows
    ([900, 33], 16, 27, 3, 32, 32, False, "any"),             # 144 rows: a column of 128 and one of 16
    ([70, 200], 16, 320, 160, 16, 16, False, "any"),          # more columns than CTAs
    ([8, 3] * 150, 2, 20, 1, 16, 16, True, "pow2"),           # 40 rows, many short sequences
    ([500, 333], 4, 32, 4, 64, 16, True, "far"),
    ([700, 90], 8, 16, 2, 128, 128, False, "far"),
    # long enough for columns of 16 rows (more than 12 tiles of 32 tokens a share on 152 SMs)
    ([2000, 0, 1, 15, 33, 1900, 70], 16, 64, 2, 64, 16, True, "any"),   # 512 rows
    ([3000, 4500, 31], 16, 32, 4, 48, 16, False, "far"),
    ([1200] * 24 + [0, 3], 4, 60, 10, 64, 64, True, "pow2"),            # 24 rows: a column of 16 and one of 8
]


@pytest.mark.parametrize("lens,nq,hq,hkv,page,block,csr,scales", MANY_ROWS)
def test_decode_many_rows(lens, nq, hq, hkv, page, block, csr, scales):
    test_decode(lens, nq, hq, hkv, page, block, csr, scales)


@pytest.mark.parametrize("lens,nq,hq", [([0, 1, 15, 16, 17, 31, 32, 33, 64, 100], 4, 16), ([3, 4, 5, 200], 5, 14),
                                        ([700, 3, 0, 2049], 3, 12)])
def test_decode_many_rows_of_a_large_pool(lens, nq, hq):
    """Short sequences in a pool of 64k tokens: the columns go by what the lists could name."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(17)
    cache = Cache(lens, 2, 32, 16, rng, True, "any")
    for w in range(2):
        cache.codes[w] = np.concatenate([cache.codes[w], np.full((2000, 32, 2, D), 0x7F, np.uint8)])
        cache.scales[w] = np.concatenate([cache.scales[w], np.full((2000, 2, 2), np.nan, np.float32)])
    q = bc.bf16(rng.standard_normal((len(lens), nq, hq, D)))
    o, lse, status = decode(attn, q.to(dev), cache, dev)
    assert status == 0
    bc.check_attention(o, lse, reference(q.double().numpy(), cache))


@pytest.mark.parametrize("nq,hq,hkv,more", [(4, 16, 2, 0), (16, 4, 2, 0), (16, 8, 2, 0), (16, 16, 2, 0), (16, 16, 2, 9)])
def test_decode_many_rows_far_queries_and_nans(nq, hq, hkv, more):
    """Queries of any size, peaked scores, and NaNs that some rows see and others do not, 32 to 128 rows a KV head."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(nq + hq)
    lens = [1500, 100, 77] + [1500] * more
    cache = Cache(lens, hkv, 64, 16, rng, scales="any")
    for size in (2.0 ** -120, 30.0, 2.0 ** 100):
        q = bc.bf16(rng.standard_normal((len(lens), nq, hq, D)) * size)
        q[0, 0, 0] = 0.0
        scale = D ** -0.5 / size if size != 30.0 else None
        o, lse, status = decode(attn, q.to(dev), cache, dev, scale=scale)
        assert status == 0
        bc.check_attention(o, lse, reference(q.double().numpy(), cache, scale=None if scale is None else float(np.float32(scale))))
    clean = o, lse
    put = [(0, 0, 0, 1499, 5), (1, 1, 1, 99 - (nq - 2), 9), (2, 1, 0, 76, 127), (2, 1, 0, 60, 0), (1, 0, 1, 98, 64)]
    for b, w, h, t, d in put:      # sequence, K or V, KV head, token, element
        cache.codes[w][cache.lists.rows[b][t // 64], t % 64, h, d] = 0x7F
    want = torch.zeros(len(lens), nq, hq, D, dtype=torch.bool)
    g = hq // hkv
    for b, w, h, t, d in put:
        first = max(0, t - (lens[b] - nq))        # the first query that sees the token
        want[b, first:, h * g:(h + 1) * g, slice(None) if w == 0 else d] = True
    o, lse, status = decode(attn, q.to(dev), cache, dev, scale=scale)
    assert status == 0
    assert torch.equal(torch.isnan(o).cpu(), want)
    assert torch.equal(o.cpu()[~want], clean[0].cpu()[~want])


def test_decode_csr_offsets_that_fall():
    """A sequence whose CSR offsets fall has an empty list: flagged, nothing of it read, the others as they are."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(23)
    cache = Cache([40, 70, 33], 2, 16, 16, rng, csr=True)     # lists of 3, 5 and 3 pages
    pages, _ = cache.lists.tensors(dev)
    indptr = torch.tensor([3, 8, 8, 0], dtype=torch.int32, device=dev)   # the second list, none, falling
    lens = torch.tensor([70, 5, 5], dtype=torch.int32, device=dev)
    q = bc.bf16(rng.standard_normal((3, 1, 4, D)))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_decode_paged_fp8_block(q.to(dev), *cache.device(dev), pages, lens, kv_indptr=indptr, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == attn.ATTN_DEV_SEQ_TOO_LONG
    ref = bc.attend(q[0].double().numpy(), *cache.values(1))
    bc.check_attention(o[:1], lse[:1], tuple(x[None] for x in ref))
    assert not o[1:].any() and torch.isneginf(lse[1:]).all()


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_decode_queries_of_any_size(size):
    """q beyond fp16's range on either side, with a scale that brings the scores back."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(2)
    cache = Cache([300, 70], 2, 32, 32, rng)
    q = bc.bf16(rng.standard_normal((2, 2, 8, D)) * size)
    q[0, 0, 0] = 0.0
    scale = D ** -0.5 / size
    o, lse, status = decode(attn, q.to(dev), cache, dev, scale=scale)
    assert status == 0
    bc.check_attention(o, lse, reference(q.double().numpy(), cache, scale=float(np.float32(scale))))


def test_decode_peaked_scores():
    """Scores hundreds apart: the running maxima move, most weights vanish."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(4)
    cache = Cache([1500, 64], 2, 64, 16, rng, scales="any")
    q = bc.bf16(rng.standard_normal((2, 1, 4, D)) * 30)
    o, lse, status = decode(attn, q.to(dev), cache, dev)
    assert status == 0
    bc.check_attention(o, lse, reference(q.double().numpy(), cache))


@pytest.mark.parametrize("scale", [-0.05, 0.0])
@pytest.mark.parametrize("nq,hq", [(1, 4), (3, 8)])
def test_decode_any_scale(scale, nq, hq):
    """Scores of the other sign, and all alike: the masks still hold."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(5)
    cache = Cache([400, 2, 33], 2, 32, 16, rng)
    q = bc.bf16(rng.standard_normal((3, nq, hq, D)))
    o, lse, status = decode(attn, q.to(dev), cache, dev, scale=scale)
    assert status == 0
    bc.check_attention(o, lse, reference(q.double().numpy(), cache, scale=float(np.float32(scale))))


def test_decode_nan_shows():
    """A NaN in a key or value that a row sees comes out as NaN; rows that do not see it are clean."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(6)
    cache = Cache([100, 100], 2, 16, 16, rng)
    q = bc.bf16(rng.standard_normal((2, 2, 4, D)))
    t = 99   # the last token: seen by the second query only
    cache.codes[0][cache.lists.rows[0][t // 16], t % 16, 1, 3] = 0x7F     # K of sequence 0, KV head 1
    cache.codes[1][cache.lists.rows[1][t // 16], t % 16, 0, 9] = 0xFF     # V of sequence 1, KV head 0
    o, lse, status = decode(attn, q.to(dev), cache, dev)
    assert status == 0
    bad = torch.isnan(o).cpu()
    want = torch.zeros_like(bad)
    want[0, 1, 2:] = True
    want[1, 1, :2, 9] = True
    assert torch.equal(bad, want)
    assert torch.equal(torch.isnan(lse).cpu(), want[..., 0])


def test_decode_same_bits_again_and_workspace_reuse():
    """Twice the same call gives the same bits, also with a workspace that calls of other shapes used between."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(7)
    big, small = Cache([9000, 50, 3000], 4, 64, 64, rng), Cache([40, 2000], 4, 16, 16, rng, csr=True)
    qb, qs = bc.bf16(rng.standard_normal((3, 16, D))).to(dev), bc.bf16(rng.standard_normal((2, 4, 16, D))).to(dev)
    need = max(attn.attn_decode_fp8_block_workspace_bytes(3, 1, 16, 4), attn.attn_decode_fp8_block_workspace_bytes(2, 4, 16, 4))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)   # scratch: whatever it holds (NaN here)
    first = decode(attn, qb, big, dev, workspace=ws)
    decode(attn, qs, small, dev, workspace=ws)
    again = decode(attn, qb, big, dev, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    alone = decode(attn, qs, small, dev)
    shared = decode(attn, qs, small, dev, workspace=ws)
    assert torch.equal(alone[0], shared[0]) and torch.equal(alone[1], shared[1])


def test_decode_flags_bad_pages_and_long_sequences():
    """A page outside the pool is left out as if its tokens were not there for the softmax; a length past the list is cut."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(9)
    cache = Cache([200, 90], 2, 16, 16, rng, csr=True)
    q = bc.bf16(rng.standard_normal((2, 1, 4, D)))
    good = cache.lists.rows[0][3]
    parts = [bc.attend(q[0].double().numpy(), *cache.values(0, skip=(3,))), bc.attend(q[1].double().numpy(), *cache.values(1))]
    ref = tuple(np.stack([p[i] for p in parts]) for i in range(4))
    for bad in (-1, cache.lists.num_pages, 2 ** 31 - 1):
        cache.lists.rows[0][3] = bad
        o, lse, status = decode(attn, q.to(dev), cache, dev)
        assert status == attn.ATTN_DEV_PAGE_OUT_OF_RANGE
        bc.check_attention(o, lse, ref)
    cache.lists.rows[0][3] = good
    pages, indptr = cache.lists.tensors(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    cache.scales[0][cache.lists.rows[0][-1]] = 0.01       # the list's whole capacity has to be readable: 208 tokens
    cache.scales[1][cache.lists.rows[0][-1]] = 0.01
    cache.codes[0][cache.lists.rows[0][-1]] = 0x30
    cache.codes[1][cache.lists.rows[0][-1]] = 0x30
    lens = torch.tensor([5000, -3], dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_decode_paged_fp8_block(q.to(dev), *cache.device(dev), pages, lens, kv_indptr=indptr, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == attn.ATTN_DEV_SEQ_TOO_LONG
    cache.lens = [208, 0]
    bc.check_attention(o, lse, reference(q.double().numpy(), cache))


def test_decode_far_offsets():
    """A pool whose byte offsets pass 32 bits: tokens at its end."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(10)
    page, hkv, n = 256, 8, 17000                      # 17000 * 256 * 8 * 128 bytes = 4.5 GB each
    if torch.cuda.mem_get_info(dev)[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    small = Cache([600], hkv, page, 64, rng)
    at = [n - 1, 3, n - 2]
    kv = [torch.zeros(n, page, hkv, D, dtype=torch.uint8, device=dev) for _ in range(2)]
    sc = [torch.zeros(n, page // 64, hkv, device=dev) for _ in range(2)]
    for w in range(2):
        for e, p in enumerate(at):
            kv[w][p] = torch.from_numpy(small.codes[w][small.lists.rows[0][e]]).to(dev)
            sc[w][p] = torch.from_numpy(small.scales[w][small.lists.rows[0][e]]).to(dev)
    table = torch.tensor([at], dtype=torch.int32, device=dev)
    lens = torch.tensor([599], dtype=torch.int32, device=dev)
    x = bc.bf16(rng.standard_normal((1, 8, D)))
    # one more token goes to the far page, then both are read
    attn.attn_kv_append_fp8_block(None, x.to(dev), x.to(dev), *kv, *sc, table, torch.tensor([600], dtype=torch.int32, device=dev))
    for w in range(2):
        bc.append_blocks(small.codes[w], small.scales[w], small.lists, 64, 0, 599, x.double().numpy())
    q = bc.bf16(rng.standard_normal((1, 1, 16, D)))
    lens += 1
    o, lse, _ = attn.attn_decode_paged_fp8_block(q.to(dev), *kv, *sc, table, lens)
    torch.cuda.synchronize()
    bc.check_attention(o, lse, reference(q.double().numpy(), small))


#  (lens, new, Hq, Hkv, page, block, csr, scales)
PREFILL = [
    ([1], [1], 4, 1, 16, 16, False, "pow2"),
    ([300, 129, 64], [300, 1, 17], 8, 2, 64, 64, False, "pow2"),
    ([90, 0, 333, 5], [40, 3, 333, 9], 15, 3, 48, 16, True, "any"),     # no cached token; more queries than tokens
    ([700], [650], 32, 4, 256, 128, False, "pow2"),
    ([260, 31, 128, 127], [129, 31, 0, 127], 7, 7, 16, 16, True, "pow2"),
]


@pytest.mark.parametrize("lens,new,hq,hkv,page,block,csr,scales", PREFILL)
def test_prefill(lens, new, hq, hkv, page, block, csr, scales):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(sum(lens) + 1)
    cache = Cache(lens, hkv, page, block, rng, csr, scales)
    q = bc.bf16(rng.standard_normal((sum(new), hq, D)))
    pages, indptr = cache.lists.tensors(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ptr = np.cumsum([0] + new)
    args = (q.to(dev), *cache.device(dev), torch.tensor(ptr, dtype=torch.int32, device=dev), pages,
            torch.tensor(lens, dtype=torch.int32, device=dev))
    # weights in bf16: half a step 2^-8, exponent range of fp32; K and V of scales that are no power of two: 2^-8 more of each
    odd = 0.0 if scales == "pow2" else 2.0 ** -8
    parts = [bc.attend(q[ptr[b]:ptr[b + 1]].double().numpy(), *cache.values(b), weight_step=2.0 ** -8 + odd, small=0.0)
             for b in range(len(lens))]
    ref = [np.concatenate([p[i] for p in parts]) for i in range(4)]
    if odd:   # a score moves by 2^-8 of the sum of its products' sizes: |s| of independent products, 16 of them in a row's bound
        reach = np.concatenate([np.full(p[1].shape, _score_reach(q[ptr[b]:ptr[b + 1]], cache.values(b)[0])) for b, p in enumerate(parts)])
        moved = 2.0 ** -8 * reach
        ref[3] = ref[3] + moved
        ref[2] = ref[2] + 2 * moved[..., None] * np.concatenate([_value_reach(cache.values(b)[1], p[0].shape) for b, p in enumerate(parts)])
    for rows in (max(1, sum(lens)), None):
        o, lse, _ = attn.attn_prefill_paged_fp8_block(*args, kv_indptr=indptr, max_kv_rows=rows, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        bc.check_attention(o, lse, ref)


def _score_reach(q, k):
    """The largest sum of |q_d k_d| / sqrt(D) of any query and key: what rounding each k_d by a part moves a score by at most."""
    if q.shape[0] == 0 or k.shape[0] == 0:
        return 0.0
    g = q.shape[1] // k.shape[1]
    q = np.abs(q.double().numpy())
    return max((q[:, h] @ np.abs(k[:, h // g]).T).max() for h in range(q.shape[1])) * D ** -0.5


def _value_reach(v, shape):
    return np.full(shape, np.abs(v).max(initial=0.0))


def test_prefill_flags():
    """A bad page reads as zeros, a length past the list and rows past max_kv_rows are cut and flagged."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(12)
    cache = Cache([100, 40], 2, 16, 16, rng, csr=True)
    q = bc.bf16(rng.standard_normal((30, 4, D)))
    ptr = torch.tensor([0, 20, 30], dtype=torch.int32, device=dev)
    keep = cache.lists.rows[0][2]
    k, v = cache.values(0)
    k[32:48] = 0
    v[32:48] = 0
    parts = [bc.attend(q[:20].double().numpy(), k, v, weight_step=2.0 ** -8, small=0.0),
             bc.attend(q[20:].double().numpy(), *cache.values(1), weight_step=2.0 ** -8, small=0.0)]
    ref = [np.concatenate([p[i] for p in parts]) for i in range(4)]
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def call(lens, rows):
        pages, indptr = cache.lists.tensors(dev)
        status.zero_()
        o, lse, _ = attn.attn_prefill_paged_fp8_block(q.to(dev), *cache.device(dev), ptr, pages,
                                                      torch.tensor(lens, dtype=torch.int32, device=dev), kv_indptr=indptr,
                                                      max_kv_rows=rows, dev_status=status)
        torch.cuda.synchronize()
        return o, lse, status.item()

    cache.lists.rows[0][2] = -5
    o, lse, bits = call([100, 40], 140)
    assert bits == attn.ATTN_DEV_PAGE_OUT_OF_RANGE
    bc.check_attention(o, lse, ref)
    cache.lists.rows[0][2] = keep
    assert call([100, 40], 140)[2] == 0
    assert call([100, 40], 139)[2] == attn.ATTN_DEV_SEQ_TOO_LONG
    assert call([100, 49], 149)[2] == attn.ATTN_DEV_SEQ_TOO_LONG
    assert call([100, 48], 148)[2] == 0


def test_shared_pages():
    """Sequences that read the same pages: together more tokens than the pool has, with the default workspace."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(21)
    cache = Cache([250], 2, 64, 32, rng)
    lens, new = [250, 180, 250, 9, 200], [250, 20, 3, 9, 1]
    table = torch.from_numpy(np.tile(cache.lists.rows[0], (5, 1))).to(dev)
    seq = torch.tensor(lens, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    k, v = cache.values(0)
    q = bc.bf16(rng.standard_normal((sum(new), 4, D)))
    at = np.cumsum([0] + new)
    ptr = torch.tensor(at, dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(q.to(dev), *cache.device(dev), ptr, table, seq, dev_status=status)
    torch.cuda.synchronize()
    parts = [bc.attend(q[at[b]:at[b + 1]].double().numpy(), k[:lens[b]], v[:lens[b]], weight_step=2.0 ** -8, small=0.0)
             for b in range(5)]
    assert status.item() == 0
    bc.check_attention(o, lse, [np.concatenate([p[i] for p in parts]) for i in range(4)])
    q = bc.bf16(rng.standard_normal((5, 1, 4, D)))
    o, lse, _ = attn.attn_decode_paged_fp8_block(q.to(dev), *cache.device(dev), table, seq, dev_status=status)
    torch.cuda.synchronize()
    parts = [bc.attend(q[b].double().numpy(), k[:lens[b]], v[:lens[b]]) for b in range(5)]
    assert status.item() == 0
    bc.check_attention(o, lse, tuple(np.stack([p[i] for p in parts]) for i in range(4)))


@pytest.mark.parametrize("n,new,hq", [(2048, 1, 4), (900, 18, 64)])
def test_prefill_many_sequences(n, new, hq):
    """The most sequences a batch may have, and more work items than are sorted (5 query blocks of 4 positions each)."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(n)
    lens = rng.integers(new, new + 20, n).tolist()
    cache = Cache(lens, 1, 16, 16, rng)
    q = bc.bf16(rng.standard_normal((n * new, hq, D)))
    pages, _ = cache.lists.tensors(dev)
    ptr = torch.arange(n + 1, dtype=torch.int32, device=dev) * new
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(q.to(dev), *cache.device(dev), ptr, pages,
                                                  torch.tensor(lens, dtype=torch.int32, device=dev), max_kv_rows=sum(lens),
                                                  dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())
    for b in [0, 1, n // 2, n - 2, n - 1] + rng.integers(0, n, 8).tolist():
        rows = slice(b * new, (b + 1) * new)
        bc.check_attention(o[rows], lse[rows], bc.attend(q[rows].double().numpy(), *cache.values(b), weight_step=2.0 ** -8, small=0.0))


def _wide_table(hkv, dev):
    """An empty batch of 64 whose block table is 131071 pages of 256 tokens wide: 2^31 - 16384 tokens."""
    codes = torch.zeros(2, 256, hkv, D, dtype=torch.uint8, device=dev)
    scales = torch.ones(2, 4, hkv, device=dev)
    return dict(q=torch.zeros(64, hkv, D, dtype=torch.bfloat16, device=dev), k_cache=codes, v_cache=codes, k_scale=scales,
                v_scale=scales, qo_indptr=torch.arange(65, dtype=torch.int32, device=dev),
                block_table=torch.zeros(64, 131071, dtype=torch.int32, device=dev),
                seq_lens=torch.ones(64, dtype=torch.int32, device=dev))


def test_prefill_default_rows_past_the_limit():
    """Page lists that hold more than a workspace may: refused by name where max_kv_rows is left out, taken where it is given."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    call = _wide_table(8, dev)
    with pytest.raises(ValueError, match="max_kv_rows"):
        attn.attn_prefill_paged_fp8_block(**call)
    with pytest.raises(attn.AttnError, match="unsupported"):      # as the entry says of what the caller asks for
        attn.attn_prefill_paged_fp8_block(**call, max_kv_rows=64 * 131071 * 256)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(**call, max_kv_rows=64)
    torch.cuda.synchronize()
    assert not o.any() and not lse.any()      # a token of zeros each


def test_out_of_memory_is_torchs():
    """A workspace that the GPU has no room for raises torch's own error, as an allocation in Python does."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    call = _wide_table(1, dev)     # 1.1 TB
    with pytest.raises(torch.OutOfMemoryError):
        attn.attn_prefill_paged_fp8_block(**call)
    o, _, _ = attn.attn_prefill_paged_fp8_block(**call, max_kv_rows=64)
    torch.cuda.synchronize()
    assert not o.any()


def test_calls_on_two_streams_at_once():
    """Decodes and prefills of two batches on two streams, each with its own workspace, give what they give alone."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(14)
    jobs = []
    for lens in ([3000, 700, 40], [100, 5000]):
        cache = Cache(lens, 2, 64, 32, rng)
        n = len(lens)
        pages, _ = cache.lists.tensors(dev)
        d = dict(q=bc.bf16(rng.standard_normal((n, 3, 8, D))).to(dev), cache=cache.device(dev), pages=pages,
                 lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                 ptr=torch.arange(n + 1, dtype=torch.int32, device=dev) * 3, stream=torch.cuda.Stream(dev))
        d["ws"] = torch.empty(attn.attn_decode_fp8_block_workspace_bytes(n, 3, 8, 2), dtype=torch.uint8, device=dev)
        d["pws"] = torch.empty(attn.attn_prefill_fp8_block_workspace_bytes(n, sum(lens), 2), dtype=torch.uint8, device=dev)
        d["rows"] = sum(lens)
        jobs.append(d)

    def run(d, stream):
        o, lse, _ = attn.attn_decode_paged_fp8_block(d["q"], *d["cache"], d["pages"], d["lens"], workspace=d["ws"], stream=stream)
        po, plse, _ = attn.attn_prefill_paged_fp8_block(d["q"].view(-1, 8, D), *d["cache"], d["ptr"], d["pages"], d["lens"],
                                                        max_kv_rows=d["rows"], workspace=d["pws"], stream=stream)
        return o, lse, po, plse

    alone = []
    for d in jobs:
        alone.append(run(d, None))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [run(d, d["stream"]) for d in jobs]
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, g))


def test_prefill_nan_stays_in_its_sequence():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(13)
    lens, new = [40, 200, 33], [40, 60, 33]
    cache = Cache(lens, 2, 16, 16, rng)
    for w in range(2):   # every code of the middle sequence's last block
        cache.codes[w][cache.lists.rows[1][12]] = 0x7F
    q = bc.bf16(rng.standard_normal((sum(new), 4, D)))
    pages, _ = cache.lists.tensors(dev)
    ptr = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(q.to(dev), *cache.device(dev), ptr, pages,
                                                  torch.tensor(lens, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    for b, rows in ((0, slice(0, 40)), (2, slice(100, 133))):
        bc.check_attention(o[rows], lse[rows], bc.attend(q[rows].double().numpy(), *cache.values(b), weight_step=2.0 ** -8, small=0.0))
    assert bool(torch.isnan(o[92:100]).all())     # the queries at tokens 192 .. 199 see it


def test_serving_loop_and_graphs():
    """Prompts appended and prefilled, then tokens appended and decoded, step by step: eagerly on a side stream, and the decode
    steps again from a captured graph whose buffers are refilled between replays; a second captured graph with a workspace of
    its own runs between them."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(21)
    hq, hkv, page, block, steps = 8, 2, 32, 16, 4
    prompts = [45, 130, 7]
    n = len(prompts)
    capacity = [p + steps for p in prompts]
    lists = bc.Lists(capacity, page, rng)
    pages, _ = lists.tensors(dev)
    table = bc.rope_table(max(capacity), D)
    cs = torch.from_numpy(table).to(dev)
    shape, blocks = (lists.num_pages, page, hkv, D), (lists.num_pages, page // block, hkv)
    ref_c = [np.zeros(shape, np.uint8) for _ in range(2)]
    ref_s = [np.zeros(blocks, np.float32) for _ in range(2)]
    dc = [torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2)]
    ds = [torch.zeros(blocks, device=dev) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def ref_append(k, v, t0s, counts):
        at = 0
        for b, (t0, m) in enumerate(zip(t0s, counts)):
            tt = np.arange(t0, t0 + m)
            turned = bc.rotate(k[at:at + m].double().numpy(), table, tt, False)
            bc.append_blocks(ref_c[0], ref_s[0], lists, block, b, t0, turned)
            bc.append_blocks(ref_c[1], ref_s[1], lists, block, b, t0, v[at:at + m].double().numpy())
            at += m

    def ref_attend(q, counts, lens, **kw):
        at, parts = 0, []
        for b, m in enumerate(counts):
            kv = [bc.cached(c, s, lists, block, b, lens[b]) for c, s in zip(ref_c, ref_s)]
            parts.append(bc.attend(q[at:at + m].double().cpu().numpy(), *kv, **kw))
            at += m
        return [np.concatenate([p[i] for p in parts]) for i in range(4)]

    total = sum(prompts)
    q, k, v = (bc.bf16(rng.standard_normal((total, h, D))) for h in (hq, hkv, hkv))
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    ptr = torch.tensor(np.cumsum([0] + prompts), dtype=torch.int32, device=dev)
    dq, dk, dv = q.to(dev), k.to(dev), v.to(dev)
    torch.cuda.synchronize()
    turned = attn.attn_kv_append_fp8_block(dq, dk, dv, *dc, *ds, pages, lens, cos_sin=cs, qo_indptr=ptr, dev_status=status,
                                           stream=side)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(turned, *dc, *ds, ptr, pages, lens, dev_status=status, stream=side)
    side.synchronize()
    ref_append(k, v, [0] * n, prompts)
    assert np.array_equal(dc[0].cpu().numpy(), ref_c[0]) and np.array_equal(dc[1].cpu().numpy(), ref_c[1])
    bc.check_attention(o, lse, ref_attend(turned, prompts, prompts, weight_step=2.0 ** -8, small=0.0), "prompts")

    # a decode step on fixed buffers, captured after one eager step (the first)
    bq, bk, bv = (torch.empty(n, h, D, dtype=torch.bfloat16, device=dev) for h in (hq, hkv, hkv))
    bl = lens.clone()
    rot, ro, rl = torch.empty_like(bq), torch.empty_like(bq), torch.empty(n, hq, device=dev)
    ws = [torch.zeros(attn.attn_decode_fp8_block_workspace_bytes(n, 1, hq, hkv), dtype=torch.uint8, device=dev) for _ in range(2)]
    other = torch.empty_like(bq)

    def step(workspace, out, stream=None):
        attn.attn_kv_append_fp8_block(bq, bk, bv, *dc, *ds, pages, bl, cos_sin=cs, q_out=rot, dev_status=status, stream=stream)
        attn.attn_decode_paged_fp8_block(rot, *dc, *ds, pages, bl, workspace=workspace, o=out, lse=rl, dev_status=status,
                                         stream=stream)

    graphs = []
    for i in range(steps):
        x = [bc.bf16(rng.standard_normal((n, h, D))) for h in (hq, hkv, hkv)]
        for buf, val in zip((bq, bk, bv), x):
            buf.copy_(val.to(dev))
        bl += 1
        torch.cuda.synchronize()
        if i == 0:
            step(ws[0], ro)
        else:
            if not graphs:
                for w, out in ((ws[0], ro), (ws[1], other)):
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g):
                        step(w, out)
                    graphs.append(g)
            ro.zero_()
            graphs[1].replay()     # the same step: appending the same tokens again changes nothing
            graphs[0].replay()
        torch.cuda.synchronize()
        assert status.item() == 0
        now = [p + i + 1 for p in prompts]
        ref_append(x[1], x[2], [t - 1 for t in now], [1] * n)
        for w in range(2):
            assert np.array_equal(dc[w].cpu().numpy(), ref_c[w]) and np.array_equal(ds[w].cpu().numpy(), ref_s[w]), i
        bc.check_attention(ro, rl, ref_attend(rot, [1] * n, now), f"step {i}")
        if graphs:
            assert torch.equal(other, ro)


def test_bf16_append_feeds_the_bf16_decode():
    """attn_kv_append followed by attn_decode_paged_splitk and attn_prefill_paged_varlen_ws over the same pages."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(31)
    hq, hkv, page = 8, 2, 64
    lens = [130, 64, 5]
    lists = bc.Lists(lens, page, rng)
    pages, _ = lists.tensors(dev)
    table = bc.rope_table(200, D)
    cs = torch.from_numpy(table).to(dev)
    kc, vc = (torch.zeros(lists.num_pages, page, hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    total = sum(lens)
    q, k, v = (bc.bf16(rng.standard_normal((total, h, D))) for h in (hq, hkv, hkv))
    ptr = np.cumsum([0] + lens)
    dl, dp = torch.tensor(lens, dtype=torch.int32, device=dev), torch.tensor(ptr, dtype=torch.int32, device=dev)
    turned = attn.attn_kv_append(q.to(dev), k.to(dev), v.to(dev), kc, vc, pages, dl, cos_sin=cs, qo_indptr=dp)
    kvp = np.cumsum([0] + [len(r) for r in lists.rows])
    flat = torch.from_numpy(np.concatenate(lists.rows)).to(dev)
    last = torch.tensor([n - (len(r) - 1) * page for n, r in zip(lens, lists.rows)], dtype=torch.int32, device=dev)
    o, lse = attn.attn_prefill_paged_varlen_ws(turned, kc, vc, dp, torch.tensor(kvp, dtype=torch.int32, device=dev), flat, last)
    last_rows = torch.tensor(ptr[1:] - 1, device=dev)
    od, ld, _ = attn.attn_decode_paged_splitk(turned[last_rows].contiguous(), kc, vc, pages, dl, 64, max(lens))
    torch.cuda.synchronize()
    t = np.concatenate([np.arange(n) for n in lens])
    kt = bc.bf16(bc.rotate(k.double().numpy(), table, t, False)).double().numpy()
    for b in range(3):
        rows = slice(ptr[b], ptr[b + 1])
        # keys that lie on a border may be rounded the other way: a bf16 step of one product in a score
        ref = list(bc.attend(turned[rows].double().cpu().numpy(), kt[rows], v[rows].double().numpy(), weight_step=2.0 ** -8, small=0.0))
        bc.check_attention(o[rows], lse[rows], ref, f"prefill {b}")
        one = [r[-1:] for r in ref]
        bc.check_attention(od[b:b + 1], ld[b:b + 1], one, f"decode {b}")

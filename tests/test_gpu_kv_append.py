"""attn_kv_append and attn_kv_append_fp8_block against the plain cache of block_cache.py.

bf16 outputs may be off by half a step, 2^-8 of the value, and by three fp32 roundings of the two products, 2^-22 of their
sizes.  Codes and scales of the 8-bit cache have to be equal: ties go to the even code, and a rotated value next to a border
falls where 64-bit arithmetic puts it."""

import numpy as np
import pytest
import torch

import block_cache as bc
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

D = 128


class Batch:
    """New tokens of a batch: ``old`` cached and ``new`` more for each sequence."""

    def __init__(self, old, new, hq, hkv, rng, scale=1.0):
        self.old, self.new, self.hq, self.hkv = old, new, hq, hkv
        self.total = sum(new)
        width = (hq + 2 * hkv) * D + 8
        flat = bc.bf16(rng.standard_normal((self.total, width)) * scale)
        self.q, self.k, self.v = (flat[:, a:b].view(self.total, -1, D) for a, b in (
            (0, hq * D), (hq * D, (hq + hkv) * D), ((hq + hkv) * D, (hq + 2 * hkv) * D)))

    def rows(self, b):
        start = sum(self.new[:b])
        return slice(start, start + self.new[b])

    def indices(self):
        return np.concatenate([np.arange(o, o + n) for o, n in zip(self.old, self.new)] + [np.zeros(0, np.int64)]).astype(np.int64)

    def lens(self, dev):
        return torch.tensor([o + n for o, n in zip(self.old, self.new)], dtype=torch.int32, device=dev)

    def indptr(self, dev):
        return torch.tensor(np.cumsum([0] + self.new), dtype=torch.int32, device=dev)


def strided(batch, dev):
    """q, k, v as parts of one tensor: token rows (Hq + 2 Hkv) D + 8 elements apart."""
    hq, hkv, t = batch.hq, batch.hkv, batch.total
    width = (hq + 2 * hkv) * D + 8
    flat = torch.zeros(t, width, dtype=torch.bfloat16, device=dev)
    parts = []
    at = 0
    for x in (batch.q, batch.k, batch.v):
        n = x.shape[1] * D
        flat[:, at:at + n] = x.reshape(t, n).to(dev)
        parts.append(flat[:, at:at + n].view(t, -1, D))
        at += n
    return parts


def check_bf16(got, want, slack):
    got = got.detach().float().cpu().double().numpy()
    over = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -22 * slack + 1e-38)
    assert got.shape == want.shape and np.all(np.isfinite(got))
    assert over.max(initial=-1) <= 0, f"over the bound by {over.max():.3e}"


#  (old lengths, new tokens, Hq, Hkv, page, rot, interleaved, csr, one token each)
BF16 = [
    ([0], [1], 4, 1, 16, 128, False, False, True),
    ([5, 0, 255, 256, 700], [1] * 5, 32, 8, 256, 128, False, False, True),
    ([5, 0, 255, 256, 700], [1] * 5, 15, 5, 64, 64, True, True, True),
    ([0, 3, 100], [37, 0, 65], 6, 2, 16, 128, True, False, False),
    ([17, 0, 0, 1], [1, 300, 0, 33], 7, 7, 1, 32, False, True, False),
    ([9, 40], [130, 5], 16, 2, 7, 96, False, True, False),
    ([9, 40], [130, 5], 3, 3, 100, 0, False, False, False),
    ([0] * 70, [2] * 70, 2, 1, 3, 16, True, False, False),     # more sequences than a warp has lanes
]


@pytest.mark.parametrize("old,new,hq,hkv,page,rot,inter,csr,one", BF16)
def test_append_bf16(old, new, hq, hkv, page, rot, inter, csr, one):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(len(old) * 100 + page)
    batch = Batch(old, new, hq, hkv, rng)
    lists = bc.Lists([o + n for o, n in zip(old, new)], page, rng, csr)
    table = bc.rope_table(1200, rot) if rot else None
    pages, indptr = lists.tensors(dev)
    shape = (lists.num_pages, page, hkv, D)
    k_cache, v_cache = (torch.full(shape, 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    q, k, v = strided(batch, dev)
    out = attn.attn_kv_append(q, k, v, k_cache, v_cache, pages, batch.lens(dev),
                              cos_sin=None if table is None else torch.from_numpy(table).to(dev),
                              qo_indptr=None if one else batch.indptr(dev), kv_indptr=indptr, interleaved=inter,
                              dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    t = batch.indices()
    x = batch.q.double().numpy()
    check_bf16(out, bc.rotate(x, table, t, inter), bc.rotate_slack(x, table, t, inter))
    want = {c: np.full(shape, 7.0) for c in "kv"}
    slack = np.zeros(shape)
    turned, sizes = (f(batch.k.double().numpy(), table, t, inter) for f in (bc.rotate, bc.rotate_slack))
    for b in range(len(old)):
        tt = t[batch.rows(b)]
        at = (lists.rows[b][tt // page], tt % page)
        want["k"][at], slack[at] = turned[batch.rows(b)], sizes[batch.rows(b)]
        want["v"][at] = batch.v[batch.rows(b)].double().numpy()
    check_bf16(k_cache, want["k"], slack)
    assert np.array_equal(v_cache.float().cpu().numpy(), want["v"].astype(np.float32))   # copied, the rest untouched


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,ragged", [(3, 4, 1, False), (400, 8, 2, False), (700, 2, 1, False), (40, 8, 2, True),
                                             (9, 72, 3, False)])
def test_append_dense_rows(n, hq, hkv, ragged, inter):
    """Rows that start on 32 bytes, from a few tokens to more than get a CTA each, more heads than a CTA has rows; both caches."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(n + hq)
    page = block = 16
    old = rng.integers(0, 14, n).tolist()
    new = rng.integers(0, 5, n).tolist() if ragged else [1] * n
    new = [min(a, 16 - o) for a, o in zip(new, old)]
    batch = Batch(old, new, hq, hkv, rng)
    lists = bc.Lists([16] * n, page, rng)
    pages, _ = lists.tensors(dev)
    table = bc.rope_table(16, 96)
    cs = torch.from_numpy(table).to(dev)
    q, k, v = (x.contiguous().to(dev) for x in (batch.q, batch.k, batch.v))
    t = batch.indices()
    turned_q, turned_k = (bc.rotate(x.double().numpy(), table, t, inter) for x in (batch.q, batch.k))
    slack = [bc.rotate_slack(x.double().numpy(), table, t, inter) for x in (batch.q, batch.k)]
    shape = (lists.num_pages, page, hkv, D)
    ptr = batch.indptr(dev) if ragged else None
    caches = [torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    out = attn.attn_kv_append(q, k, v, *caches, pages, batch.lens(dev), cos_sin=cs, qo_indptr=ptr, interleaved=inter)
    codes = [np.full(shape, 0x38, np.uint8) for _ in range(2)]
    scales = [np.full((lists.num_pages, 1, hkv), 2.0 ** -8, np.float32) for _ in range(2)]
    dc = [torch.from_numpy(x.copy()).to(dev) for x in codes]
    ds = [torch.from_numpy(x.copy()).to(dev) for x in scales]
    out8 = attn.attn_kv_append_fp8_block(q, k, v, *dc, *ds, pages, batch.lens(dev), cos_sin=cs, qo_indptr=ptr,
                                         interleaved=inter)
    torch.cuda.synchronize()
    check_bf16(out, turned_q, slack[0])
    assert torch.equal(out, out8)
    rows = torch.tensor([lists.rows[b][0] for b in range(n) for _ in range(new[b])], device=dev).long()
    at = torch.from_numpy(t).to(dev)
    check_bf16(caches[0][rows, at], turned_k, slack[1])
    assert torch.equal(caches[1][rows, at], v)
    for b in range(n):
        if new[b]:
            bc.append_blocks(codes[0], scales[0], lists, block, b, old[b], turned_k[batch.rows(b)])
            bc.append_blocks(codes[1], scales[1], lists, block, b, old[b], batch.v[batch.rows(b)].double().numpy())
    for w in range(2):
        assert np.array_equal(ds[w].cpu().numpy(), scales[w])
        assert np.array_equal(dc[w].cpu().numpy(), codes[w])


@pytest.mark.parametrize("size", [2.0 ** -133, 2.0 ** -126, 2.0 ** -118, 2.0 ** -101, 2.0 ** 126])
def test_append_fp8_block_rotated_far_from_one(size):
    """Keys at the ends of bf16's range, where fp32's products are subnormal or overflow: codes as from exact rotations."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(17)
    table = bc.rope_table(40, 64)
    cs = torch.from_numpy(table).to(dev)
    for new, ragged in (([1, 1, 1], False), ([20, 3, 33], True)):
        batch = Batch([0, 0, 0], new, 1, 2, rng, scale=size)
        batch.k[:, :, 5] = 0.0
        lists = bc.Lists([64] * 3, 64, rng)
        pages, _ = lists.tensors(dev)
        shape, blocks = (lists.num_pages, 64, 2, D), (lists.num_pages, 2, 2)
        codes, scales = [np.zeros(shape, np.uint8) for _ in range(2)], [np.zeros(blocks, np.float32) for _ in range(2)]
        dc = [torch.from_numpy(x.copy()).to(dev) for x in codes]
        ds = [torch.from_numpy(x.copy()).to(dev) for x in scales]
        k, v = batch.k.contiguous(), batch.v.contiguous()
        attn.attn_kv_append_fp8_block(None, k.to(dev), v.to(dev), *dc, *ds, pages, batch.lens(dev), cos_sin=cs,
                                      qo_indptr=batch.indptr(dev) if ragged else None)
        torch.cuda.synchronize()
        turned = bc.rotate(k.double().numpy(), table, batch.indices(), False)
        for b in range(3):
            bc.append_blocks(codes[0], scales[0], lists, 32, b, 0, turned[batch.rows(b)])
            bc.append_blocks(codes[1], scales[1], lists, 32, b, 0, v[batch.rows(b)].double().numpy())
        for w in range(2):
            assert np.array_equal(ds[w].cpu().numpy(), scales[w])
            got = dc[w].cpu().numpy()
            assert np.array_equal(bc.E4M3[got], bc.E4M3[codes[w]]), (new, "kv"[w])


@pytest.mark.parametrize("block", [32, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_append_fp8_block_rotated_past_fp32(inter, block):
    """Keys whose rotation passes fp32's range, or comes near its end: the code of the exact value, whether a token comes alone
    or within a prompt (blocks that stay in shared memory and ones that do not).  Infinities and NaN beside them."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(41 + block)
    table = bc.rope_table(300, D)
    table[7] = np.float32(np.sqrt(0.5))                       # cosines and sines alike
    cs = torch.from_numpy(table).to(dev)
    for new, ragged in (([1, 1, 1], False), ([20, 3, 33], True), ([250, 130, 9], True)):
        t = np.concatenate([np.arange(n) for n in new])
        total = len(t)
        k = bc.bf16(rng.uniform(0.7, 0.99, (total, 2, D)) * rng.choice([-1.0, 1.0], (total, 2, D)) * 2.0 ** 128)
        k[0, 0], k[-1, 1] = 3.0e38, -3.0e38                   # 4.2e38 in every element of one half at position 7
        k[1, 0, 3:9] = float("inf")
        k[2, 1, 60:70] = float("nan")
        pos = t.copy()
        pos[[0, -1]] = 7
        lists = bc.Lists([256] * 3, 256, rng)
        pages, _ = lists.tensors(dev)
        shape, blocks = (lists.num_pages, 256, 2, D), (lists.num_pages, 256 // block, 2)
        codes, scales = np.zeros(shape, np.uint8), np.zeros(blocks, np.float32)
        dc = [torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2)]
        ds = [torch.zeros(blocks, device=dev) for _ in range(2)]
        ptr = np.cumsum([0] + new)
        attn.attn_kv_append_fp8_block(None, k.to(dev), k.to(dev), *dc, *ds, pages, torch.tensor(new, dtype=torch.int32, device=dev),
                                      cos_sin=cs, positions=torch.tensor(pos, dtype=torch.int32, device=dev), interleaved=inter,
                                      qo_indptr=torch.tensor(ptr, dtype=torch.int32, device=dev) if ragged else None)
        torch.cuda.synchronize()
        turned = bc.rotate(k.double().numpy(), table, pos, inter)
        assert np.nanmax(np.abs(np.where(np.isinf(turned), 0, turned))) > 4.2e38
        for b in range(3):
            bc.append_blocks(codes, scales, lists, block, b, 0, turned[ptr[b]:ptr[b + 1]])
        assert np.array_equal(ds[0].cpu().numpy(), scales)
        got, want = bc.E4M3[dc[0].cpu().numpy()], bc.E4M3[codes]
        assert np.array_equal(np.isnan(got), np.isnan(want)), new
        off = np.argwhere(np.nan_to_num(got) != np.nan_to_num(want))
        assert not len(off), (new, len(off), off[:3], got[tuple(off[0])], want[tuple(off[0])])


def test_append_positions_in_place_padding_and_keys_only():
    """Positions of the caller's, q rotated in place, padded entries of length 0 and rows of no sequence left alone, no q."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(3)
    table = bc.rope_table(5000, 128)
    batch = Batch([10, 0, 3], [1, 1, 1], 8, 2, rng)
    lists = bc.Lists([11, 1, 4], 16, rng)
    pages, _ = lists.tensors(dev)
    lens = torch.tensor([11, 0, 4], dtype=torch.int32, device=dev)      # the second entry is padding
    pos = np.array([4321, -9, 17])
    shape = (lists.num_pages, 16, 2, D)
    k_cache, v_cache = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    q = batch.q.contiguous().to(dev)
    k, v = batch.k.contiguous().to(dev), batch.v.contiguous().to(dev)
    cs = torch.from_numpy(table).to(dev)
    got = attn.attn_kv_append(q, k, v, k_cache, v_cache, pages, lens, cos_sin=cs,
                              positions=torch.tensor(pos, dtype=torch.int32, device=dev), q_out=q, dev_status=status)
    torch.cuda.synchronize()
    assert got is q and status.item() == 0
    want = bc.rotate(batch.q.double().numpy(), table, np.where(pos < 0, 0, pos), False)
    want[1] = batch.q[1].double().numpy()
    check_bf16(q, want, bc.rotate_slack(batch.q.double().numpy(), table, np.where(pos < 0, 0, pos), False))
    kk = bc.rotate(batch.k.double().numpy(), table, np.where(pos < 0, 0, pos), False)
    ref = np.zeros(shape)
    for b, t in ((0, 10), (2, 3)):
        ref[lists.rows[b][t // 16], t % 16] = kk[b]
    check_bf16(k_cache, ref, np.full(shape, 30.0))
    assert np.count_nonzero(k_cache[lists.rows[1][0]].float().cpu().numpy()) == 0
    # rows behind the last sequence: their q_out stays, and keys alone
    ptr = torch.tensor([0, 1, 1, 2], dtype=torch.int32, device=dev)
    out = torch.full((3, 8, D), 5.0, dtype=torch.bfloat16, device=dev)
    attn.attn_kv_append(q, k, v, k_cache, v_cache, pages, torch.tensor([11, 0, 4], dtype=torch.int32, device=dev), cos_sin=cs,
                        qo_indptr=ptr, q_out=out, dev_status=status)
    k2, v2 = torch.zeros_like(k_cache), torch.zeros_like(v_cache)
    none = attn.attn_kv_append(None, k, v, k2, v2, pages, torch.tensor([11, 0, 4], dtype=torch.int32, device=dev),
                               cos_sin=cs, qo_indptr=ptr, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and none is None
    assert torch.all(out[2] == 5.0) and not torch.any(torch.all(out[:2] == 5.0, dim=-1))
    assert torch.equal(k2[lists.rows[2][0], 3], k_cache[lists.rows[2][0], 3])


#  (steps of new tokens per sequence, Hq, Hkv, page, block, rot, interleaved, csr)
FP8 = [
    ([[1], [1], [1]], 4, 1, 16, 16, 128, False, False),
    ([[64, 1, 63], [1, 64, 2], [5, 130, 1]], 8, 8, 128, 64, 128, False, False),
    ([[17, 0, 250], [1, 1, 1], [1, 1, 1], [31, 7, 16]], 6, 3, 48, 16, 64, True, True),
    ([[300], [1], [300]], 5, 5, 256, 256, 96, False, True),
    ([[33, 9], [40, 200]], 4, 2, 96, 32, 0, False, False),
    ([[3] * 70, [1] * 70], 1, 1, 16, 16, 16, True, True),
]


@pytest.mark.parametrize("steps,hq,hkv,page,block,rot,inter,csr", FP8)
def test_append_fp8_block_steps(steps, hq, hkv, page, block, rot, inter, csr):
    """Several appends in a row: blocks are begun, joined, grown in scale and finished; codes and scales are equal."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(len(steps) * 1000 + page + block)
    n = len(steps[0])
    capacity = [sum(s[b] for s in steps) for b in range(n)]
    lists = bc.Lists(capacity, page, rng, csr)
    pages, indptr = lists.tensors(dev)
    table = bc.rope_table(max(capacity), rot) if rot else None
    cs = None if table is None else torch.from_numpy(table).to(dev)
    shape, blocks = (lists.num_pages, page, hkv, D), (lists.num_pages, page // block, hkv)
    start = rng.integers(0, 127, shape, dtype=np.uint8)
    codes = [start.copy(), start[::-1].copy()]
    scales = [np.full(blocks, 2.0 ** 40, dtype=np.float32) for _ in range(2)]   # pages had another owner
    dc = [torch.from_numpy(c.copy()).to(dev) for c in codes]
    ds = [torch.from_numpy(s.copy()).to(dev) for s in scales]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    old = [0] * n
    for i, new in enumerate(steps):
        batch = Batch(old, list(new), hq, hkv, rng, scale=[1.0, 30.0, 0.01, 5.0][i % 4])
        q, k, v = strided(batch, dev)
        one = all(x == 1 for x in new) and i % 2 == 1
        out = attn.attn_kv_append_fp8_block(q, k, v, *dc, *ds, pages, batch.lens(dev), cos_sin=cs, interleaved=inter,
                                            qo_indptr=None if one else batch.indptr(dev), kv_indptr=indptr,
                                            dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        t = batch.indices()
        x = batch.q.double().numpy()
        check_bf16(out, bc.rotate(x, table, t, inter), bc.rotate_slack(x, table, t, inter))
        turned, values = bc.rotate(batch.k.double().numpy(), table, t, inter), batch.v.double().numpy()
        for b in range(n):
            if new[b]:
                bc.append_blocks(codes[0], scales[0], lists, block, b, old[b], turned[batch.rows(b)])
                bc.append_blocks(codes[1], scales[1], lists, block, b, old[b], values[batch.rows(b)])
        for which in range(2):
            assert np.array_equal(ds[which].cpu().numpy(), scales[which]), f"scales of {'kv'[which]}, step {i}"
            got = dc[which].cpu().numpy()
            assert np.array_equal(got, codes[which]), f"codes of {'kv'[which]}, step {i}: {np.argwhere(got != codes[which])[:4]}"
        old = [o + m for o, m in zip(old, new)]


@pytest.mark.parametrize("inter,page,block", [(False, 32, 16), (True, 64, 32), (False, 64, 64), (True, 256, 256)])
def test_append_fp8_block_many_heads_positions_and_type(inter, page, block):
    """240 + 2 x 120 heads (so many blocks that each takes as few warps as hold it), positions of their own, tensors of the
    float8 type."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(31)
    hq, hkv, new = 240, 120, [40, 25] if block < 256 else [200, 7]
    lists = bc.Lists(new, page, rng)
    pages, _ = lists.tensors(dev)
    batch = Batch([0, 0], new, hq, hkv, rng)
    table = bc.rope_table(900, 128)
    pos = rng.permutation(sum(new)) * 13 % 900
    shape, blocks = (lists.num_pages, page, hkv, D), (lists.num_pages, page // block, hkv)
    dc = [torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
    ds = [torch.zeros(blocks, device=dev) for _ in range(2)]
    q, k, v = strided(batch, dev)
    out = attn.attn_kv_append_fp8_block(q, k, v, *dc, *ds, pages, batch.lens(dev), cos_sin=torch.from_numpy(table).to(dev),
                                        interleaved=inter, qo_indptr=batch.indptr(dev),
                                        positions=torch.tensor(pos, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    x = batch.q.double().numpy()
    check_bf16(out, bc.rotate(x, table, pos, inter), bc.rotate_slack(x, table, pos, inter))
    for got, scale, want in zip(dc, ds, (bc.rotate(batch.k.double().numpy(), table, pos, inter), batch.v.double().numpy())):
        codes, scales = np.zeros(shape, np.uint8), np.zeros(blocks, np.float32)
        for b in range(2):
            bc.append_blocks(codes, scales, lists, block, b, 0, want[batch.rows(b)])
        assert np.array_equal(scale.cpu().numpy(), scales)
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), codes)


def test_append_fp8_block_borders():
    """Ties between codes, sizes at 448 * 2^e and one step beside it, zeros, subnormal and huge values, NaN and infinities."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    block = 16
    rows = []
    mids = (bc._POS[1:] + bc._POS[:-1]) / 2
    rows.append(np.concatenate([mids, [448.0, 0.0]]))                                  # ties at scale 1
    rows.append(np.concatenate([-mids, [448.0, -0.0]]) * 2.0 ** -30)
    rows.append(np.full(D, 1.75 * 2.0 ** 9))                                           # 448 * 2: scale 2
    rows.append(np.full(D, (1.75 + 2.0 ** -7) * 2.0 ** 9))                             # a step above: scale 4
    rows.append(np.zeros(D))
    rows.append(np.full(D, 2.0 ** -133))                                               # below the smallest scale's codes
    rows.append(np.full(D, 2.0 ** 127))
    rows.append(np.where(np.arange(D) % 3 == 0, np.nan, 3.0))
    rows.append(np.where(np.arange(D) == 5, np.inf, np.where(np.arange(D) == 6, -np.inf, 0.5)))
    rows.append(np.full(D, np.inf))
    rows.append(np.full(D, -0.0))
    x = bc.bf16(np.stack(rows)[:, None, :])                                            # one block each: a sequence each
    n = x.shape[0]
    rng = np.random.default_rng(0)
    lists = bc.Lists([1] * n, block, rng)
    pages, _ = lists.tensors(dev)
    shape, blocks = (lists.num_pages, block, 1, D), (lists.num_pages, 1, 1)
    codes = [np.zeros(shape, np.uint8) for _ in range(2)]
    scales = [np.ones(blocks, np.float32) for _ in range(2)]
    dc = [torch.from_numpy(c.copy()).to(dev) for c in codes]
    ds = [torch.from_numpy(s.copy()).to(dev) for s in scales]
    table = np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], axis=1).astype(np.float32)   # a turn by 0
    xd = x.to(dev)
    attn.attn_kv_append_fp8_block(None, xd, xd, *dc, *ds, pages, torch.ones(n, dtype=torch.int32, device=dev),
                                  cos_sin=torch.from_numpy(table).to(dev))
    torch.cuda.synchronize()
    vals = x.double().numpy()
    with np.errstate(invalid="ignore"):
        turned = bc.rotate(vals, table, np.zeros(n, np.int64), False)
    for b in range(n):
        bc.append_blocks(codes[0], scales[0], lists, block, b, 0, turned[b:b + 1])
        bc.append_blocks(codes[1], scales[1], lists, block, b, 0, vals[b:b + 1])
    for which in range(2):
        assert np.array_equal(ds[which].cpu().numpy(), scales[which])
        got = dc[which].cpu().numpy()
        live = bc.E4M3[got]
        want = bc.E4M3[codes[which]]
        assert np.array_equal(np.isnan(live), np.isnan(want))
        assert np.array_equal(np.nan_to_num(live), np.nan_to_num(want)), "kv"[which]


def test_append_fp8_block_old_scales():
    """A block with a stored scale that is no power of two counts as the next one above; 0 stands for codes of zero."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(8)
    block, n = 32, 5
    lists = bc.Lists([20] * n, block, rng)
    pages, _ = lists.tensors(dev)
    shape, blocks = (lists.num_pages, block, 2, D), (lists.num_pages, 1, 2)
    codes = [rng.integers(0, 126, shape, dtype=np.uint8) for _ in range(2)]
    scales = [np.ones(blocks, np.float32) for _ in range(2)]
    for b, s in enumerate([0.3, 0.0, 2.0 ** -20, 3.0e5, 2.0 ** -140]):
        for w in range(2):
            scales[w][lists.rows[b][0], 0] = s
    dc = [torch.from_numpy(c.copy()).to(dev) for c in codes]
    ds = [torch.from_numpy(s.copy()).to(dev) for s in scales]
    x = bc.bf16(rng.standard_normal((n, 2, D)))
    attn.attn_kv_append_fp8_block(None, x.to(dev), x.to(dev), *dc, *ds, pages,
                                  torch.full((n,), 20, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    for w in range(2):
        for b in range(n):
            bc.append_blocks(codes[w], scales[w], lists, block, b, 19, x[b:b + 1].double().numpy())
        assert np.array_equal(ds[w].cpu().numpy(), scales[w])
        assert np.array_equal(dc[w].cpu().numpy(), codes[w])


def test_append_flags_bad_pages_and_positions():
    """A missing page, an index past the list and a position off the table set their bits and leave their tokens out."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(5)
    table = torch.from_numpy(bc.rope_table(50, 128)).to(dev)
    for fp8 in (False, True):
        for what, bit in (("page", attn.ATTN_DEV_PAGE_OUT_OF_RANGE), ("list", attn.ATTN_DEV_SEQ_TOO_LONG),
                          ("position", attn.ATTN_DEV_POSITION_OUT_OF_RANGE)):
            batch = Batch([20, 3], [1, 1], 4, 2, rng)
            lists = bc.Lists([32, 16], 16, rng)
            if what == "page":
                lists.rows[0] = np.array([lists.rows[0][0], lists.num_pages], dtype=np.int32)
            if what == "list":
                lists.rows[0] = lists.rows[0][:1]
            lists.csr = True
            pages, indptr = lists.tensors(dev)
            pos = torch.tensor([50 if what == "position" else 20, 3], dtype=torch.int32, device=dev)
            shape = (lists.num_pages, 16, 2, D)
            status = torch.zeros(1, dtype=torch.int32, device=dev)
            q, k, v = (x.contiguous().to(dev) for x in (batch.q, batch.k, batch.v))
            q_out = torch.full_like(q, 9.0)
            kw = dict(cos_sin=table, kv_indptr=indptr, positions=pos, q_out=q_out, dev_status=status)
            if fp8:
                caches = [torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2)]
                scales = [torch.zeros(lists.num_pages, 1, 2, device=dev) for _ in range(2)]
                attn.attn_kv_append_fp8_block(q, k, v, *caches, *scales, pages, batch.lens(dev), **kw)
            else:
                caches = [torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)]
                attn.attn_kv_append(q, k, v, *caches, pages, batch.lens(dev), **kw)
            torch.cuda.synchronize()
            assert status.item() == bit, (fp8, what, status.item())
            for c in caches:   # only the second sequence's token is there
                there = torch.nonzero(c.view(torch.uint8).reshape(lists.num_pages * 16, -1).any(dim=1)).flatten().tolist()
                assert there == [int(lists.rows[1][0]) * 16 + 3], (fp8, what)
            assert bool(torch.all(q_out[0] == 9.0)) == (what == "position")
            assert not bool(torch.all(q_out[1] == 9.0))


@pytest.mark.parametrize("fp8", [False, True])
def test_append_no_tokens(fp8):
    """A step whose sequences all bring nothing: an empty result, the cache as it was."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    caches = [torch.full((2, 16, 2, D), 7, dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev) for _ in range(2)]
    scales = [torch.full((2, 1, 2), 0.5, device=dev) for _ in range(2)] if fp8 else []
    x = [torch.zeros(0, h, D, dtype=torch.bfloat16, device=dev) for h in (4, 2, 2)]
    call = attn.attn_kv_append_fp8_block if fp8 else attn.attn_kv_append
    out = call(*x, *caches, *scales, torch.zeros(2, 1, dtype=torch.int32, device=dev),
               torch.tensor([3, 0], dtype=torch.int32, device=dev), qo_indptr=torch.zeros(3, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert out.shape == x[0].shape and out.dtype == torch.bfloat16
    assert all((c == 7).all() for c in caches) and all((s == 0.5).all() for s in scales)


def test_binding_refuses_wrong_tensors():
    """Types, shapes, strides and devices that a call does not take raise ValueError, statuses AttnError; nothing is written."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    i32 = dict(dtype=torch.int32, device=dev)
    q, k = (torch.ones(2, h, D, dtype=torch.bfloat16, device=dev) for h in (4, 2))
    c8 = torch.zeros(3, 32, 2, D, dtype=torch.uint8, device=dev)
    cb = torch.zeros(3, 32, 2, D, dtype=torch.bfloat16, device=dev)
    sc = torch.ones(3, 2, 2, device=dev)
    table, lens, ptr = torch.zeros(2, 1, **i32), torch.ones(2, **i32), torch.tensor([0, 1, 2], **i32)

    def append(match, error=ValueError, fp8=True, **kw):
        a = dict(q=q, k=k, v=k, k_cache=c8 if fp8 else cb, v_cache=c8 if fp8 else cb, block_table=table, seq_lens=lens)
        if fp8:
            a.update(k_scale=sc, v_scale=sc)
        a.update(kw)
        with pytest.raises(error, match=match):
            (attn.attn_kv_append_fp8_block if fp8 else attn.attn_kv_append)(**a)

    for fp8 in (False, True):
        append("seq_lens", fp8=fp8, seq_lens=lens.long())
        append("block_table", fp8=fp8, seq_lens=torch.ones(3, **i32))
        append("block_table", fp8=fp8, block_table=table.cpu())
        append("bfloat16", fp8=fp8, k=k.float())
        append("bfloat16", fp8=fp8, q=q.half())
        append("dense", fp8=fp8, q=torch.zeros(2, D, 4, dtype=torch.bfloat16, device=dev).transpose(1, 2))
        append("same shape", fp8=fp8, v=q)
        append("same tokens", fp8=fp8, q=q[:1])
        append("q_out", fp8=fp8, q_out=q[:, :2].contiguous())
        append("q_out without q", fp8=fp8, q=None, q_out=q)
        append("qo_indptr", fp8=fp8, qo_indptr=lens)
        append("kv_indptr", fp8=fp8, block_table=lens, kv_indptr=lens)
        append("positions", fp8=fp8, positions=ptr)
        append("cos_sin", fp8=fp8, cos_sin=torch.zeros(9, 16, dtype=torch.float64, device=dev))
        append("unsupported", attn.AttnError, fp8=fp8, cos_sin=torch.zeros(9, 18, device=dev))
        append("invalid", attn.AttnError, fp8=fp8, cos_sin=torch.zeros(9, 144, device=dev))
        append("invalid", attn.AttnError, fp8=fp8, k=k[:1].expand(2, 2, D))
        append("invalid", attn.AttnError, fp8=fp8, k=torch.zeros(2 * 2 * D + 4, dtype=torch.bfloat16, device=dev)[4:].view(2, 2, D))
        append("dev_status", fp8=fp8, dev_status=lens.long())
    append("k_cache", k_cache=cb)
    append("v_cache", v_cache=c8[:2])
    append("contiguous", k_cache=c8.transpose(1, 2).contiguous().transpose(1, 2))
    append("blocks", k_scale=torch.ones(3, 5, 2, device=dev))
    append("v_scale", v_scale=torch.ones(3, 1, 2, device=dev))
    append("heads", k=q, v=q)
    append("k_cache", fp8=False, k_cache=c8)
    append("unsupported", attn.AttnError, k_scale=torch.ones(3, 4, 2, device=dev), v_scale=torch.ones(3, 4, 2, device=dev))
    for f, extra in ((attn.attn_decode_paged_fp8_block, ()), (attn.attn_prefill_paged_fp8_block, (ptr,))):
        with pytest.raises(ValueError, match="q must"):
            f(q[0], c8, c8, sc, sc, *extra, table, lens)
        with pytest.raises(ValueError, match="head dimension"):
            f(q[..., :64].contiguous(), c8, c8, sc, sc, *extra, table, lens)
        with pytest.raises(attn.AttnError, match="workspace"):
            f(q, c8, c8, sc, sc, *extra, table, lens, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
        with pytest.raises(ValueError, match="lse"):
            f(q, c8, c8, sc, sc, *extra, table, lens, lse=torch.zeros(2, 4, dtype=torch.float64, device=dev))
    torch.cuda.synchronize()
    assert not torch.any(c8) and not torch.any(cb) and bool(torch.all(sc == 1)) and bool(torch.all(q == 1))

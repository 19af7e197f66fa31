"""Calls of the serving cache's entries that a serving loop makes now and then: rows of no sequence around a batch, sequences
with fewer tokens than new rows, steps captured once and replayed over other lengths, the largest batches."""

import numpy as np
import pytest
import torch

import block_cache as bc
from parity import gpu_or_skip
from test_gpu_fp8_block import Cache

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("block,page", [(16, 48), (64, 64)])
@pytest.mark.parametrize("fp8", [False, True])
def test_ragged_append_rows_of_no_sequence_and_negative_indices(fp8, block, page):
    """Rows before the first and behind the last sequence stay out, and of a sequence with more new rows than tokens the first
    ones do: neither cache nor q_out takes them."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(block)
    hq, hkv = 6, 2
    ptr = np.array([5, 25, 25, 61, 130])
    lens = [3, 0, 100, 69]                       # the first has 20 rows for 3 tokens
    total = 140
    q, k, v = (bc.bf16(rng.standard_normal((total, h, D))) for h in (hq, hkv, hkv))
    lists = bc.Lists(lens, page, rng)
    pages, _ = lists.tensors(dev)
    table = bc.rope_table(128, D)
    shape, blocks = (lists.num_pages, page, hkv, D), (lists.num_pages, page // block, hkv)
    kind = torch.uint8 if fp8 else torch.bfloat16
    caches = [torch.full(shape, 7, dtype=kind, device=dev) for _ in range(2)]
    scales = [torch.ones(blocks, device=dev) for _ in range(2)] if fp8 else []
    out = torch.full((total, hq, D), 9.0, dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    call = attn.attn_kv_append_fp8_block if fp8 else attn.attn_kv_append
    call(q.to(dev), k.to(dev), v.to(dev), *caches, *scales, pages, torch.tensor(lens, dtype=torch.int32, device=dev),
         cos_sin=torch.from_numpy(table).to(dev), qo_indptr=torch.tensor(ptr, dtype=torch.int32, device=dev), q_out=out,
         dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    taken = np.zeros(total, bool)
    codes = [np.full(shape, 7, np.uint8) for _ in range(2)]
    want_s = [np.ones(blocks, np.float32) for _ in range(2)]
    for b, n in enumerate(lens):
        t = n - (ptr[b + 1] - ptr[b]) + np.arange(ptr[b + 1] - ptr[b])
        rows, t = np.arange(ptr[b], ptr[b + 1])[t >= 0], t[t >= 0]
        taken[rows] = True
        if not len(t):
            continue
        x = q[rows].double().numpy()
        want, slack = (f(x, table, t, False) for f in (bc.rotate, bc.rotate_slack))
        assert np.all(np.abs(out[rows].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * slack)
        for w, y in enumerate((bc.rotate(k[rows].double().numpy(), table, t, False), v[rows].double().numpy())):
            if fp8:
                bc.append_blocks(codes[w], want_s[w], lists, block, b, int(t[0]), y)
            else:
                at = (lists.rows[b][t // page], t % page)
                got = caches[w].double().cpu().numpy()[at]
                room = bc.rotate_slack(k[rows].double().numpy(), table, t, False) if w == 0 else 0.0
                assert np.all(np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -22 * room)
    assert taken.sum() == 3 + 36 + 69 and bool((out[torch.from_numpy(~taken).to(dev)] == 9).all())
    if fp8:
        for w in range(2):
            assert np.array_equal(scales[w].cpu().numpy(), want_s[w]) and np.array_equal(caches[w].cpu().numpy(), codes[w])
    else:
        assert all(int((c == 7).all(dim=-1).all(dim=-1).sum()) == lists.num_pages * page - taken.sum() for c in caches)


def test_prefill_rows_of_no_sequence_stay():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(3)
    lens, ptr = [150, 40, 300], np.array([7, 57, 57, 300])
    cache = Cache(lens, 2, 48, 16, rng)
    pages, _ = cache.lists.tensors(dev)
    q = bc.bf16(rng.standard_normal((320, 8, D)))
    o = torch.full((320, 8, D), 9.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((320, 8), 9.0, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    attn.attn_prefill_paged_fp8_block(q.to(dev), *cache.device(dev), torch.tensor(ptr, dtype=torch.int32, device=dev), pages,
                                      torch.tensor(lens, dtype=torch.int32, device=dev), max_kv_rows=sum(lens), o=o, lse=lse,
                                      dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for part in (slice(0, 7), slice(300, 320)):
        assert bool((o[part] == 9).all()) and bool((lse[part] == 9).all())
    for b in range(3):
        rows = slice(ptr[b], ptr[b + 1])
        if ptr[b + 1] > ptr[b]:
            bc.check_attention(o[rows], lse[rows], bc.attend(q[rows].double().numpy(), *cache.values(b), weight_step=2.0 ** -8, small=0.0))


def test_steps_captured_and_replayed_over_other_lengths():
    """A prompt step (ragged append, prefill) and a decode over the same cache, captured once each, the latter twice with a
    workspace each, and replayed over other lengths and inputs: equal bits to eager calls.  Among the lengths are ones for which
    the decode cuts no sequence."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(9)
    n, hq, hkv, page, block, total, cap = 3, 8, 2, 64, 32, 200, 2048
    lists = bc.Lists([cap] * n, page, rng)
    pages, _ = lists.tensors(dev)
    cs = torch.from_numpy(bc.rope_table(cap, D)).to(dev)
    start = Cache([cap] * n, hkv, page, block, rng)
    start.lists = lists
    kept = [torch.from_numpy(np.where(np.isnan(x), 0.01, x) if x.dtype == np.float32 else x % 127).to(dev) for x in start.codes + start.scales]
    cache = [x.clone() for x in kept]
    bufs = [torch.empty(total, h, D, dtype=torch.bfloat16, device=dev) for h in (hq, hkv, hkv)]
    ptr, lens = torch.zeros(n + 1, dtype=torch.int32, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
    turned, o = (torch.zeros(total, hq, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    lse = torch.zeros(total, hq, device=dev)
    dq = torch.empty(n, 2, hq, D, dtype=torch.bfloat16, device=dev)
    do = [torch.empty_like(dq) for _ in range(3)]
    dl = [torch.empty(n, 2, hq, device=dev) for _ in range(3)]
    ws = [torch.empty(attn.attn_decode_fp8_block_workspace_bytes(n, 2, hq, hkv), dtype=torch.uint8, device=dev) for _ in range(3)]
    pws = torch.empty(attn.attn_prefill_fp8_block_workspace_bytes(n, n * cap, hkv), dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def prompts():
        attn.attn_kv_append_fp8_block(*bufs, *cache, pages, lens, cos_sin=cs, qo_indptr=ptr, q_out=turned, dev_status=status)
        attn.attn_prefill_paged_fp8_block(turned, *cache, ptr, pages, lens, max_kv_rows=n * cap, workspace=pws, o=o, lse=lse,
                                          dev_status=status)

    def answer(i):
        attn.attn_decode_paged_fp8_block(dq, *cache, pages, lens, workspace=ws[i], o=do[i], lse=dl[i], dev_status=status)

    def fill(seed, at, after):
        g = np.random.default_rng(seed)
        for x in bufs + [dq]:
            x.copy_(bc.bf16(g.standard_normal(tuple(x.shape))).to(dev))
        ptr.copy_(torch.tensor(at, dtype=torch.int32))
        lens.copy_(torch.tensor(after, dtype=torch.int32))
        for x, y in zip(cache, kept):
            x.copy_(y)
        for x in [turned, o, lse] + do + dl:
            x.zero_()

    fill(0, [0, 100, 150, 200], [100, 50, 50])
    prompts(), answer(0)
    torch.cuda.synchronize()
    graphs = []
    for f in (prompts, lambda: answer(1), lambda: answer(2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for seed, (at, after) in enumerate([([0, 100, 150, 200], [100, 50, 50]), ([0, 1, 1, 200], [2048, 0, 199]),
                                        ([0, 70, 160, 200], [90, 96, 40]), ([0, 0, 0, 200], [5, 2047, 1500]),
                                        ([3, 3, 90, 190], [1, 700, 100])]):
        fill(seed, at, after)
        prompts(), answer(0)
        torch.cuda.synchronize()
        want = [x.clone() for x in cache + [turned, o, lse, do[0], dl[0]]]
        fill(seed, at, after)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert status.item() == 0
        for i in (1, 2):
            got = cache + [turned, o, lse, do[i], dl[i]]
            assert all(torch.equal(x, y) for x, y in zip(got, want)), (seed, i)


@pytest.mark.parametrize("top", [40, 300])
def test_decode_of_the_largest_batch(top):
    """4096 sequences, with and without cuts among them; every 512th and the longest are checked."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    rng = np.random.default_rng(top)
    lens = rng.integers(0, top, 4096).tolist()
    lens[7], lens[4095] = 0, 2 * top
    cache = Cache(lens, 1, 16, 16, rng, csr=True)
    q = bc.bf16(rng.standard_normal((4096, 1, 2, D)))
    pages, indptr = cache.lists.tensors(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse, _ = attn.attn_decode_paged_fp8_block(q.to(dev), *cache.device(dev), pages, torch.tensor(lens, dtype=torch.int32, device=dev),
                                                 kv_indptr=indptr, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and bool(torch.isfinite(o.float()).all())
    empty = torch.tensor([n == 0 for n in lens], device=dev)
    assert torch.equal(torch.isneginf(lse[:, 0]).any(dim=1), empty) and not bool(o[empty].any())
    for b in sorted({*range(0, 4096, 512), 4095, 7, 8, int(np.argmax(lens[:4095]))}):
        bc.check_attention(o[b], lse[b], bc.attend(q[b].double().numpy(), *cache.values(b)))

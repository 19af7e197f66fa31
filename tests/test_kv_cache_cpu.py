"""Refusals of the paged cache's writers and of the block-scaled cache's readers: on the host, before anything is enqueued,
through the C ABI and through the Python binding; and the sizes of the workspaces."""

import ctypes

import numpy as np
import pytest
import torch

import block_cache as bc

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import causal_gqa_flashattention_attn_gb300 as attn
    return attn.lib()


def _append(L, fp8, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=4096, ks=1024, vs=1024, cs=FAKE, max_pos=100, rot=128, inter=0, pos=None, qo=FAKE,
             lens=FAKE, table=FAKE, kvp=None, mp=4, qout=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, B=2, T=0, Hq=32, Hkv=8,
             D=128, pages=8, ps=64, block=32)
    a.update(kw)
    head = [a[n] for n in ("q", "k", "v", "qs", "ks", "vs", "cs", "max_pos", "rot", "inter", "pos", "qo", "lens", "table", "kvp",
                           "mp", "qout", "kc", "vc")]
    sizes = [a[n] for n in ("B", "T", "Hq", "Hkv", "D", "pages", "ps")]
    if fp8:
        return L.attn_kv_append_fp8_block(*head, a["ksc"], a["vsc"], *sizes, a["block"], None, None)
    return L.attn_kv_append(*head, *sizes, None, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_validation(L, fp8):
    assert _append(L, fp8) == 0                              # no new tokens: nothing to do
    assert _append(L, fp8, q=None, k=None, v=None, qout=None) == 0
    for name in ("k", "v", "kc", "vc", "table", "lens"):
        assert _append(L, fp8, T=2, **{name: None}) == -1, name
    for name in ("q", "k", "v", "kc", "vc", "cs", "qout"):
        assert _append(L, fp8, **{name: ODD}) == -1, name    # misaligned
    assert _append(L, fp8, T=2, q=None) == -1                # q_out without q
    assert _append(L, fp8, T=2, qout=None) == -1
    assert _append(L, fp8, q=None, qout=None) == 0
    assert _append(L, fp8, qs=4100) == -1                    # rows that are not 16-byte aligned
    assert _append(L, fp8, ks=1016) == -1                    # rows that overlap
    assert _append(L, fp8, vs=-1024) == -1
    assert _append(L, fp8, qs=8192, qout=FAKE, q=FAKE) == -1   # in place, but q is not dense
    assert _append(L, fp8, q=ctypes.c_void_p(0x20000), qs=8192) == 0
    assert _append(L, fp8, qo=None) == -1                    # one token each: total_q = B
    assert _append(L, fp8, T=-1) == -1
    assert _append(L, fp8, B=0) == -1
    assert _append(L, fp8, Hq=30) == -1
    assert _append(L, fp8, pages=0) == -1
    assert _append(L, fp8, ps=0) == -1
    assert _append(L, fp8, mp=0) == -1
    assert _append(L, fp8, mp=0, kvp=FAKE) == 0
    assert _append(L, fp8, D=64) == -2
    assert _append(L, fp8, rot=-16) == -1
    assert _append(L, fp8, rot=144) == -1
    assert _append(L, fp8, rot=24) == -2
    assert _append(L, fp8, cs=None) == -1
    assert _append(L, fp8, max_pos=0) == -1
    assert _append(L, fp8, cs=None, max_pos=0, rot=0) == 0
    assert _append(L, fp8, inter=2) == -1
    assert _append(L, fp8, pages=1 << 25) == -2              # 2^31 rows
    assert _append(L, fp8, T=(1 << 31) - 1) == -2            # a grid of that many CTAs and more
    if fp8:
        assert _append(L, fp8, ksc=None) == -1
        assert _append(L, fp8, vsc=None) == -1
        assert _append(L, fp8, block=0) == -1
        assert _append(L, fp8, block=48) == -1               # does not divide the page
        assert _append(L, fp8, block=8) == -2
    else:
        assert _append(L, fp8, ps=7) == 0                    # any page size


def _decode(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, kvp=None, mp=4, lens=FAKE, B=2, nq=1, Hq=32, Hkv=8, D=128,
             pages=8, ps=64, block=32, scale=0.1, ws=FAKE, bytes=0, o=FAKE, lse=None)
    a.update(kw)
    return L.attn_decode_paged_fp8_block(*a.values(), None, None)


def test_decode_validation(L):
    for name in ("q", "k", "v", "ks", "vs", "table", "lens", "o"):
        assert _decode(L, **{name: None}) == -1, name
    for name in ("q", "k", "v", "o"):
        assert _decode(L, **{name: ODD}) == -1, name
    assert _decode(L, nq=0) == -1
    assert _decode(L, nq=17) == -2
    assert _decode(L, Hq=30) == -1
    assert _decode(L, D=64) == -2
    assert _decode(L, block=48) == -1
    assert _decode(L, block=8) == -2
    assert _decode(L, scale=float("nan")) == -1
    assert _decode(L, B=4097) == -2
    assert _decode(L, B=4096, mp=1 << 18) == -2              # tiles past int
    assert _decode(L, B=4096, mp=(1 << 31) - 1, ps=(1 << 31) - 64, pages=1, block=64) == -2   # and past 64 bits
    assert _decode(L, Hq=1 << 20, Hkv=1 << 20) == -2
    assert _decode(L, ws=None) == -3
    assert _decode(L, ws=ODD) == -3
    import causal_gqa_flashattention_attn_gb300 as attn
    assert attn.attn_decode_fp8_block_workspace_bytes(0, 1, 32, 8) == 0
    assert attn.attn_decode_fp8_block_workspace_bytes(2, 17, 32, 8) == 0
    assert attn.attn_decode_fp8_block_workspace_bytes(2, 1, 30, 8) == 0
    # heads beyond what the entry takes, whose rows would pass 32 bits
    assert attn.attn_decode_fp8_block_workspace_bytes(1, 16, 1 << 28, 1) == 0
    assert attn.attn_decode_fp8_block_workspace_bytes(1, 1, (1 << 31) - 1, 1) == 0
    if torch.cuda.is_available():
        assert _decode(L) == -3                              # a workspace of no bytes
    else:
        assert _decode(L) == -4                              # no device


def _prefill(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, qo=FAKE, table=FAKE, kvp=None, mp=4, lens=FAKE, B=2, T=0, Hq=32, Hkv=8,
             D=128, pages=8, ps=64, block=32, rows=300, scale=0.1, ws=FAKE, bytes=1 << 40, o=FAKE, lse=None)
    a.update(kw)
    return L.attn_prefill_paged_fp8_block(*a.values(), None, None)


def test_prefill_validation(L):
    import causal_gqa_flashattention_attn_gb300 as attn
    need = attn.attn_prefill_fp8_block_workspace_bytes(2, 300, 8)
    # K and V copies of 300 rows, each of 2 sequences up to a multiple of 128: ceil((300 + 2 * 127) / 128) * 128 = 640 rows;
    # 4096 words of order; 5 page words, rounded to 16 bytes
    assert need == 2 * 640 * 8 * 128 * 2 + 4096 * 4 + 32
    assert attn.attn_prefill_fp8_block_workspace_bytes(2, 0, 8) == 0
    assert attn.attn_prefill_fp8_block_workspace_bytes(1, (1 << 31) - 1, 8) == 0     # beyond what the entry takes
    assert attn.attn_prefill_fp8_block_workspace_bytes(1, 1 << 30, (1 << 31) - 1) == 0
    assert _prefill(L, bytes=need) == 0
    assert _prefill(L, bytes=need - 1) == -3
    assert _prefill(L, ws=None) == -3
    assert _prefill(L, ws=ODD) == -3
    for name in ("q", "k", "v", "ks", "vs", "qo", "table", "lens", "o"):
        assert _prefill(L, T=2, **{name: None}) == -1, name
    assert _prefill(L, q=None, o=None) == 0
    for name in ("q", "k", "v", "o"):
        assert _prefill(L, **{name: ODD}) == -1, name
    assert _prefill(L, T=-1) == -1
    assert _prefill(L, rows=0) == -1
    assert _prefill(L, scale=float("inf")) == -1
    assert _prefill(L, scale=0.0) == -2 and _prefill(L, scale=-0.1) == -2
    assert _prefill(L, Hq=30) == -1
    assert _prefill(L, D=64) == -2
    assert _prefill(L, block=8) == -2
    assert _prefill(L, Hq=129, Hkv=1) == -2
    assert _prefill(L, B=2049) == -2
    assert _prefill(L, T=1 << 22) == -2
    assert _prefill(L, rows=(1 << 31) - 100) == -2


def test_binding_refuses_host_tensors(L):
    import causal_gqa_flashattention_attn_gb300 as attn
    q, k = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(3, 32, 2, 128, dtype=torch.uint8)
    scales = torch.ones(3, 2, 2)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        attn.attn_kv_append_fp8_block(q, k, k, cache, cache, scales, scales, table, lens)
    with pytest.raises(ValueError, match="current CUDA device"):
        attn.attn_kv_append(q, k, k, cache, cache, table, lens)
    with pytest.raises(ValueError, match="current CUDA device"):
        attn.attn_decode_paged_fp8_block(q, cache, cache, scales, scales, table, lens)
    with pytest.raises(ValueError, match="current CUDA device"):
        attn.attn_prefill_paged_fp8_block(q, cache, cache, scales, scales, lens, table, lens)
    with pytest.raises(ValueError, match="k_scale"):
        attn.attn_kv_append_fp8_block(q, k, k, cache, cache, None, scales, table, lens)
    with pytest.raises(ValueError, match="must be a tensor"):
        attn.attn_kv_append(q, None, k, cache, cache, table, lens)


def test_plain_cache_rounds_as_e4m3():
    """The tests' own conversion against torch's, ties and both ends of the range among the values."""
    x = np.random.default_rng(0).standard_normal(20000) * 100
    mids = (bc._POS[1:] + bc._POS[:-1]) / 2
    x = np.clip(np.concatenate([x, mids, -mids, bc._POS, np.arange(100) * 2.0 ** -11]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(bc.e4m3_code(x), want)
    assert bc.e4m3_code([np.nan, np.inf, -np.inf]).tolist() == [0x7F, 0x7E, 0xFE]
    assert [bc.scale_of(np.array([v])) for v in (0.0, 448.0, 448.5, 224.0, 2.0 ** -140)] == [0.0, 1.0, 2.0, 0.5, 2.0 ** -126]

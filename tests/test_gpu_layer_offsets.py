"""Offsets that fall, so that the sequences share rows and together name many times what the tensors hold."""

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu


def _falling(n, count, dev):
    """0, n, 0, n, ...: every other sequence owns all n rows."""
    return (torch.arange(count + 1, device=dev) % 2 * n).to(torch.int32)


def test_single_tokens_past_32_bits_of_tiles():
    """2048 sequences of 2^24 keys: 2^31 tiles, where counts of tiles in 32 bits turn negative."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    n, count = 1 << 24, 4096
    k = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device=dev)
    q = torch.randn(count, 1, 64, device=dev).to(torch.bfloat16)
    o, lse = torch.full_like(q, 7.0), torch.full((count, 1), 7.0, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    attn.attn_cross_decode(q, k, k, _falling(n, count, dev), o=o, lse=lse, dev_status=status)
    assert status.item() == attn.ATTN_DEV_SEQ_TOO_LONG and (o == 7).all() and (lse == 7).all()
    # few keys each: the sequences that share them are computed
    status.zero_()
    lens = (torch.arange(count, device=dev) % 50).to(torch.int32)
    attn.attn_cross_decode(q, k, k, _falling(n, count, dev), kv_lens=lens, o=o, lse=lse, dev_status=status)
    want = torch.where((torch.arange(count, device=dev) % 2 == 0) & (lens > 0), lens.double().log(), -float("inf"))
    assert status.item() == 0 and (o == 0).all()
    ragged.check("lse", lse[:, 0], want, torch.full_like(want, 1e-5))


def test_single_tokens_that_share_keys():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [1], [700], 8, 2, 128, seed=71)
    q = x.q.expand(5, 8, 128).contiguous()
    o, lse, _ = attn.attn_cross_decode(q, x.k, x.v, _falling(700, 5, dev))
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    for b in (0, 2, 4):
        ragged.check("o", o[b:b + 1], want_o, tol_o)
        ragged.check("lse", lse[b:b + 1], want_l, tol_l)
    for b in (1, 3):
        assert (o[b] == 0).all() and (lse[b] == -float("inf")).all()


@pytest.mark.parametrize("causal", [False, True])
def test_ragged_batches(causal):
    """1024 sequences of the same 40000 queries and keys: what a call may work on is bounded by the tensors, and the next call
    over the same workspace is right."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [40000], [64], 2, 1, 64, seed=72, causal=False)
    at, kv = _falling(40000, 2047, dev), _falling(64, 2047, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse = torch.full_like(x.q, 7.0), torch.full((40000, 2), 7.0, device=dev)
    attn.attn_varlen_fwd(x.q, x.k, x.v, at, kv, causal=causal, o=o, lse=lse, dev_status=status)
    attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, at, kv, causal=causal, dev_status=status)
    assert status.item() == 0
    if not causal:   # the first sequence's rows are all there, whoever else writes the same
        want_o, want_l, tol_o, tol_l = ragged.forward(x)
        ragged.check("o", o, want_o, tol_o)
    y = ragged.Batch(dev, [300, 70], [200, 90], 2, 1, 64, seed=73, causal=causal)
    o, lse, _ = attn.attn_varlen_fwd(y.q, y.k, y.v, **y.args())
    want_o, want_l, tol_o, tol_l = ragged.forward(y)
    ragged.check("o", o, want_o, tol_o)
    ragged.check("lse", lse, want_l, tol_l)
    want, tol = ragged.backward(y, o, lse)
    for label, got, w, t in zip(("dq", "dk", "dv"), attn.attn_varlen_bwd(y.do, y.q, y.k, y.v, o, lse, **y.args()), want, tol):
        ragged.check(label, got, w, t)

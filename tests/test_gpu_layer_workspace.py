"""Workspace sizes of the layer's operators: those of calls that the entries refuse are 0."""

import pytest

from parity import gpu_or_skip

pytestmark = pytest.mark.gpu


def test_sizes_of_refused_calls():
    gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    fwd, bwd = attn.attn_varlen_fwd_workspace_bytes, attn.attn_varlen_bwd_workspace_bytes
    good = (1, 4, 100000, 8, 2, 128)   # B, total_q, total_kv, Hq, Hkv, D
    assert fwd(*good) >= 4 * 8 * 2 * 129 * 4 and bwd(*good) > 0
    for at, value in ((0, 0), (0, 2049), (1, 1 << 22), (1, -1), (2, 1 << 30), (2, -1), (3, 7), (3, 258), (4, 3), (5, 96), (5, 256)):
        bad = list(good)
        bad[at] = value
        assert fwd(*bad) == 0 and bwd(*bad) == 0, bad
    most = (1 << 31) - 1
    assert fwd(most, most, most, most, most, most) == 0 and bwd(most, most, most, most, most, most) == 0
    assert fwd(1, 1, 1, 1 << 24, 1 << 24, 128) == 0 and bwd(1, 1, 1, 1 << 24, 1 << 24, 128) == 0   # rows of 2^31 elements
    assert attn.attn_cross_decode_workspace_bytes(4096, 1, 32, 8) > 0
    for bad in ((4097, 1, 32, 8), (4096, 16, 1 << 15, 1 << 12), (0, 1, 32, 8), (1, 17, 32, 8)):
        assert attn.attn_cross_decode_workspace_bytes(*bad) == 0
    assert attn.attn_qk_norm_rope_bwd_workspace_bytes(0, 4, 0) > 0
    for bad in ((-1, 4, 2), (5, 0, 0), (1 << 28, 8, 1), (5, 4, 2, 96)):
        assert attn.attn_qk_norm_rope_bwd_workspace_bytes(*bad) == 0

"""Sizes that the norms with rotation and attention over contiguous keys refuse: on the host, before anything is enqueued."""

import pytest

from test_layer_cpu import L, _norm, _norm_bwd, _varlen, _varlen_bwd   # noqa: F401  (L is the fixture)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_rows(L, call):   # noqa: F811
    """Rows are counted in int, some steps of the grid ahead of the last one."""
    most, wide = (1 << 31) - (1 << 20), 1 << 38
    strides = dict(qs=wide, qos=wide) if call is _norm else dict(qs=wide, dqos=wide, dqs=wide)
    for tokens in (0, 1):   # (no tokens: the sides' parts of the grid go by the heads all the same)
        assert call(L, T=tokens, Hq=most, Hkv=1, **strides) == -2
    assert call(L, T=0, Hq=most - 8, **strides) == 0
    assert call(L, T=1 << 17, Hq=1 << 13, Hkv=1 << 13, ks=1 << 20, **strides,
                **(dict(kos=1 << 20) if call is _norm else dict(dkos=1 << 20, dks=1 << 20))) == -2


def _rows(call, heads):
    """Token rows of every argument as far apart as `heads` heads of 128 need."""
    names = ("qs", "ks", "vs") if call is _varlen else ("qs", "ks", "vs", "dos", "os", "dqs", "dks", "dvs")
    return {name: heads * 128 for name in names}


@pytest.mark.parametrize("call", [_varlen, _varlen_bwd])
def test_heads_of_attention(L, call):   # noqa: F811
    """A token's row has fewer than 2^31 elements; rows and work items are counted in int, a step of the grid ahead."""
    for heads, sequences in ((1 << 24, 1), ((1 << 20) - 1, 2047)):
        assert call(L, T=1, S=1, B=sequences, Hq=heads, Hkv=heads, **_rows(call, heads)) == -2
        assert call(L, T=0, S=0, B=sequences, Hq=heads, Hkv=heads, **_rows(call, heads)) == (-2 if heads == 1 << 24 else 0)

"""Sizes that the norms with rotation and attention over contiguous keys refuse: on the host, before anything is enqueued."""

import pytest

from test_layer_cpu import L, _norm, _norm_bwd   # noqa: F401  (L is the fixture)


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

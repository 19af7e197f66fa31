"""Sizes that the norms with rotation and attention over contiguous keys refuse: on the host, before anything is enqueued."""

import ctypes

import pytest

from test_layer_cpu import FAKE, L, _norm, _norm_bwd, _varlen, _varlen_bwd   # noqa: F401  (L is the fixture)


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


@pytest.mark.parametrize("call", [_varlen, _varlen_bwd])
def test_limits_of_attention(L, call):   # noqa: F811
    """Each bound that the header gives, passed by one (no call gets as far as a launch)."""
    assert call(L, Hq=129, Hkv=1, T=2, **_rows(call, 129)) == -2
    assert call(L, Hq=128, Hkv=1, S=0, **_rows(call, 128)) == 0
    assert call(L, T=1 << 22) == -2 and call(L, S=1 << 30) == -2 and call(L, B=2049) == -2
    assert call(L, S=1 << 28, Hkv=8) == -2
    assert call(L, T=1, Hq=8, Hkv=8, S=(1 << 28) + 1) == -2
    for stride in ("qs", "ks", "vs") + (("dos",) if call is _varlen_bwd else ()):
        assert call(L, **{stride: 1 << 38}) == -2, stride


def test_limits_of_single_tokens(L):   # noqa: F811
    def call(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, ks=1 << 20, vs=1 << 20, kv=FAKE, lens=None, B=2, nq=1, S=10, Hq=32, Hkv=8, D=128,
                 scale=0.1, ws=None, bytes=0, o=ctypes.c_void_p(0x20000), lse=None)
        a.update(kw)
        return L.attn_cross_decode(*a.values(), None, None)

    assert call() == -3                                   # sizes are fine, the workspace is not there
    assert call(Hq=1 << 16, Hkv=1 << 12, nq=16) == -2     # 2^20 rows a sequence
    assert call(Hq=(1 << 16) - 16, Hkv=16, nq=16) == -3
    assert call(Hq=1 << 15, Hkv=1 << 12, nq=16, B=4096) == -2
    assert call(Hq=1 << 15, Hkv=1 << 12, nq=16, B=4095) == -3
    assert call(S=1 << 30) == -2 and call(S=(1 << 30) - 1) == -3
    assert call(ks=1 << 38) == -2 and call(vs=1 << 38) == -2 and call(B=4097) == -2 and call(nq=17) == -2

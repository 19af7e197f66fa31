"""Refusals of the norms with rotation and of attention over contiguous keys: on the host, before anything is enqueued, through
the C ABI and through the Python binding."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)
NO_DEVICE = not torch.cuda.is_available()


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import causal_gqa_flashattention_attn_gb300 as attn
    return attn.lib()


def _norm(L, **kw):
    a = dict(q=FAKE, k=FAKE, qs=4096, ks=1024, qw=FAKE, kw=FAKE, wt=0, eps=1e-6, cs=FAKE, max_pos=100, rot=128, inter=0, pos=None,
             qo=FAKE, ko=FAKE, qos=4096, kos=1024, T=0, Hq=32, Hkv=8, D=128)
    a.update(kw)
    return L.attn_qk_norm_rope(*a.values(), None, None)


def _norm_bwd(L, **kw):
    a = dict(dqo=FAKE, dko=FAKE, dqos=4096, dkos=1024, q=FAKE, k=FAKE, qs=4096, ks=1024, qw=FAKE, kw=FAKE, wt=0, eps=1e-6, cs=FAKE,
             max_pos=100, rot=128, inter=0, pos=None, dq=FAKE, dk=FAKE, dqs=4096, dks=1024, dqw=None, dkw=None, T=0, Hq=32, Hkv=8,
             D=128, ws=None, bytes=0)
    a.update(kw)
    return L.attn_qk_norm_rope_bwd(*a.values(), None, None)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_validation(L, call):
    assert call(L) == 0                                       # no tokens: nothing to do
    absent = dict(k=None, Hkv=0, ks=0, kw=None)
    absent.update(dict(ko=None, kos=0) if call is _norm else dict(dko=None, dkos=0, dk=None, dks=0))
    assert call(L, **absent) == 0                             # queries alone
    assert call(L, **{**absent, "kw": FAKE}) == -1
    assert call(L, Hq=0, Hkv=0) == -1
    for name in ("q", "k") + (("qo", "ko") if call is _norm else ("dqo", "dko", "dq", "dk")):
        assert call(L, T=2, **{name: None}) == -1, name
        assert call(L, **{name: ODD}) == -1, name
    for name in ("qw", "kw", "cs"):
        assert call(L, **{name: ODD}) == -1, name
    for name in ("qs", "qos" if call is _norm else "dqs"):
        assert call(L, **{name: 4100}) == -1
        assert call(L, **{name: 4088}) == -1
    if call is _norm:
        assert call(L, q=FAKE, qo=FAKE, qs=8192, ks=1024, kos=1024, ko=ctypes.c_void_p(0x20000)) == -1   # in place, other strides
    assert call(L, T=-1) == -1
    assert call(L, eps=0.0) == -1 and call(L, eps=float("nan")) == -1
    assert call(L, eps=0.0, qw=None, kw=None) == 0            # rotation alone
    assert call(L, wt=2) == -2
    assert call(L, D=96, qs=8192, ks=8192) in (-1, -2)
    assert call(L, rot=-16) == -1 and call(L, rot=144) == -1
    assert call(L, rot=24) == -2
    assert call(L, cs=None) == -1 and call(L, max_pos=0) == -1 and call(L, inter=2) == -1
    assert call(L, cs=None, max_pos=0, rot=0) == 0
    assert call(L, T=1 << 26) == -2


def test_norm_backward_workspace(L):
    import causal_gqa_flashattention_attn_gb300 as attn
    assert _norm_bwd(L, dqw=FAKE) == -3
    assert _norm_bwd(L, dqw=FAKE, ws=ODD, bytes=1 << 30) == -3
    assert _norm_bwd(L, dqw=FAKE, qw=None) == -1
    assert _norm_bwd(L, dqw=FAKE, ws=FAKE) == (-4 if NO_DEVICE else -3)
    assert attn.attn_qk_norm_rope_bwd_workspace_bytes(5, 4, 2, 96) == 0
    # both sides' sums into one buffer
    assert _norm_bwd(L, dqw=FAKE, dkw=FAKE, ws=FAKE, bytes=1 << 30) == -1


def _varlen(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=4096, ks=1024, vs=1024, qo=FAKE, kv=FAKE, lens=None, causal=0, B=2, T=0, S=10, Hq=32, Hkv=8,
             D=128, scale=0.1, ws=None, bytes=0, o=FAKE, lse=None)
    a.update(kw)
    return L.attn_varlen_fwd(*a.values(), None, None)


def _varlen_bwd(L, **kw):
    a = dict(do=FAKE, q=FAKE, k=FAKE, v=FAKE, o=FAKE, dos=4096, qs=4096, ks=1024, vs=1024, os=4096, lse=FAKE, dlse=None, qo=FAKE,
             kv=FAKE, lens=None, causal=0, B=2, T=0, S=0, Hq=32, Hkv=8, D=128, scale=0.1, ws=FAKE, bytes=0, dq=FAKE, dk=FAKE,
             dv=FAKE, dqs=4096, dks=1024, dvs=1024)
    a.update(kw)
    return L.attn_varlen_bwd(*a.values(), None, None)


@pytest.mark.parametrize("call", [_varlen, _varlen_bwd])
def test_varlen_validation(L, call):
    assert call(L) == 0                                       # no queries (backward: and no keys)
    for name in ("q", "o") + (("do", "lse", "dq") if call is _varlen_bwd else ()):
        assert call(L, T=2, S=10, **{name: None}) == -1, name
    for name in ("k", "v") + (("dk", "dv") if call is _varlen_bwd else ()):
        assert call(L, T=2, S=10, **{name: None}) == -1, name
    for name in ("qo", "kv"):
        assert call(L, **{name: None}) == -1, name
    for name in ("q", "k", "v", "o") + (("do", "dq", "dk", "dv") if call is _varlen_bwd else ()):
        assert call(L, **{name: ODD}) == -1, name
    for name in ("qs",) + (("dos", "os", "dqs") if call is _varlen_bwd else ()):
        assert call(L, **{name: 4100}) == -1 and call(L, **{name: 4088}) == -1, name
    for name in ("ks", "vs") + (("dks", "dvs") if call is _varlen_bwd else ()):
        assert call(L, **{name: 1028}) == -1 and call(L, **{name: 1016}) == -1, name
    assert call(L, qs=1 << 38) == -2 and call(L, ks=1 << 38) == -2
    assert call(L, B=0) == -1 and call(L, T=-1) == -1 and call(L, S=-1) == -1
    assert call(L, Hq=30) == -1
    assert call(L, causal=2) == -1
    assert call(L, scale=float("inf")) == -1
    assert call(L, scale=0.0) == -2 and call(L, scale=-0.1) == -2
    assert call(L, D=96) == -2
    assert call(L, Hq=129, Hkv=1, qs=1 << 20, dos=1 << 20, os=1 << 20, dqs=1 << 20) == -2 if call is _varlen_bwd else True
    assert call(L, B=2049) == -2
    assert call(L, T=1 << 22) == -2
    assert call(L, S=1 << 30) == -2


def test_varlen_backward_workspace(L):
    import causal_gqa_flashattention_attn_gb300 as attn
    if NO_DEVICE:
        assert _varlen_bwd(L, T=2, S=10) == -4
    else:
        assert _varlen_bwd(L, T=2, S=10) == -3
        assert _varlen_bwd(L, T=2, S=10, ws=None) == -3
        assert _varlen_bwd(L, T=2, S=10, ws=ODD, bytes=1 << 40) == -3
    assert attn.attn_varlen_bwd_workspace_bytes(2, 10, 10, 30, 8) == 0
    assert attn.attn_varlen_fwd_workspace_bytes(0, 10, 10, 32, 8) == 0


def test_cross_decode_validation(L):
    def call(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, ks=1024, vs=1024, kv=FAKE, lens=None, B=2, nq=1, S=10, Hq=32, Hkv=8, D=128, scale=0.1,
                 ws=FAKE, bytes=0, o=FAKE, lse=None)
        a.update(kw)
        return L.attn_cross_decode(*a.values(), None, None)

    import causal_gqa_flashattention_attn_gb300 as attn
    for name in ("q", "k", "v", "kv", "o"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: ODD}) == -1, name
    assert call(ks=1028) == -1 and call(vs=1016) == -1 and call(ks=1 << 38) == -2
    assert call(B=0) == -1 and call(nq=0) == -1 and call(S=-1) == -1 and call(Hq=30) == -1
    assert call(scale=float("nan")) == -1
    assert call(nq=17) == -2 and call(D=96) == -2 and call(B=4097) == -2 and call(S=1 << 30) == -2
    assert call(Hq=1 << 20, Hkv=1) == -2
    assert call(ws=None) == -3 and call(ws=ODD) == -3
    assert call() == (-4 if NO_DEVICE else -3)
    assert attn.attn_cross_decode_workspace_bytes(2, 17, 32, 8) == 0
    assert attn.attn_cross_decode_workspace_bytes(2, 1, 30, 8) == 0
    assert attn.attn_cross_decode_workspace_bytes(2, 1, 32, 8, 96) == 0


def test_binding_refuses_host_tensors(L):
    import causal_gqa_flashattention_attn_gb300 as attn
    q, k = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    at = torch.tensor([0, 2], dtype=torch.int32)
    lse = torch.zeros(2, 4)
    for call in (lambda: attn.attn_qk_norm_rope(q, k), lambda: attn.attn_qk_norm_rope_bwd(q, k, q, k),
                 lambda: attn.attn_varlen_fwd(q, k, k, at, at), lambda: attn.attn_varlen_bwd(q, q, k, k, q, lse, at, at),
                 lambda: attn.attn_cross_decode(q, k, k, at)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    with pytest.raises(ValueError, match="must be a tensor"):
        attn.attn_qk_norm_rope(None, None)
    with pytest.raises(ValueError, match="must be a tensor"):
        attn.attn_varlen_fwd(None, k, k, at, at)

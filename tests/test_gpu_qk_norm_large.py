"""Norms with rotation past 32 bits of a token's elements."""

import pytest
import torch

from parity import gpu_or_skip
from test_gpu_qk_norm import F32, _backward, _forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot", [0, 64])
def test_a_token_past_32_bits(rot):
    """One token of 2^24 + 77 heads of 128: the last ones lie 2^31 elements behind the first."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    heads, d, eps = (1 << 24) + 77, 128, 1e-6
    gen = torch.Generator(device=dev).manual_seed(rot)
    x, dy = (torch.randn(1, heads, d, generator=gen, device=dev, dtype=torch.bfloat16) for _ in range(2))
    w = 1 + 0.3 * torch.randn(d, generator=gen, device=dev)
    table = pos = None
    if rot:
        a = torch.arange(5, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device=dev).double() / rot)
        table, pos = torch.cat([a.cos(), a.sin()], 1).float(), torch.tensor([3], dtype=torch.int32, device=dev)
    more = dict(eps=eps, cos_sin=table, positions=pos)
    y, none = attn.attn_qk_norm_rope(x, None, w, None, **more)
    assert none is None
    dx, _, dw, _, _ = attn.attn_qk_norm_rope_bwd(dy, None, x, None, w, None, **more)
    want_w = torch.zeros(d, dtype=torch.float64, device=dev)
    size_w = torch.zeros_like(want_w)
    step = 1 << 20
    for at in range(0, heads, step):
        part = slice(at, min(at + step, heads))
        want, tol = _forward(x[:, part], w, eps, table, pos, False)
        assert ((y[:, part].double() - want).abs() <= tol).all(), at
        want, tol, sums, bound = _backward(dy[:, part], x[:, part], w, eps, table, pos, False)
        assert ((dx[:, part].double() - want).abs() <= tol).all(), at
        want_w += sums
        size_w += bound / (128 * F32)
    # a lane adds up its rows one after another: the grid has 2 CTAs an SM of 16 groups of lanes (at least 100 SMs), then 128
    # roundings as in the small cases
    chain = heads / (2 * 100 * 16) + 128
    assert ((dw.double() - want_w).abs() <= chain * F32 * size_w).all()

"""The layer's operators as torch.autograd.Function's two methods: torch's own differentiation through them, against float64."""

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu


def test_through_torchs_differentiation():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn

    class Normed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk):
            ctx.save_for_backward(q, k, wq, wk)
            return attn.attn_qk_norm_rope(q, k, wq, wk)

        @staticmethod
        def backward(ctx, dq, dk):
            return attn.attn_qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors)[:4]

    class Attended(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, at):
            o, lse, _ = attn.attn_varlen_fwd(q, k, v, at, at, causal=True)
            ctx.save_for_backward(q, k, v, o, lse, at)
            return o

        @staticmethod
        def backward(ctx, d_o):
            q, k, v, o, lse, at = ctx.saved_tensors
            return (*attn.attn_varlen_bwd(d_o.contiguous(), q, k, v, o, lse, at, at, causal=True)[:3], None)

    x = ragged.Batch(dev, [70, 200], [70, 200], 8, 2, 128, causal=True, seed=51)
    gen = torch.Generator(device=dev).manual_seed(52)
    w = [(1 + 0.2 * torch.randn(128, generator=gen, device=dev)).requires_grad_() for _ in range(2)]
    leaves = [t.clone().requires_grad_() for t in (x.q, x.k, x.v)]
    o = Attended.apply(*Normed.apply(leaves[0], leaves[1], *w), leaves[2], x.qo)
    (o * x.do).sum().backward()

    same = [t.detach().double().requires_grad_() for t in (*leaves, *w)]
    q, k = (t * (t * t).mean(dim=-1, keepdim=True).add(1e-6).rsqrt() * u for t, u in ((same[0], same[3]), (same[1], same[4])))
    want = []
    for a, b in ((0, 70), (70, 270)):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(4, dim=1)) * x.scale
        s = s.masked_fill(~torch.ones(b - a, b - a, dtype=torch.bool, device=dev).tril(), -float("inf"))
        want.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, dim=-1), same[2][a:b].repeat_interleave(4, dim=1)))
    (torch.cat(want) * x.do.double()).sum().backward()
    # norms over a tensor: a handful of roundings to bf16 one after another, 2^-8 of a value each at most and independent from
    # value to value, two of them (the normed rows, in scores of size up to 8) twice that; six units bound them together
    for got, t in zip((*leaves, *w), same):
        assert (got.grad.double() - t.grad).norm() <= 6 * 2.0 ** -8 * t.grad.norm()

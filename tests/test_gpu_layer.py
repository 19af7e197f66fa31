"""The layer's operators one after another, as a decoder uses them: norms with rotation, causal self attention, cross attention
to an encoder's states, their gradients back to the projections; then single tokens over the same states."""

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

HQ, HKV, D = 8, 2, 128


def _rotated(x, table, pos):
    c, s = (u[:, None, :] for u in table.double()[pos.long()].split(table.shape[1] // 2, dim=1))
    a, b = x.split(D // 2, dim=-1)
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1)


def _normed(x, w, eps):
    return x * (x * x).mean(dim=-1, keepdim=True).add(eps).rsqrt() * w


def _attended(q, k, v, q_len, kv_len, causal):
    out, a, b = [], 0, 0
    for n, m in zip(q_len, kv_len):
        s = torch.einsum("ihd,jhd->hij", q[a:a + n], k[b:b + m].repeat_interleave(HQ // HKV, dim=1)) * D ** -0.5
        if causal:
            s = s.masked_fill(~torch.ones(n, m, dtype=torch.bool, device=q.device).tril(m - n), -float("inf"))
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, dim=-1), v[b:b + m].repeat_interleave(HQ // HKV, dim=1)))
        a, b = a + n, b + m
    return torch.cat(out)


def test_training_step_and_single_tokens():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    gen = torch.Generator(device=dev).manual_seed(1)
    q_len, states = [50, 130, 7], [90, 33, 260]
    tq, ts, eps = sum(q_len), sum(states), 1e-6
    qkv = torch.randn(tq, (HQ + 2 * HKV), D, generator=gen, device=dev).to(torch.bfloat16)     # self attention's projection
    cq = torch.randn(tq, HQ, D, generator=gen, device=dev).to(torch.bfloat16)                  # cross attention's queries
    ckv = torch.randn(ts, 2 * HKV, D, generator=gen, device=dev).to(torch.bfloat16)            # and its keys and values
    w = [1 + 0.2 * torch.randn(D, generator=gen, device=dev) for _ in range(4)]
    grad_out = [torch.randn(tq, HQ, D, generator=gen, device=dev).to(torch.bfloat16) for _ in range(2)]
    a = torch.arange(200, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device=dev).double() / D)
    table = torch.cat([a.cos(), a.sin()], 1).float()
    pos = torch.cat([torch.arange(n, device=dev) for n in q_len]).to(torch.int32)
    qo = torch.tensor([0, 50, 180, 187], dtype=torch.int32, device=dev)
    so = torch.tensor([0, 90, 123, 383], dtype=torch.int32, device=dev)

    # forward
    q, k = attn.attn_qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], w[0], w[1], eps=eps, cos_sin=table, positions=pos)
    v = qkv[:, HQ + HKV:]
    o1, lse1, _ = attn.attn_varlen_fwd(q, k, v, qo, qo, causal=True)
    cqn, _ = attn.attn_qk_norm_rope(cq, None, w[2], None, eps=eps)
    _, ckn = attn.attn_qk_norm_rope(None, ckv[:, :HKV], None, w[3], eps=eps)
    o2, lse2, _ = attn.attn_varlen_fwd(cqn, ckn, ckv[:, HKV:], qo, so)
    # backward, into the projections' gradients
    d_qkv, d_ckv = torch.empty_like(qkv), torch.empty_like(ckv)
    attn.attn_varlen_bwd(grad_out[0], q, k, v, o1, lse1, qo, qo, causal=True, d_q=d_qkv[:, :HQ], d_k=d_qkv[:, HQ:HQ + HKV],
                         d_v=d_qkv[:, HQ + HKV:])
    dw = list(attn.attn_qk_norm_rope_bwd(d_qkv[:, :HQ], d_qkv[:, HQ:HQ + HKV], qkv[:, :HQ], qkv[:, HQ:HQ + HKV], w[0], w[1],
                                         eps=eps, cos_sin=table, positions=pos, d_q=d_qkv[:, :HQ],
                                         d_k=d_qkv[:, HQ:HQ + HKV])[2:4])
    d_cq, _, _, _ = attn.attn_varlen_bwd(grad_out[1], cqn, ckn, ckv[:, HKV:], o2, lse2, qo, so, d_k=d_ckv[:, :HKV],
                                         d_v=d_ckv[:, HKV:])
    d_cq, _, dwq, _, _ = attn.attn_qk_norm_rope_bwd(d_cq, None, cq, None, w[2], None, eps=eps)
    _, _, _, dwk, _ = attn.attn_qk_norm_rope_bwd(None, d_ckv[:, :HKV], None, ckv[:, :HKV], None, w[3], eps=eps, d_k=d_ckv[:, :HKV])
    dw += [dwq, dwk]

    # the same in float64 by torch's own differentiation
    p = [t.double().requires_grad_() for t in (qkv, cq, ckv, *w)]
    y1 = _attended(_rotated(_normed(p[0][:, :HQ], p[3], eps), table, pos),
                   _rotated(_normed(p[0][:, HQ:HQ + HKV], p[4], eps), table, pos), p[0][:, HQ + HKV:], q_len, q_len, True)
    y2 = _attended(_normed(p[1], p[5], eps), _normed(p[2][:, :HKV], p[6], eps), p[2][:, HKV:], q_len, states, False)
    (y1 * grad_out[0].double()).sum().add((y2 * grad_out[1].double()).sum()).backward()
    # Norms over the whole tensor: each result has passed a handful of bf16 roundings (the normed rows, P or dS, the gradient
    # in between, itself), each at most 2^-8 of a value and independent from value to value.  Scores of size up to 8 turn the
    # normed rows' rounding into at most 2 * 2^-8 * 8 / sqrt(D) of each weight (independent over D products): six units of
    # 2^-8 bound the relative norm of every result.
    for name, got, want in [("o self", o1, y1), ("o cross", o2, y2), ("d qkv", d_qkv, p[0].grad), ("d cq", d_cq, p[1].grad),
                            ("d ckv", d_ckv, p[2].grad)] + [(f"dw{i}", x, y.grad) for i, (x, y) in enumerate(zip(dw, p[3:]))]:
        off = (got.double() - want.detach()).norm() / want.detach().norm()
        assert off <= 6 * 2.0 ** -8, (name, off.item())

    # a generated token of every sequence reads the states as the last position of a prompt would
    last = torch.tensor([49, 179, 186], device=dev)
    o3, lse3, _ = attn.attn_cross_decode(cqn[last], ckn, ckv[:, HKV:], so)
    x = ragged.Batch(dev, [1, 1, 1], states, HQ, HKV, D)
    x.q, x.k, x.v = cqn[last], ckn, ckv[:, HKV:]
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    ragged.check("o", o3, want_o, tol_o)
    ragged.check("lse", lse3, want_l, tol_l)
    assert (o3.double() - o2[last].double()).abs().max() <= 2 * tol_o.max()

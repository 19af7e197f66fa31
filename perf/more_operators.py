"""Measured cases of attention between sequences of two lengths, forward, backward and for single tokens, and of the norms
and rotation of its queries and keys.

Five operators of an attention layer, each from its definition in elementary torch operations (``own = False``) or through
the library's entry points (``own = True``):

  norm         RMS norm of every head of the queries and keys by a weight, then their rotation by the positions' angles
  norm_bwd     its gradient: to queries, keys and both weights
  attend       attention of a ragged batch over keys and values of other lengths: every key (cross attention to an encoder's
               states) or causal, aligned to the ends
  attend_bwd   its gradient: to queries, keys and values
  decode       1..16 queries per sequence (one token, the beams of a search) over an encoder's states

A case holds sizes; the lengths of its sequences follow from ``layout``, the values from the seed given to ``prepare``.
Keys of a sequence are its first ``len`` rows of ``[kv_indptr[b], kv_indptr[b + 1])``; with ``padded`` those are as many for
all, as a padded encoder batch leaves them.
"""

import math
import random

import torch

own = False


# --------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode loop
        dict(name="norm 1 token", op="norm", T=1, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, fused=True, far=700),
        # the queries and keys of a step's prompts, interleaved pairs, a part of the head rotated
        dict(name="norm prompts", op="norm", T=16384, Hq=32, Hkv=4, D=128, rot=64, interleaved=True, fused=False, far=4096),
        # a short odd batch of small heads
        dict(name="norm_bwd odd batch", op="norm_bwd", T=777, Hq=15, Hkv=3, D=64, rot=64, interleaved=False, fused=True,
             far=300),
        # a training batch of four sequences of 4096
        dict(name="norm_bwd training batch", op="norm_bwd", T=16384, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             fused=True, far=4096),
        # short texts attend to padded encoder states (frames of a recording), small heads without groups
        dict(name="attend texts to frames", op="attend", B=6, Hq=12, Hkv=12, D=64, q_lo=1, q_hi=77, kv_lo=200, kv_hi=1500,
             causal=False, padded=True, fused=True, layout=1),
        # long prompts attend to long encoder states
        dict(name="attend prompts to states", op="attend", B=4, Hq=32, Hkv=8, D=128, q_lo=2048, q_hi=2048, kv_lo=4096,
             kv_hi=4096, causal=False, padded=False, fused=True, layout=2),
        # the causal layer beside it: a ragged batch of documents
        dict(name="attend causal documents", op="attend", B=8, Hq=32, Hkv=4, D=128, q_lo=256, q_hi=4096, kv_lo=0, kv_hi=0,
             causal=True, padded=False, fused=True, layout=3),
        # a small odd batch, groups of five, padded, a sequence without keys
        dict(name="attend_bwd odd batch", op="attend_bwd", B=5, Hq=15, Hkv=3, D=64, q_lo=5, q_hi=300, kv_lo=0, kv_hi=700,
             causal=False, padded=True, fused=False, layout=4),
        # training of cross attention to long states
        dict(name="attend_bwd prompts to states", op="attend_bwd", B=4, Hq=32, Hkv=8, D=128, q_lo=2048, q_hi=2048, kv_lo=4096,
             kv_hi=4096, causal=False, padded=False, fused=True, layout=5),
        # training of the causal layer on documents of very different lengths
        dict(name="attend_bwd causal documents", op="attend_bwd", B=8, Hq=32, Hkv=8, D=128, q_lo=256, q_hi=4096, kv_lo=0,
             kv_hi=0, causal=True, padded=False, fused=True, layout=6),
        # one token of one sequence over an encoder's states: latency
        dict(name="decode 1 sequence", op="decode", B=1, Hq=32, Hkv=8, D=128, q_lo=1, q_hi=1, kv_lo=1500, kv_hi=1500,
             causal=False, padded=False, fused=True, layout=7),
        # four beams of each of 64 sequences over states of very different lengths
        dict(name="decode 64 x 4 beams", op="decode", B=64, Hq=32, Hkv=8, D=128, q_lo=4, q_hi=4, kv_lo=512, kv_hi=6400,
             causal=False, padded=True, fused=True, layout=8),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng, op):
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 12])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    while hkv * group > 32:
        group = rng.choice([1, 2])
    case = dict(op=op, Hq=hkv * group, Hkv=hkv, D=d, fused=rng.random() < 0.5)
    if op in ("norm", "norm_bwd"):
        case.update(T=_between(rng, 1, 16384), rot=rng.choice([0, 16, 32, 64, d]), interleaved=rng.random() < 0.5,
                    far=_between(rng, 2, 32768))
        return case
    case.update(causal=False, padded=rng.random() < 0.5, layout=rng.randrange(1 << 20))
    if op == "decode":
        n = rng.choice([1, 1, 1, 2, 4, 5, 8, 16])
        case.update(B=_between(rng, 1, 64), q_lo=n, q_hi=n, kv_lo=rng.choice([0, 1, 50]), kv_hi=_between(rng, 60, 8192))
        return case
    case.update(B=_between(rng, 1, 10), q_lo=1, q_hi=_between(rng, 2, 4096))
    if rng.random() < 0.45:
        # the sequences' own keys, sometimes behind a cached prefix (kv_lo .. kv_hi tokens more than queries)
        case.update(causal=True, kv_lo=0, kv_hi=rng.choice([0, 0, _between(rng, 2, 2048)]))
    else:
        case.update(kv_lo=rng.choice([0, 1, 50]), kv_hi=_between(rng, 60, 8192))
    return case


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "attend", "attend", "attend_bwd", "attend_bwd", "decode"])
    most = [work(c) for c in listed() if c["op"] == op]
    while True:
        case = _drawn(rng, op)
        need = work(case)
        if all(need[k] <= max(m[k] for m in most) for k in need):
            return case


def _lengths(case):
    """(queries, keys) of the sequences; a causal case's kv_lo .. kv_hi count its keys before the queries."""
    rng = random.Random(case["layout"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    kv = [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"])]
    if case["causal"]:
        kv = [a + b for a, b in zip(q, kv)]
    elif case["kv_lo"] == 0 and case["B"] > 1:
        kv[1] = 0   # a sequence whose states are all padding
    return q, kv


def work(case):
    hq, hkv, d = case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("norm", "norm_bwd"):
        n = case["T"] * (hq + hkv) * d
        table = min(case["T"], case["far"]) * case["rot"] * 4 + 4 * case["T"]
        turned = case["T"] * (hq + hkv) * case["rot"]
        if case["op"] == "norm":
            return {"bytes": 4 * n + table + 8 * d, "flops": 4 * n + 3 * turned}
        return {"bytes": 6 * n + table + 16 * d, "flops": 11 * n + 3 * turned}
    q, kv = _lengths(case)
    if case["causal"]:
        pairs = sum(max(0, m - n + i + 1) for n, m in zip(q, kv) for i in range(n))
    else:
        pairs = sum(n * m for n, m in zip(q, kv))
    rows, keys = sum(q) * hq, sum(kv) * hkv
    lists = 8 * case["B"] + 8
    if case["op"] != "attend_bwd":   # q, o, lse; k, v
        return {"bytes": rows * (4 * d + 4) + keys * 4 * d + lists, "flops": 4 * pairs * hq * d}
    # q, o, d_o, lse, d_q; k, v, d_k, d_v
    return {"bytes": rows * (8 * d + 4) + keys * 8 * d + lists, "flops": 10 * pairs * hq * d}


# ------------------------------------------------------------------------------------------------------- the inputs

def _heads(rows, heads, d, gen, dev, fused):
    """Normal bf16 [rows, h, d] for each h of `heads`: the parts of one projection's output, or tensors of their own."""
    if fused:
        x = torch.randn(rows, sum(heads) * d, generator=gen, device=dev).to(torch.bfloat16)
        return [p.view(rows, -1, d) for p in x.split([h * d for h in heads], dim=1)]
    return [torch.randn(rows, h, d, generator=gen, device=dev).to(torch.bfloat16) for h in heads]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d = case["Hq"], case["Hkv"], case["D"]
    s = dict(case=case)
    if case["op"] in ("norm", "norm_bwd"):
        t = case["T"]
        # heads of a projection differ in size; v is the part that the norm leaves alone
        s["q"], s["k"], _ = _heads(t, (hq, hkv, hkv), d, gen, dev, case["fused"])
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(d, generator=gen, device=dev) for _ in range(2))
        s["eps"], s["interleaved"] = 1e-6, case["interleaved"]
        start = int(torch.randint(0, case["far"], (1,), generator=gen, device=dev))
        s["positions"] = ((start + torch.arange(t, device=dev)) % case["far"]).to(torch.int32)
        s["cos_sin"] = None
        if case["rot"]:
            freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
            angle = torch.arange(case["far"], dtype=torch.float64, device=dev)[:, None] * freq
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        if case["op"] == "norm_bwd":
            s["dq"], s["dk"] = _heads(t, (hq, hkv), d, gen, dev, False)
        return s
    q, kv = _lengths(case)
    room = [max(kv)] * case["B"] if case["padded"] else kv
    total_q, total_kv = sum(q), sum(room)
    s["new"], s["lens"] = q, kv
    s["q_at"] = [sum(q[:b]) for b in range(case["B"])]
    s["kv_at"] = [sum(room[:b]) for b in range(case["B"])]
    s["qo_indptr"] = torch.tensor(s["q_at"] + [total_q], dtype=torch.int32, device=dev)
    s["kv_indptr"] = torch.tensor(s["kv_at"] + [total_kv], dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev) if case["padded"] else None
    if case["causal"] and total_q == total_kv:   # one projection makes all three
        s["q"], s["k"], s["v"] = _heads(total_q, (hq, hkv, hkv), d, gen, dev, case["fused"])
    else:
        s["q"], = _heads(total_q, (hq,), d, gen, dev, False)
        s["k"], s["v"] = _heads(total_kv, (hkv, hkv), d, gen, dev, case["fused"])
    s["scale"], s["causal"] = d ** -0.5, case["causal"]
    if case["op"] == "decode":
        s["q"] = s["q"].view(case["B"], case["q_hi"], hq, d)
    if case["op"] == "attend_bwd":
        s["o"], s["lse"] = _plain_attend(s)    # what the forward pass left
        s["do"], = _heads(total_q, (hq,), d, gen, dev, False)
    return s


# -------------------------------------------------------------------------------------------------------------- run

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_norm(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    return attn.attn_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], eps=s["eps"], cos_sin=s["cos_sin"],
                                  positions=s["positions"], interleaved=s["interleaved"])


def _own_norm_bwd(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    if "workspace" not in s:   # kept by the program from step to step
        need = attn.attn_qk_norm_rope_bwd_workspace_bytes(*s["q"].shape[:2], *s["k"].shape[1:])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    return attn.attn_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], eps=s["eps"], cos_sin=s["cos_sin"],
                                      positions=s["positions"], interleaved=s["interleaved"], workspace=s["workspace"])[:4]


def _own_attend(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    if "workspace" not in s:
        need = attn.attn_varlen_fwd_workspace_bytes(s["case"]["B"], s["q"].shape[0], s["k"].shape[0], s["q"].shape[1],
                                                    *s["k"].shape[1:])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["q"].device)
    o, lse, _ = attn.attn_varlen_fwd(s["q"], s["k"], s["v"], s["qo_indptr"], s["kv_indptr"], kv_lens=s["kv_lens"],
                                     causal=s["causal"], scale=s["scale"], workspace=s["workspace"])
    return o, lse


def _own_attend_bwd(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    if "workspace" not in s:
        need = attn.attn_varlen_bwd_workspace_bytes(s["case"]["B"], s["q"].shape[0], s["k"].shape[0], s["q"].shape[1],
                                                    *s["k"].shape[1:])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    return attn.attn_varlen_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["qo_indptr"], s["kv_indptr"],
                                kv_lens=s["kv_lens"], causal=s["causal"], scale=s["scale"], workspace=s["workspace"])[:3]


def _own_decode(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    if "workspace" not in s:
        need = attn.attn_cross_decode_workspace_bytes(*s["q"].shape[:3], *s["k"].shape[1:])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    o, lse, _ = attn.attn_cross_decode(s["q"], s["k"], s["v"], s["kv_indptr"], kv_lens=s["kv_lens"], scale=s["scale"],
                                       workspace=s["workspace"])
    return o, lse


_OWN = dict(norm=_own_norm, norm_bwd=_own_norm_bwd, attend=_own_attend, attend_bwd=_own_attend_bwd, decode=_own_decode)


def _turned(x, s, back):
    """x [T, H, D] with its first values turned by their positions' angles, or turned back."""
    if s["cos_sin"] is None:
        return x
    half = s["cos_sin"].shape[1] // 2
    c, n = (a[:, None, :] for a in s["cos_sin"][s["positions"].long()].split(half, dim=1))
    n = -n if back else n
    first, rest = x[..., :2 * half], x[..., 2 * half:]
    if s["interleaved"]:
        a, b = first[..., 0::2], first[..., 1::2]
        y = torch.stack([a * c - b * n, a * n + b * c], dim=-1).flatten(-2)
    else:
        a, b = first[..., :half], first[..., half:]
        y = torch.cat([a * c - b * n, a * n + b * c], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _plain_norm(s):
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.float()
        r = 1 / ((x * x).mean(dim=-1, keepdim=True) + s["eps"]).sqrt()
        out.append(_turned(x * r * w, s, False).to(torch.bfloat16))
    return tuple(out)


def _plain_norm_bwd(s):
    dx, dw = [], []
    for dy, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
        x, u = x.float(), _turned(dy.float(), s, True)
        r = 1 / ((x * x).mean(dim=-1, keepdim=True) + s["eps"]).sqrt()
        dw.append((u * x * r).sum(dim=(0, 1), dtype=torch.float64).float())
        g = u * w
        dx.append((r * (g - x * (r * r * (g * x).mean(dim=-1, keepdim=True)))).to(torch.bfloat16))
    return dx[0], dx[1], dw[0], dw[1]


def _scores(s, q, k, n, m):
    """Scaled scores [Hkv, G, n, m] of one sequence, those that its queries do not see at -inf."""
    hkv = k.shape[1]
    score = (q.view(n, hkv, -1, q.shape[-1]).permute(1, 2, 0, 3).reshape(hkv, -1, q.shape[-1])
             @ k.permute(1, 2, 0)).view(hkv, -1, n, m) * s["scale"]
    if s["causal"]:
        i, j = torch.arange(n, device=q.device)[:, None], torch.arange(m, device=q.device)
        score = score.masked_fill(j > i + (m - n), -math.inf)
    return score


def _sequences(s):
    q = s["q"].flatten(0, -3)
    for n, m, a, b in zip(s["new"], s["lens"], s["q_at"], s["kv_at"]):
        yield slice(a, a + n), slice(b, b + m), q[a:a + n].float(), s["k"][b:b + m].float(), s["v"][b:b + m].float()


def _plain_attend(s):
    o = torch.zeros_like(s["q"], memory_format=torch.contiguous_format)
    lse = torch.full(s["q"].shape[:-1], -math.inf, device=o.device)
    o_rows, lse_rows = o.view(-1, *o.shape[-2:]), lse.view(-1, o.shape[-2])
    for at, _, q, k, v in _sequences(s):
        n, m = q.shape[0], k.shape[0]
        if m == 0:
            continue
        score = _scores(s, q, k, n, m)
        top = score.amax(dim=-1, keepdim=True).clamp(min=-1e30)
        p = (score - top).exp()
        total = p.sum(dim=-1, keepdim=True)
        x = (p.flatten(1, 2) @ v.transpose(0, 1)).view(*p.shape[:3], -1) / total.clamp(min=1e-37)
        o_rows[at] = x.permute(2, 0, 1, 3).flatten(1, 2).to(o.dtype)
        lse_rows[at] = (top + total.log())[..., 0].permute(2, 0, 1).flatten(1)
    return o, lse


def _plain_attend_bwd(s):
    dq = torch.zeros_like(s["q"], memory_format=torch.contiguous_format)
    dk = torch.zeros_like(s["k"], memory_format=torch.contiguous_format)
    dv = torch.zeros_like(dk)
    for at, keys, q, k, v in _sequences(s):
        n, m, hkv = q.shape[0], k.shape[0], k.shape[1]
        if m == 0:
            continue

        def rows(x):   # [n, Hq, ...] as [Hkv, G * n, ...]
            x = x.view(n, hkv, -1, x.shape[-1]).permute(1, 2, 0, 3)
            return x.reshape(hkv, -1, x.shape[-1])

        do = s["do"][at].float()
        delta = rows((do * s["o"][at].float()).sum(dim=-1)[..., None])
        lse = rows(s["lse"][at][..., None].clamp(min=-1e30))
        p = (_scores(s, q, k, n, m).flatten(1, 2) - lse).exp()
        ds = p * (rows(do) @ v.permute(1, 2, 0) - delta) * s["scale"]
        dv[keys] = (p.transpose(1, 2) @ rows(do)).transpose(0, 1).to(dv.dtype)
        dk[keys] = (ds.transpose(1, 2) @ rows(q)).transpose(0, 1).to(dk.dtype)
        x = (ds @ k.transpose(0, 1)).view(hkv, -1, n, k.shape[-1])
        dq[at] = x.permute(2, 0, 1, 3).flatten(1, 2).to(dq.dtype)
    return dq, dk, dv


_PLAIN = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, attend=_plain_attend, attend_bwd=_plain_attend_bwd,
              decode=_plain_attend)


# ------------------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    return _EXACT[case["op"]](prepare(case, seed))


def _turn(z, s, sign):
    """The rotation as a product of complex numbers, in place on the float64 tensor z [T, H, D]."""
    if s["cos_sin"] is None:
        return z
    rot = s["cos_sin"].shape[1]
    row = s["cos_sin"].double()[s["positions"].long()]
    by = torch.complex(row[:, :rot // 2], sign * row[:, rot // 2:])[:, None, :]
    part = z[..., :rot]
    pairs = part.unflatten(-1, (rot // 2, 2)) if s["interleaved"] else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
    z[..., :rot] = (w if s["interleaved"] else w.transpose(-1, -2)).flatten(-2)
    return z


def _exact_norm(s):
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        out.append(_turn(x / torch.sqrt(size ** 2 / x.shape[-1] + s["eps"]) * w.double(), s, 1))
    return tuple(out)


def _exact_norm_bwd(s):
    """Through the unit vector n = x / rms: dL/dx = (I - n n^T / D) (w * u) / rms, dL/dw = sum n * u."""
    dx, dw = [], []
    for dy, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
        x = x.double()
        rms = torch.sqrt(torch.einsum("thd,thd->th", x, x) / x.shape[-1] + s["eps"])[..., None]
        n, u = x / rms, _turn(dy.double(), s, -1)
        dw.append(torch.einsum("thd,thd->d", n, u))
        along = torch.einsum("thd,thd,d->th", n, u, w.double())[..., None] / x.shape[-1]
        dx.append((u * w.double() - n * along) / rms)
    return dx[0], dx[1], dw[0], dw[1]


def _seen(s, n, m, device):
    if not s["causal"]:
        return torch.ones(n, m, dtype=torch.bool, device=device)
    return torch.ones(n, m, dtype=torch.bool, device=device).tril(m - n)


def _exact_attend(s):
    q = s["q"].flatten(0, -3)
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    group = q.shape[1] // s["k"].shape[1]
    for n, m, a, b in zip(s["new"], s["lens"], s["q_at"], s["kv_at"]):
        if m == 0:
            continue
        hidden = ~_seen(s, n, m, q.device)
        for h in range(q.shape[1]):
            k, v = s["k"][b:b + m, h // group].double(), s["v"][b:b + m, h // group].double()
            score = torch.einsum("id,td->it", q[a:a + n, h].double(), k) * s["scale"]
            score[hidden] = -math.inf
            lse[a:a + n, h] = torch.logsumexp(score, dim=-1)
            weight = torch.softmax(score, dim=-1)
            weight[hidden.all(dim=-1)] = 0
            o[a:a + n, h] = weight @ v
    return o.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def _exact_attend_bwd(s):
    q, do = s["q"], s["do"]
    dq = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device=q.device) for _ in range(2))
    group = q.shape[1] // s["k"].shape[1]
    for n, m, a, b in zip(s["new"], s["lens"], s["q_at"], s["kv_at"]):
        if m == 0:
            continue
        seen = _seen(s, n, m, q.device)
        for h in range(q.shape[1]):
            kh = h // group
            k, v = s["k"][b:b + m, kh].double(), s["v"][b:b + m, kh].double()
            x, g = q[a:a + n, h].double(), do[a:a + n, h].double()
            lse = s["lse"][a:a + n, h].double()[:, None]
            weight = torch.where(seen, torch.exp(torch.einsum("id,td->it", x, k) * s["scale"] - lse), 0.0)
            inner = torch.einsum("id,id->i", g, s["o"][a:a + n, h].double())[:, None]
            slope = weight * (torch.einsum("id,td->it", g, v) - inner)
            dq[a:a + n, h] = s["scale"] * (slope @ k)
            dk[b:b + m, kh] += s["scale"] * torch.einsum("it,id->td", slope, x)
            dv[b:b + m, kh] += torch.einsum("it,id->td", weight, g)
    return dq, dk, dv


_EXACT = dict(norm=_exact_norm, norm_bwd=_exact_norm_bwd, attend=_exact_attend, attend_bwd=_exact_attend_bwd,
              decode=_exact_attend)

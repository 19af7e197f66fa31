"""Measured cases of the paged KV cache's writer and of its 8-bit form's readers.

Four operators of a serving loop, each from its definition in elementary torch operations (``own = False``) or through
the library's entry points (``own = True``):

  append     rotates new queries and keys by their positions and writes the keys and values into a bf16 paged cache
  append8    the same into an e4m3 cache with one power-of-two scale per block of tokens and KV head
  decode8    causal attention of 1..16 queries per sequence over the 8-bit cache (single tokens, speculative decoding)
  prefill8   causal attention of a ragged batch of prompts over the 8-bit cache

A case holds sizes; the lengths of its sequences follow from ``layout``, the values and the order of the pages from the
seed given to ``prepare``.  Token t of a sequence lies in entry t // page of its page list.  The 8-bit cache holds
``code * scale``: codes ``[pages, page, Hkv, 128]`` e4m3, scales ``[pages, page / block, Hkv]`` float32.
"""

import math
import random

import torch

own = False

D = 128
E4M3_MAX = 448.0


# --------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one sequence: the smallest call of an interactive decode loop
        dict(name="append 1 token", op="append", B=1, Hq=32, Hkv=8, kv_lo=700, kv_hi=700, new_lo=1, new_hi=1, page=256,
             block=64, rot=128, interleaved=False, csr=False, fused=True, layout=1),
        # a decode step of a batch of 64
        dict(name="append decode batch", op="append", B=64, Hq=32, Hkv=8, kv_lo=1, kv_hi=2048, new_lo=1, new_hi=1, page=256,
             block=64, rot=128, interleaved=False, csr=False, fused=True, layout=2),
        # a ragged batch of prompts behind cached prefixes, page size 1, interleaved pairs, a part of the head rotated
        dict(name="append prompts", op="append", B=8, Hq=32, Hkv=4, kv_lo=1200, kv_hi=4096, new_lo=256, new_hi=2048, page=1,
             block=1, rot=64, interleaved=True, csr=True, fused=False, layout=3),
        # the decode step of a batch of 64 into the 8-bit cache: most tokens join a block that is partly filled
        dict(name="append8 decode batch", op="append8", B=64, Hq=32, Hkv=8, kv_lo=1, kv_hi=2048, new_lo=1, new_hi=1, page=256,
             block=64, rot=128, interleaved=False, csr=False, fused=True, layout=4),
        # short chunks of odd lengths that start and end inside blocks, few KV heads, small pages
        dict(name="append8 odd chunks", op="append8", B=13, Hq=15, Hkv=3, kv_lo=40, kv_hi=700, new_lo=1, new_hi=333, page=48,
             block=16, rot=64, interleaved=True, csr=True, fused=True, layout=5),
        # long prompts
        dict(name="append8 prompts", op="append8", B=8, Hq=32, Hkv=8, kv_lo=1024, kv_hi=4096, new_lo=1024, new_hi=4096,
             page=256, block=64, rot=128, interleaved=False, csr=False, fused=True, layout=6),
        # one sequence, one query: latency
        dict(name="decode8 1 sequence", op="decode8", B=1, Hq=32, Hkv=8, kv_lo=1000, kv_hi=1000, new_lo=1, new_hi=1, page=64,
             block=64, csr=False, layout=7),
        # speculative decoding, 4 queries per sequence, one of a model's two shards of KV heads, odd lengths, small blocks
        dict(name="decode8 4 queries", op="decode8", B=24, Hq=16, Hkv=2, kv_lo=3, kv_hi=9000, new_lo=4, new_hi=4, page=32,
             block=16, csr=True, layout=8),
        # 16 sequences of 16384 tokens
        dict(name="decode8 16 x 16384", op="decode8", B=16, Hq=32, Hkv=8, kv_lo=16384, kv_hi=16384, new_lo=1, new_hi=1,
             page=256, block=64, csr=False, layout=9),
        # 64 sequences of very different lengths
        dict(name="decode8 ragged batch", op="decode8", B=64, Hq=32, Hkv=8, kv_lo=512, kv_hi=32768, new_lo=1, new_hi=1,
             page=256, block=64, csr=False, layout=10),
        # three short prompts of odd lengths, a group of five heads
        dict(name="prefill8 short prompts", op="prefill8", B=3, Hq=15, Hkv=3, kv_lo=90, kv_hi=600, new_lo=40, new_hi=300,
             page=48, block=16, csr=True, layout=11),
        # the ragged prompts of a scheduler step, behind cached prefixes
        dict(name="prefill8 ragged batch", op="prefill8", B=8, Hq=32, Hkv=4, kv_lo=1200, kv_hi=4096, new_lo=256, new_hi=2048,
             page=64, block=64, csr=False, layout=12),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append8", "decode8", "decode8", "prefill8"])
    hkv = rng.choice([1, 2, 3, 4, 5, 6, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    while hkv * group > 32:
        group = rng.choice([1, 2, 3, 4])
    block = rng.choice([16, 32, 64, 128])
    page = block * rng.choice([1, 2, 3, 4])
    case = dict(op=op, Hq=hkv * group, Hkv=hkv, page=page, block=block, csr=rng.random() < 0.5, layout=rng.randrange(1 << 20))
    if op in ("append", "append8"):
        if rng.random() < 0.4:   # a decode step
            case.update(B=_between(rng, 1, 256), kv_lo=1, kv_hi=_between(rng, 2, 2048), new_lo=1, new_hi=1)
        else:                    # prompts
            hi = _between(rng, 2, 2048)
            case.update(B=_between(rng, 1, 8), kv_lo=1, kv_hi=hi + _between(rng, 1, 2048), new_lo=1, new_hi=hi)
        case.update(rot=rng.choice([0, 32, 64, 96, 128, 128]), interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
    elif op == "decode8":
        q_len = rng.choice([1, 1, 1, 2, 3, 4, 8, 16])
        batch = _between(rng, 1, 64)
        case.update(B=batch, kv_lo=rng.choice([0, 1, 20]), kv_hi=_between(rng, 30, 16384 if batch <= 32 else 8192),
                    new_lo=q_len, new_hi=q_len)
    else:
        hi = _between(rng, 2, 1500)
        case.update(B=_between(rng, 1, 8), kv_lo=1, kv_hi=hi + _between(rng, 1, 2048), new_lo=1, new_hi=hi)
    return case


def _lengths(case):
    """(lengths after the new tokens, new tokens) of the sequences."""
    rng = random.Random(case["layout"])
    lens = [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    if case["op"] != "decode8":
        lens = [max(n, 1) for n in lens]
        new = [min(a, n) for a, n in zip(new, lens)]
    return lens, new


def work(case):
    lens, new = _lengths(case)
    hq, hkv, total = case["Hq"], case["Hkv"], sum(new)
    lists = 4 * sum(-(-n // case["page"]) for n in lens) + 8 * case["B"]
    if case["op"] in ("append", "append8"):
        angles = len(set(t for n, m in zip(lens, new) for t in range(n - m, n))) * case["rot"] * 4
        read = total * (hq + 2 * hkv) * D * 2 + angles + lists
        if case["op"] == "append":
            written = total * (hq + 2 * hkv) * D * 2
        else:
            blocks = sum(-(-n // case["block"]) - (n - m) // case["block"] for n, m in zip(lens, new))
            written = total * (hq * 2 + 2 * hkv) * D + 2 * blocks * hkv * 4
        # two products and a sum for each rotated value, a product for each quantised one
        return {"bytes": read + written, "flops": total * ((hq + hkv) * case["rot"] * 3 + (case["op"] == "append8") * 2 * hkv * D)}
    seen = sum(max(0, n - m + i + 1) for n, m in zip(lens, new) for i in range(m))
    kv = sum(lens) * hkv * D * 2 + 2 * sum(-(-n // case["block"]) for n in lens) * hkv * 4
    return {"bytes": kv + total * hq * (D * 4 + 4) + lists, "flops": 4 * seen * hq * D}


# ------------------------------------------------------------------------------------------------------- the inputs

def _quantised_pool(pages, page, block, hkv, gen, dev):
    """Codes and scales of a pool filled with normal values whose size differs from head to head, block by block."""
    x = torch.randn(pages, page // block, block, hkv, D, generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn(hkv, 1, generator=gen, device=dev))
    top = x.abs().amax(dim=(2, 4))
    scale = _scale_of(top).float()
    x /= scale[:, :, None, :, None]
    return x.to(torch.float8_e4m3fn).view(pages, page, hkv, D), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lengths(case)
    page, batch, hq, hkv = case["page"], case["B"], case["Hq"], case["Hkv"]
    counts = [-(-n // page) for n in lens]
    n_pages = max(1, sum(counts))
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    s = dict(case=case, batch=batch, block=case["block"], seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             qo_indptr=torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32), kv_indptr=None)
    starts = torch.tensor([0] + counts, device=dev).cumsum(0)
    if case["csr"]:
        s["kv_indptr"] = starts.to(torch.int32)
        s["pages"] = order
    else:
        width = max(1, max(counts))
        at = starts[:-1, None] + torch.arange(width, device=dev)
        has = torch.arange(width, device=dev) < torch.tensor(counts, device=dev)[:, None]
        s["pages"] = torch.where(has, order[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
    total = sum(new)
    if case["op"] in ("append", "append8"):
        rot = case["rot"]
        if case["fused"]:   # the three parts of one projection's output
            qkv = torch.randn(total, (hq + 2 * hkv) * D, generator=gen, device=dev).to(torch.bfloat16)
            s["q"], s["k"], s["v"] = (x.view(total, -1, D) for x in qkv.split([hq * D, hkv * D, hkv * D], dim=1))
        else:
            s["q"], s["k"], s["v"] = (torch.randn(total, h, D, generator=gen, device=dev).to(torch.bfloat16)
                                      for h in (hq, hkv, hkv))
        s["cos_sin"] = None
        if rot:
            freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
            angle = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * freq
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        s["interleaved"] = case["interleaved"]
        s["q_out"] = torch.empty(total, hq, D, dtype=torch.bfloat16, device=dev)
        s["one_each"] = case["new_hi"] == 1
        if case["op"] == "append":
            s["k_cache"], s["v_cache"] = (torch.zeros(n_pages, page, hkv, D, dtype=torch.bfloat16, device=dev)
                                          for _ in range(2))
    if case["op"] != "append":
        s["k_cache"], s["k_scale"] = _quantised_pool(n_pages, page, case["block"], hkv, gen, dev)
        s["v_cache"], s["v_scale"] = _quantised_pool(n_pages, page, case["block"], hkv, gen, dev)
    if case["op"] == "decode8":
        q_len = case["new_hi"]
        s["q"] = torch.randn(batch, q_len, hq, D, generator=gen, device=dev).to(torch.bfloat16)
    elif case["op"] == "prefill8":
        s["q"] = torch.randn(total, hq, D, generator=gen, device=dev).to(torch.bfloat16)
        s["rows"] = sum(lens)   # what the scheduler knows of the step: its cached tokens
    s["longest"], s["most"] = max(lens), max(max(new), 1)
    return s


# -------------------------------------------------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_append(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    attn.attn_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["seq_lens"],
                        cos_sin=s["cos_sin"], qo_indptr=None if s["one_each"] else s["qo_indptr"], kv_indptr=s["kv_indptr"],
                        interleaved=s["interleaved"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_append8(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    attn.attn_kv_append_fp8_block(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                  s["pages"], s["seq_lens"], cos_sin=s["cos_sin"],
                                  qo_indptr=None if s["one_each"] else s["qo_indptr"], kv_indptr=s["kv_indptr"],
                                  interleaved=s["interleaved"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _own_decode8(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    if "workspace" not in s:   # kept by the program from step to step
        need = attn.attn_decode_fp8_block_workspace_bytes(*s["q"].shape[:3], s["k_cache"].shape[2])
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=s["q"].device)
    o, lse, _ = attn.attn_decode_paged_fp8_block(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                 s["pages"], s["seq_lens"], kv_indptr=s["kv_indptr"],
                                                 workspace=s["workspace"])
    return o, lse


def _own_prefill8(s):
    import causal_gqa_flashattention_attn_gb300 as attn
    if "workspace" not in s:   # kept by the program from step to step
        need = attn.attn_prefill_fp8_block_workspace_bytes(s["batch"], s["rows"], s["k_cache"].shape[2])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    o, lse, _ = attn.attn_prefill_paged_fp8_block(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                  s["qo_indptr"], s["pages"], s["seq_lens"], kv_indptr=s["kv_indptr"],
                                                  max_kv_rows=s["rows"], workspace=s["workspace"])
    return o, lse


_OWN = dict(append=_own_append, append8=_own_append8, decode8=_own_decode8, prefill8=_own_prefill8)


def _page_of(s, b, t):
    """The pool page of token t of sequence b (tensors of one shape)."""
    entry = t // s["case"]["page"]
    if s["kv_indptr"] is None:
        return s["pages"][b, entry].long()
    return s["pages"][s["kv_indptr"][b].long() + entry].long()


def _new_tokens(s):
    """Sequence and cache index of every new token."""
    counts = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(s["batch"], device=counts.device), counts, output_size=s["q"].shape[0])
    i = torch.arange(b.numel(), device=b.device) - s["qo_indptr"][b].long()
    return b, (s["seq_lens"].long() - counts)[b] + i


def _rotated(x, s, t, dtype):
    """x [T, H, D] with its first values turned by the angles of positions t, in `dtype`."""
    x = x.to(dtype)
    if s["cos_sin"] is None:
        return x
    half = s["cos_sin"].shape[1] // 2
    c, n = (a[:, None, :] for a in s["cos_sin"][t].to(dtype).split(half, dim=1))
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if s["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack([a * c - b * n, a * n + b * c], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        y = torch.cat([a * c - b * n, a * n + b * c], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _plain_append(s):
    b, t = _new_tokens(s)
    page, slot = _page_of(s, b, t), t % s["case"]["page"]
    s["q_out"].copy_(_rotated(s["q"], s, t, torch.float32))
    s["k_cache"][page, slot] = _rotated(s["k"], s, t, torch.float32).to(torch.bfloat16)
    s["v_cache"][page, slot] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _power(e):
    """2^e in 64 bits for whole e, made of its bits: pow and exp2 may be a last place off."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale_of(top):
    """The smallest power of two (2^-126 at least) that brings values of size `top` into e4m3's range; 0 for 0."""
    m, e = torch.frexp(top)
    return torch.where(top > 0, _power(torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)), 0.0)


def _codes_of(x):
    """The e4m3 code of each value, ties to even, in 64 bits: a value next to a border stays on its side of it."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp(min=-9))
    return ((x / step).round() * step).to(torch.float8_e4m3fn)


def _plain_append8(s):
    block, dev = s["block"], s["q"].device
    per_page = s["case"]["page"] // block
    b, t = _new_tokens(s)
    page, slot = _page_of(s, b, t), t % s["case"]["page"]
    s["q_out"].copy_(_rotated(s["q"], s, t, torch.float32))
    at = page * per_page + slot // block                       # the pool's block of each token
    # the tokens already in the blocks that the sequences' new tokens join
    first = s["seq_lens"].long() - (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    old_t = (first - first % block)[:, None] + torch.arange(block, device=dev)
    old_b, old_t = torch.nonzero(old_t < first[:, None])[:, 0], old_t[old_t < first[:, None]]
    old_page, old_slot = _page_of(s, old_b, old_t), old_t % s["case"]["page"]
    old_at = old_page * per_page + old_slot // block
    for x, cache, scale in ((_rotated(s["k"], s, t, torch.float64), s["k_cache"], s["k_scale"]),
                            (s["v"].double(), s["v_cache"], s["v_scale"])):
        flat = scale.view(-1, scale.shape[-1])
        top = torch.zeros_like(flat, dtype=torch.float64)
        top.index_reduce_(0, at, x.abs().amax(dim=-1), "amax")
        before = torch.zeros_like(flat)
        before[old_at] = flat[old_at]
        now = torch.maximum(_scale_of(top), before.double())
        kept = (cache[old_page, old_slot].double() * (before.double() / now.clamp(min=2.0 ** -140))[old_at][..., None])
        cache[old_page, old_slot] = _codes_of(kept)
        cache[page, slot] = _codes_of(x / now.clamp(min=2.0 ** -140)[at][..., None])
        flat[at] = now[at].float()
    return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _cached(s, codes, scales):
    """The values [B, Hkv, longest, D] that the sequences have in the cache; zeros behind their ends."""
    page, block = s["case"]["page"], s["block"]
    length = max(s["longest"], 1)
    b, t = torch.meshgrid(torch.arange(s["batch"], device=codes.device), torch.arange(length, device=codes.device), indexing="ij")
    has = t < s["seq_lens"][:, None]
    p = torch.where(has, _page_of(s, torch.where(has, b, 0), torch.where(has, t, 0)), 0).clamp(min=0)
    x = codes[p, t % page].float() * scales[p, (t % page) // block][..., None]
    return torch.where(has[..., None, None], x, 0.0).transpose(1, 2)


def _attended(s, q, new):
    """Attention of q [B, n, Hq, D] (rows behind new[b] hold anything) over the sequences: (O, LSE) with rows that see nothing
    at O = 0 and LSE = -inf."""
    batch, n, hq, _ = q.shape
    hkv = s["k_cache"].shape[2]
    k, v = _cached(s, s["k_cache"], s["k_scale"]), _cached(s, s["v_cache"], s["v_scale"])
    q = q.float().view(batch, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, D)
    score = (q @ k.transpose(2, 3)).view(batch, hkv, hq // hkv, n, -1) * D ** -0.5
    last = (s["seq_lens"] - new)[:, None] + torch.arange(n, device=q.device)            # the last token that a query sees
    seen = torch.arange(score.shape[-1], device=q.device) <= last[..., None]             # [B, n, L]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.view(batch, hkv, -1, p.shape[-1]) @ v).view(batch, hkv, -1, n, D) / total.clamp(min=1e-37)
    lse = (top + total.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, D).to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(batch, n, hq)


def _plain_decode8(s):
    return _attended(s, s["q"], torch.full_like(s["seq_lens"], s["q"].shape[1]))


def _plain_prefill8(s):
    new = s["qo_indptr"][1:] - s["qo_indptr"][:-1]
    i = torch.arange(s["most"], device=new.device)
    has = i < new[:, None]
    rows = torch.where(has, s["qo_indptr"][:-1, None] + i, 0)
    o, lse = _attended(s, s["q"][rows], new)
    return o[has], lse[has]


_PLAIN = dict(append=_plain_append, append8=_plain_append8, decode8=_plain_decode8, prefill8=_plain_prefill8)


# ------------------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lengths(case)
    lists = []
    for i, n in enumerate(lens):
        count = -(-n // case["page"])
        row = s["pages"][i, :count] if s["kv_indptr"] is None else s["pages"][int(s["kv_indptr"][i]):][:count]
        lists.append(row.long())
    return (_exact_append if case["op"] in ("append", "append8") else _exact_attention)(case, s, lens, new, lists)


def _exact_turn(x, table, positions, interleaved):
    out = x.double()
    if table is None:
        return out
    rot = table.shape[1]
    z = torch.complex(table[positions, :rot // 2].double(), table[positions, rot // 2:].double())[:, None, :]
    part = out[..., :rot]
    pairs = part.unflatten(-1, (rot // 2, 2)) if interleaved else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    out[..., :rot] = (w if interleaved else w.transpose(-1, -2)).flatten(-2)
    return out


def _exact_e4m3(y):
    """The nearest of e4m3's values, ties to the even one."""
    size = y.abs()
    borders = torch.tensor([2.0 ** i for i in range(-5, 10)], dtype=torch.float64, device=y.device)
    unit = borders[torch.searchsorted(borders, size, right=True)] / 16    # a value in [2^i, 2^(i+1)) has the unit 2^(i-3)
    return torch.sign(y) * torch.round(size / unit) * unit


def _exact_append(case, s, lens, new, lists):
    page, block = case["page"], case["block"]
    q_out = torch.empty(s["q_out"].shape, dtype=torch.float64, device=s["q"].device)
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    scales = [s["k_scale"].double(), s["v_scale"].double()] if case["op"] == "append8" else []
    row = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        t = torch.arange(n - m, n, device=q_out.device)
        own_rows = slice(row, row + m)
        row += m
        q_out[own_rows] = _exact_turn(s["q"][own_rows], s["cos_sin"], t, case["interleaved"])
        fresh = (_exact_turn(s["k"][own_rows], s["cos_sin"], t, case["interleaved"]), s["v"][own_rows].double())
        for which in range(2):
            x = fresh[which]
            if case["op"] == "append":
                caches[which][lists[i][t // page], t % page] = x
                continue
            for j in range((n - m) // block, (n - 1) // block + 1):
                lo, hi = max(j * block, n - m), min((j + 1) * block, n)
                p, slot = lists[i][j * block // page], j * block % page
                part = x[lo - (n - m):hi - (n - m)]
                top = part.abs().amax(dim=(0, 2)).cpu()
                need = torch.tensor([0.0 if v == 0 else 2.0 ** max(-126, math.ceil(math.log2(v / E4M3_MAX))) for v in top.tolist()],
                                    dtype=torch.float64, device=x.device)
                there = lo - j * block
                old = scales[which][p, slot // block] if there else torch.zeros_like(need)
                unit = torch.maximum(need, old)
                safe = torch.where(unit > 0, unit, 1.0)[:, None]
                cells = caches[which][p, slot:slot + block]
                cells[:there] = _exact_e4m3(cells[:there] * old[:, None] / safe)
                cells[there:there + hi - lo] = _exact_e4m3(part / safe)
                scales[which][p, slot // block] = unit
    return (q_out, *caches, *scales)


def _exact_attention(case, s, lens, new, lists):
    page, block, hkv, group = case["page"], case["block"], case["Hkv"], case["Hq"] // case["Hkv"]
    if work(case)["flops"] > 2e12:
        return None
    q = s["q"].flatten(0, -3)
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    row = 0
    for n, m, pages in zip(lens, new, lists):
        t = torch.arange(n, device=q.device)
        for h in range(hkv):
            if n == 0:
                continue
            at = (pages[t // page], t % page)
            k = s["k_cache"][at[0], at[1], h].double() * s["k_scale"][at[0], at[1] // block, h].double()[:, None]
            v = s["v_cache"][at[0], at[1], h].double() * s["v_scale"][at[0], at[1] // block, h].double()[:, None]
            for g in range(h * group, (h + 1) * group):
                score = torch.einsum("id,td->it", q[row:row + m, g].double(), k) / math.sqrt(D)
                score[t[None, :] > (n - m + torch.arange(m, device=q.device))[:, None]] = -math.inf
                lse[row:row + m, g] = torch.logsumexp(score, dim=-1)
                sees = lse[row:row + m, g] > -math.inf
                o[row:row + m, g] = torch.where(sees[:, None], torch.softmax(score, dim=-1).nan_to_num(0.0) @ v, 0.0)
        row += m
    return o.view(s["q"].shape), lse.view(s["q"].shape[:-1])

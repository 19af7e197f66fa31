"""A plain paged KV cache in numpy float64, bf16 or block-scaled e4m3: what the appends write and what attention over the
cache gives, with the error bounds of the GPU's roundings (test infrastructure)."""

import numpy as np
import torch

import oracle

E4M3 = np.array([oracle.fp8_e4m3_value(i) for i in range(256)], dtype=np.float64)
_POS = E4M3[:0x7F]   # codes 0 .. 0x7E: 0 .. 448, rising


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16)


def e4m3_code(y):
    """The code of each value: nearest, ties to the even code, beyond 448 the last one, NaN to 0x7F."""
    y = np.asarray(y, dtype=np.float64)
    size = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), 448.0)
    hi = np.searchsorted(_POS, size)            # _POS[hi - 1] < size <= _POS[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - size, size - _POS[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    code = np.where(take_hi, hi, lo).astype(np.uint8)
    code |= (np.signbit(y).astype(np.uint8) << 7)
    return np.where(np.isnan(y), np.uint8(0x7F), code)


def scale_of(x):
    """The scale of a block's finite values: smallest 2^e >= 2^-126 with max / 2^e <= 448."""
    x = np.abs(x[np.isfinite(x)])
    top = x.max() if x.size else 0.0
    if top == 0.0:
        return 0.0
    m, e = np.frexp(top)
    return float(np.ldexp(1.0, max(-126, int(e) - (9 if m <= 0.875 else 8))))


def rotate(x, table, positions, interleaved):
    """x [T, H, D] float64 with its first R values turned; table [max_pos, R] (cosines, sines) or None."""
    x = np.array(x, dtype=np.float64)
    if table is None or table.shape[1] == 0:
        return x
    rot = table.shape[1]
    c = table[positions, :rot // 2].astype(np.float64)[:, None, :]
    s = table[positions, rot // 2:].astype(np.float64)[:, None, :]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    with np.errstate(invalid="ignore"):
        out_a, out_b = a * c - b * s, a * s + b * c
    x[..., ia], x[..., ib] = out_a, out_b
    return x


def rotate_slack(x, table, positions, interleaved):
    """|a c| + |b s| of each rotated value (the size its fp32 rounding errors go by), 0 elsewhere."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    out = np.zeros_like(x)
    if table is None or table.shape[1] == 0:
        return out
    rot = table.shape[1]
    c, s = (np.abs(z.astype(np.float64))[:, None, :] for z in np.split(table[positions], 2, axis=1))
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c + b * s, a * s + b * c
    return out


def rope_table(max_pos, rot, base=10000.0):
    a = np.arange(max_pos)[:, None] / base ** (np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


class Lists:
    """Page lists of a batch whose sequences may grow to ``capacity`` tokens each: a shuffled pool with ``spare`` pages more,
    as a block table (entries past a sequence's pages are -1) or as a CSR list."""

    def __init__(self, capacity, page, rng, csr=False, spare=2):
        self.page, self.csr = page, csr
        counts = [-(-n // page) for n in capacity]
        self.num_pages = max(1, sum(counts) + spare)
        order = rng.permutation(self.num_pages).astype(np.int32)
        self.rows, at = [], 0
        for c in counts:
            self.rows.append(order[at:at + c])
            at += c
        self.spare = order[at:]

    def tensors(self, dev):
        """(block_table, kv_indptr or None) on ``dev``."""
        if self.csr:
            flat = np.concatenate(self.rows + [np.zeros(1, np.int32)])   # one entry more, never read
            ptr = np.cumsum([0] + [len(r) for r in self.rows]).astype(np.int32)
            return torch.from_numpy(flat).to(dev), torch.from_numpy(ptr).to(dev)
        width = max(1, max(len(r) for r in self.rows))
        table = np.full((len(self.rows), width), -1, dtype=np.int32)
        for b, r in enumerate(self.rows):
            table[b, :len(r)] = r
        return torch.from_numpy(table).to(dev), None


def append_blocks(codes, scales, lists, block, b, t0, x):
    """Write x [n, Hkv, D] (float64, finite or not) at tokens t0 .. of sequence b into codes / scales, in place."""
    page = lists.page
    n = x.shape[0]
    for j in range(t0 // block, (t0 + n - 1) // block + 1):
        lo, hi = max(j * block, t0), min((j + 1) * block, t0 + n)
        p, slot = lists.rows[b][j * block // page], j * block % page
        for h in range(x.shape[1]):
            part = x[lo - t0:hi - t0, h]
            now = scale_of(part)
            there = lo - j * block
            if there:
                old = float(scales[p, slot // block, h])
                m, e = np.frexp(old)
                before = 0.0 if old <= 0 else float(np.ldexp(1.0, int(e) - (1 if m == 0.5 else 0)))
                now = max(now, before)
                if now != old:
                    cells = codes[p, slot:slot + there, h]
                    codes[p, slot:slot + there, h] = e4m3_code(E4M3[cells] * (old / now if now else 0.0))
            scales[p, slot // block, h] = now
            with np.errstate(invalid="ignore"):
                codes[p, slot + there:slot + there + hi - lo, h] = e4m3_code(part / now if now else part * 0.0)


def cached(codes, scales, lists, block, b, n, skip=()):
    """The values [n', Hkv, D] of sequence b's first n tokens, without those on the list entries in ``skip``."""
    t = np.array([i for i in range(n) if i // lists.page not in skip], dtype=np.int64)
    if t.size == 0:
        return np.zeros((0,) + codes.shape[2:])
    p = np.asarray(lists.rows[b])[t // lists.page]
    return E4M3[codes[p, t % lists.page]] * scales[p, (t % lists.page) // block].astype(np.float64)[..., None]


def attend(q, k, v, scale=None, weight_step=2.0 ** -11, small=2.0 ** -25):
    """Causal (bottom-right) attention of q [n, Hq, D] over k, v [len, Hkv, D] in float64: (o, lse, o_tol, lse_tol).

    The tolerances count the GPU's roundings: a score is a sum of 128 exact products in fp32, so it is off by less than 2^-16
    of the sum of their sizes (128 additions of half a step 2^-24 each, twice over for the tensor cores' truncation), and by
    2^-20 of itself for the scale factors; q's elements below 2^-14 of the row's largest one are fp16 subnormals, off by 2^-25
    of it.  A weight is rounded by ``weight_step`` of itself, or, where 16 bits cannot hold it, by ``small`` of the largest
    weight times scale; O is rounded to bf16, 2^-8 of itself."""
    n, hq, d = q.shape
    length, hkv = k.shape[0], k.shape[1]
    g = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    o, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    o_tol, lse_tol = np.zeros((n, hq, d)), np.zeros((n, hq))
    seen = np.arange(length)[None, :] <= (length - n + np.arange(n))[:, None]
    for h in range(hq):
        kh, vh, qh = k[:, h // g], v[:, h // g], q[:, h]
        s = qh @ kh.T * scale
        ds = (2.0 ** -16 * (np.abs(qh) @ np.abs(kh).T) + 2.0 ** -25 * np.abs(qh).max(1, initial=0)[:, None] *
              np.abs(kh).sum(1)[None, :]) * abs(scale) + 2.0 ** -20 * np.abs(s)
        for i in range(n):
            at = seen[i]
            if not at.any():
                continue
            top = s[i, at].max()
            w = np.exp(s[i, at] - top)
            total = w.sum()
            lse[i, h] = top + np.log(total)
            o[i, h] = w @ vh[at] / total
            reach = w @ np.abs(vh[at]) / total
            off = ds[i, at].max()
            lse_tol[i, h] = off + 2.0 ** -18 * (1 + abs(lse[i, h]))
            vmax = (w[:, None] * np.abs(vh[at])).max() if at.any() else 0.0
            o_tol[i, h] = (2.0 ** -8 * np.abs(o[i, h]) + (weight_step + 2.0 ** -18 + 2 * off) * reach * (1 + 2 * off) +
                           at.sum() * small * 448 * vmax / total + 1e-30)
    return o, lse, o_tol, lse_tol


def check_attention(o, lse, ref, what=""):
    o_ref, lse_ref, o_tol, lse_tol = ref
    o, lse = o.detach().float().cpu().double().numpy(), lse.detach().cpu().double().numpy()
    assert o.shape == o_ref.shape and lse.shape == lse_ref.shape, (o.shape, o_ref.shape)
    dead = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), dead), f"{what}: -inf pattern"
    assert np.all(o[dead] == 0), f"{what}: rows that see nothing"
    assert np.all(np.isfinite(o)), f"{what}: non-finite O"
    over = np.abs(o - o_ref) - o_tol
    assert over.max(initial=-1) <= 0, f"{what}: O over its bound by {over.max():.3e} at {np.unravel_index(over.argmax(), o.shape)}"
    lo = np.where(dead, -1.0, np.abs(np.where(dead, 0, lse) - np.where(dead, 0, lse_ref)) - lse_tol)
    assert lo.max(initial=-1) <= 0, f"{what}: LSE over its bound by {lo.max():.3e}"

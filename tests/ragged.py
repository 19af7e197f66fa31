"""Ragged batches over contiguous keys for the tests: inputs, the attention and its gradient in float64 from their
definitions, and how far the library's outputs may be from them.

The bounds count every rounding: a bf16 value is off by at most 2^-8 of itself (BF), an fp32 sum of n terms by n 2^-23 of
the sum of their sizes (twice half a step each: the tensor core's order and alignment are its own), an exponential by 2^-20
of itself (the approximation, its argument's product with log2 e, the sum's own terms)."""

import math

import torch

BF, F32, EXP = 2.0 ** -8, 2.0 ** -23, 2.0 ** -20


class Batch:
    """Queries and keys of sequences, `room` key rows of which `kv` count (None: all), `lead` and `tail` rows of no sequence
    before and behind them."""

    def __init__(self, dev, q, kv, hq, hkv, d, room=None, causal=False, lead=0, tail=0, seed=0, fused=False, size=1.0,
                 padding=None, scale=None):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.q_len, self.kv_len, self.hq, self.hkv, self.d, self.causal = list(q), list(kv), hq, hkv, d, causal
        room = list(kv) if room is None else list(room)
        self.q_at = [lead + sum(q[:b]) for b in range(len(q) + 1)]
        self.kv_at = [lead + sum(room[:b]) for b in range(len(q) + 1)]
        self.total_q, self.total_kv = self.q_at[-1] + tail, self.kv_at[-1] + tail
        self.qo = torch.tensor(self.q_at, dtype=torch.int32, device=dev)
        self.kvp = torch.tensor(self.kv_at, dtype=torch.int32, device=dev)
        self.lens = torch.tensor(kv, dtype=torch.int32, device=dev) if room != list(kv) else None
        self.scale = d ** -0.5 if scale is None else scale

        def rows(n, heads):
            return (size * torch.randn(n, heads, d, generator=gen, device=dev)).to(torch.bfloat16)

        self.q = rows(self.total_q, hq)
        if fused:   # keys and values as parts of one projection's output
            both = rows(self.total_kv, 2 * hkv)
            self.k, self.v = both[:, :hkv], both[:, hkv:]
        else:
            self.k, self.v = rows(self.total_kv, hkv), rows(self.total_kv, hkv)
        self.do = rows(self.total_q, hq)
        if padding is not None:   # what lies in the key rows that do not count
            seen = torch.zeros(self.total_kv, dtype=torch.bool, device=dev)
            for b, n in enumerate(kv):
                seen[self.kv_at[b]:self.kv_at[b] + n] = True
            self.k[~seen] = padding
            self.v[~seen] = padding

    def args(self):
        return dict(qo_indptr=self.qo, kv_indptr=self.kvp, kv_lens=self.lens, causal=self.causal, scale=self.scale)

    def heads(self):
        """(query rows, head, key rows, KV head, hidden [n, m]) of every sequence and head."""
        for b, (n, m) in enumerate(zip(self.q_len, self.kv_len)):
            rows, keys = slice(self.q_at[b], self.q_at[b] + n), slice(self.kv_at[b], self.kv_at[b] + m)
            hidden = torch.zeros(n, m, dtype=torch.bool, device=self.q.device)
            if self.causal:
                hidden = ~torch.ones(n, m, dtype=torch.bool, device=self.q.device).tril(m - n)
            for h in range(self.hq):
                yield rows, h, keys, h // (self.hq // self.hkv), hidden

    def sequence_rows(self):
        """Which query rows and key rows belong to a sequence."""
        q = torch.zeros(self.total_q, dtype=torch.bool, device=self.q.device)
        kv = torch.zeros(self.total_kv, dtype=torch.bool, device=self.q.device)
        q[self.q_at[0]:self.q_at[-1]] = True
        kv[self.kv_at[0]:self.kv_at[-1]] = True
        return q, kv


def forward(x, q=None, k=None, v=None):
    """(o, lse, bound of o, bound of lse) in float64."""
    q, k, v = (a.double() if b is None else b for a, b in ((x.q, q), (x.k, k), (x.v, v)))
    o = torch.zeros(x.total_q, x.hq, x.d, dtype=torch.float64, device=q.device)
    lse = torch.full((x.total_q, x.hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    for rows, h, keys, kh, hidden in x.heads():
        if hidden.numel() == 0:
            continue
        s = (q[rows, h] @ k[keys, kh].T * x.scale).masked_fill(hidden, -math.inf)
        # error of a score: the sum of d products, and the products with scale and log2 e
        ds = (x.d * F32 * (q[rows, h].abs() @ k[keys, kh].abs().T) * abs(x.scale) + 4 * F32 * s.abs()).masked_fill(hidden, 0)
        ds = ds.amax(dim=-1)
        top = s.amax(dim=-1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(s - top)
        total = p.sum(dim=-1, keepdim=True)
        p = p / total.clamp(min=1e-300)
        o[rows, h] = p @ v[keys, kh]
        lse[rows, h] = (top + total.log())[:, 0]
        size = p @ v[keys, kh].abs()
        n = hidden.shape[1]
        tol_o[rows, h] = (BF + 2 * EXP + 2 * n * F32 + 2 * ds[:, None]) * size + BF * o[rows, h].abs()
        tol_l[rows, h] = ds + EXP + n * F32 + 4 * F32 * lse[rows, h].abs().nan_to_num(0, 0, 0)
    return o, lse, tol_o, tol_l


def backward(x, o, lse, do=None, d_lse=None):
    """((dq, dk, dv), their bounds) in float64 from what the forward pass left."""
    q, k, v, o, do = x.q.double(), x.k.double(), x.v.double(), o.double(), (x.do if do is None else do).double()
    grads = [torch.zeros(a.shape, dtype=torch.float64, device=q.device) for a in (q, k, v)]
    tols = [torch.zeros_like(a) for a in grads]
    dq, dk, dv = grads
    tq, tk, tv = tols
    for rows, h, keys, kh, hidden in x.heads():
        if hidden.numel() == 0:
            continue
        qh, kk, vv, g = q[rows, h], k[keys, kh], v[keys, kh], do[rows, h]
        l = lse[rows, h].double()[:, None]
        s = qh @ kk.T * x.scale
        p = torch.where(hidden | (l == -math.inf), 0.0, torch.exp(s - l))
        err = (x.d * F32 * (qh.abs() @ kk.abs().T) * abs(x.scale) + 8 * F32 * (s.abs() + l.abs().nan_to_num(0, 0, 0)) + EXP)
        delta = (g * o[rows, h]).sum(dim=-1, keepdim=True)
        t_delta = x.d * F32 * (g * o[rows, h]).abs().sum(dim=-1, keepdim=True)
        if d_lse is not None:
            delta = delta - d_lse[rows, h].double()[:, None]
            t_delta = t_delta + F32 * delta.abs()
        dp = g @ vv.T
        ds = p * (dp - delta)
        # dS: P's error, those of dP and delta, and its own rounding to bf16
        t_ds = ds.abs() * (err + BF + 4 * F32) + p * (x.d * F32 * (g.abs() @ vv.abs().T) + t_delta + 2 * F32 * (dp.abs() + delta.abs()))
        n, m = hidden.shape
        group = x.hq // x.hkv
        dq[rows, h] = x.scale * (ds @ kk)
        tq[rows, h] = abs(x.scale) * ((t_ds + m * F32 * ds.abs()) @ kk.abs())
        dk[keys, kh] += x.scale * (ds.T @ qh)
        tk[keys, kh] += abs(x.scale) * ((t_ds + n * group * F32 * ds.abs()).T @ qh.abs())
        dv[keys, kh] += p.T @ g
        tv[keys, kh] += (p * (err + BF + n * group * F32)).T @ g.abs()
    return grads, [t + BF * a.abs() for t, a in zip(tols, grads)]


def check(name, got, want, tol, rows=None):
    """Every element within its bound, infinities where they belong."""
    got = got.double()
    if rows is not None:
        got, want, tol = got[rows], want[rows], tol[rows]
    infinite = torch.isinf(want)
    assert torch.equal(torch.isinf(got), infinite), f"{name}: infinities differ"
    off = torch.where(infinite, 0.0, (got - want).abs() - tol)
    assert not torch.isnan(off).any(), f"{name}: NaN"
    assert off.numel() == 0 or off.max() <= 0, f"{name}: {off.max():.3e} beyond the bound (of {tol.flatten()[off.argmax()]:.3e})"

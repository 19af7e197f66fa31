"""Single tokens' attention to an encoder's states against float64: one query, beams, padded and ragged batches, sequences
without keys, pieces of long ones."""

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

# q_len, keys, Hq, Hkv, D, options
CASES = {
    "one key": (1, [1], 4, 2, 128, {}),
    "one sequence": (1, [1500], 32, 8, 128, dict(fused=True)),
    "tile edges": (1, [15, 16, 17, 31, 32, 33], 8, 2, 128, {}),
    "small heads, beams": (5, [100, 1, 64, 300], 6, 6, 64, dict(room=[300] * 4)),
    "no keys": (2, [0, 40, 0, 0, 900], 8, 2, 128, dict(room=[10, 40, 0, 7, 900])),
    "no keys at all": (1, [0, 0], 8, 2, 64, {}),
    "two groups of rows": (4, [700, 33], 24, 2, 128, {}),
    "16 queries": (16, [500, 20, 4], 20, 4, 64, dict(fused=True)),
    "16 queries of 32 heads over 1": (16, [260], 32, 1, 128, {}),
    "group of 7": (1, [2000, 3, 90], 28, 4, 128, {}),
    "uneven batch": (1, [8000, 1, 16, 4097, 0, 250], 8, 2, 128, dict(room=[8000, 8000, 16, 5000, 8, 300])),
    "many short": (1, [(i * 13) % 90 for i in range(300)], 4, 4, 64, {}),
    "rows of no sequence": (3, [60, 200], 8, 4, 128, dict(lead=11, tail=30)),
    "large scores": (1, [900, 100], 8, 2, 128, dict(size=4.0)),
    "negative scale": (2, [300], 8, 2, 64, dict(scale=-0.2)),
}


def _batch(dev, name, **more):
    nq, kv, hq, hkv, d, options = CASES[name]
    options = {**options, **more}
    lead, tail = options.pop("lead", 0), options.pop("tail", 0)
    x = ragged.Batch(dev, [nq] * len(kv), kv, hq, hkv, d, seed=len(name), lead=lead, tail=tail, **options)
    q = x.q[lead:lead + nq * len(kv)].view(len(kv), nq, hq, d)
    return x, q


@pytest.mark.parametrize("name", CASES)
def test_decode(name):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x, q = _batch(dev, name, padding=float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse, ws = attn.attn_cross_decode(q, x.k, x.v, x.kvp, kv_lens=x.lens, scale=x.scale, dev_status=status)
    assert status.item() == 0
    clean, _ = _batch(dev, name)
    want_o, want_l, tol_o, tol_l = ragged.forward(clean)
    rows, _ = x.sequence_rows()
    ragged.check("o", o.view(-1, x.hq, x.d), want_o[rows], tol_o[rows])
    ragged.check("lse", lse.view(-1, x.hq), want_l[rows], tol_l[rows])
    if q.shape[1] == 1:
        o3, lse3, _ = attn.attn_cross_decode(q[:, 0], x.k, x.v, x.kvp, kv_lens=x.lens, scale=x.scale, workspace=ws)
        assert torch.equal(o3, o[:, 0]) and torch.equal(lse3, lse[:, 0])


def test_replay_with_other_lengths_and_streams():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [2] * 4, [900, 3, 40, 0], 8, 2, 128, room=[1000] * 4, seed=3)
    y = ragged.Batch(dev, [2] * 4, [0, 1000, 999, 17], 8, 2, 128, room=[1000] * 4, seed=4)
    q = x.q.view(4, 2, 8, 128)
    ws = torch.empty(attn.attn_cross_decode_workspace_bytes(4, 2, 8, 2), dtype=torch.uint8, device=dev)
    o, lse = torch.empty_like(q), torch.empty(4, 2, 8, device=dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    attn.attn_cross_decode(q, x.k, x.v, x.kvp, kv_lens=x.lens, workspace=ws, o=o, lse=lse, stream=side)
    side.synchronize()
    eager = o.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        attn.attn_cross_decode(q, x.k, x.v, x.kvp, kv_lens=x.lens, workspace=ws, o=o, lse=lse, stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])
    for a, b in ((x.q, y.q), (x.k, y.k), (x.v, y.v), (x.lens, y.lens)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want_o, want_l, tol_o, tol_l = ragged.forward(y)
    ragged.check("o", o.view(-1, 8, 128), want_o, tol_o)
    ragged.check("lse", lse.view(-1, 8), want_l, tol_l)


def test_two_streams_and_the_largest_batch():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    xs = [ragged.Batch(dev, [1], [3000 + 500 * i], 8, 2, 128, seed=i) for i in range(2)]
    alone = [attn.attn_cross_decode(x.q, x.k, x.v, x.kvp)[:2] for x in xs]
    streams = [torch.cuda.Stream(dev) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [attn.attn_cross_decode(x.q, x.k, x.v, x.kvp, stream=s)[:2] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    lens = [(i * 37) % 23 for i in range(4096)]
    x = ragged.Batch(dev, [1] * 4096, lens, 2, 1, 64, seed=5)
    o, lse, _ = attn.attn_cross_decode(x.q, x.k, x.v, x.kvp)
    # every sequence in one padded tensor
    at = torch.tensor(x.kv_at[:-1], device=dev)[:, None] + torch.arange(23, device=dev)
    there = torch.arange(23, device=dev) < torch.tensor(lens, device=dev)[:, None]
    k, v = (torch.where(there[..., None], t[:, 0].double()[at.clamp(max=x.total_kv - 1)], 0.0) for t in (x.k, x.v))
    s = (x.q.double() @ k.transpose(1, 2) * x.scale).masked_fill(~there[:, None], -float("inf"))
    want = torch.softmax(s, dim=-1).nan_to_num(0.0) @ v
    # 2^-8 of every weight and of the result, as the other cases' bounds, with |v| below 6
    assert (o.double() - want).abs().max() <= 2 * ragged.BF * 6
    ragged.check("lse", lse, torch.logsumexp(s, dim=-1), torch.full_like(lse, 1e-4, dtype=torch.float64))


def test_rows_past_32_bits():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [1, 1], [32600, 400], 4, 1, 128, seed=13)
    k, v = (torch.empty(33000, 1 << 16, dtype=torch.bfloat16, device=dev)[:, :128].view(33000, 1, 128) for _ in range(2))
    k.copy_(x.k)
    v.copy_(x.v)
    o, lse, _ = attn.attn_cross_decode(x.q, k, v, x.kvp)
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    ragged.check("o", o, want_o, tol_o)
    ragged.check("lse", lse, want_l, tol_l)


def test_refusals_and_offsets_outside():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [1, 1], [40, 60], 4, 2, 128)
    o, lse, _ = attn.attn_cross_decode(x.q, x.k, x.v, x.kvp)
    wide = torch.tensor([-9, 40, 1 << 30], dtype=torch.int32, device=dev)
    lens = torch.tensor([1 << 30, 60], dtype=torch.int32, device=dev)
    o2, lse2, _ = attn.attn_cross_decode(x.q, x.k, x.v, wide, kv_lens=lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for bad in (dict(q=x.q.float()), dict(q=x.q[0]), dict(k=x.k[:50]), dict(v=x.v.transpose(0, 1)), dict(kv_indptr=x.kvp[:2]),
                dict(kv_indptr=x.kvp.long()), dict(kv_lens=x.kvp), dict(q=x.q[:, :, :64]), dict(lse=lse[:1])):
        with pytest.raises(ValueError):
            attn.attn_cross_decode(**{**dict(q=x.q, k=x.k, v=x.v, kv_indptr=x.kvp), **bad})
    for q in (torch.empty(2, 17, 4, 128, dtype=torch.bfloat16, device=dev), torch.empty(2, 3, 128, dtype=torch.bfloat16, device=dev)):
        with pytest.raises(attn.AttnError):
            attn.attn_cross_decode(q, x.k, x.v, x.kvp)
    with pytest.raises(attn.AttnError) as e:
        attn.attn_cross_decode(x.q, x.k, x.v, x.kvp, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    assert e.value.status == -3

"""Attention of ragged batches to contiguous keys and its gradient against float64: all keys (cross attention) and causal,
padded batches, sequences without keys or queries, groups that do not divide a tile, strides, rows of no sequence."""

import pytest
import torch

import ragged
from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

# queries, keys, Hq, Hkv, D, options
CASES = {
    "one token": ([1], [1], 4, 2, 128, {}),
    "one token, causal": ([1], [1], 4, 2, 128, dict(causal=True)),
    "tile edges": ([127, 128, 129], [128, 129, 127], 4, 4, 128, {}),
    "tile edges, causal": ([127, 128, 129], [128, 129, 127], 4, 4, 128, dict(causal=True)),
    "small heads": ([77, 1, 33], [300, 150, 1], 6, 6, 64, dict(room=[300, 300, 300])),
    "small heads, causal": ([77, 300, 33], [77, 300, 95], 4, 2, 64, dict(causal=True)),
    "no keys, no queries": ([5, 0, 40, 0], [0, 17, 200, 0], 8, 2, 128, dict(room=[64, 64, 200, 0])),
    "no keys at all": ([5, 9], [0, 0], 8, 2, 128, {}),
    "no keys, padded": ([5, 9], [0, 0], 8, 2, 128, dict(room=[3, 140])),
    "rows that see nothing, causal": ([300, 64], [120, 10], 8, 2, 128, dict(causal=True)),
    "group of 5": ([100, 26, 51], [260, 128, 77], 15, 3, 128, dict(fused=True)),
    "group of 7, causal": ([100, 18, 37], [260, 18, 300], 14, 2, 64, dict(causal=True, fused=True)),
    "group of 32": ([50, 3], [200, 90], 32, 1, 128, {}),
    "group of 128": ([9], [150], 128, 1, 64, {}),
    "group of 100, causal": ([9], [150], 100, 1, 128, dict(causal=True)),
    "many short": ([i % 9 for i in range(70)], [(i * 7) % 40 for i in range(70)], 4, 1, 128, {}),
    # several items a CTA, of one tile and of two
    "many items": ([37 * i % 400 for i in range(48)], [91 * i % 700 for i in range(48)], 16, 8, 64, {}),
    "many items, causal": ([37 * i % 400 for i in range(40)], [37 * i % 400 for i in range(40)], 12, 12, 128, dict(causal=True)),
    "long keys, few queries": ([3, 20], [4000, 2500], 8, 2, 128, dict(room=[4000, 4000])),
    "long keys, few queries, causal": ([64], [3000], 4, 2, 64, dict(causal=True)),
    "long queries, few keys": ([3000], [70], 4, 2, 128, {}),
    "rows of no sequence": ([40, 130], [150, 90], 8, 4, 128, dict(lead=7, tail=140, room=[200, 90])),
    "rows of no sequence, parts": ([4], [1500], 8, 4, 128, dict(lead=3, tail=9)),
    "large scores": ([90], [500], 4, 2, 128, dict(size=4.0)),
    "odd scale, causal": ([90], [500], 4, 2, 64, dict(causal=True, scale=0.37)),
}


def _batch(dev, name, **more):
    q, kv, hq, hkv, d, options = CASES[name]
    return ragged.Batch(dev, q, kv, hq, hkv, d, seed=len(name), **{**options, **more})


def _forward(attn, x, **more):
    status = torch.zeros(1, dtype=torch.int32, device=x.q.device)
    o = torch.full((x.total_q, x.hq, x.d), 7.0, dtype=torch.bfloat16, device=x.q.device)
    lse = torch.full((x.total_q, x.hq), 7.0, device=x.q.device)
    attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args(), o=o, lse=lse, dev_status=status, **more)
    assert status.item() == 0
    return o, lse


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = _batch(dev, name, padding=float("nan"))
    o, lse = _forward(attn, x)
    want_o, want_l, tol_o, tol_l = ragged.forward(_batch(dev, name))
    of_seq, _ = x.sequence_rows()
    ragged.check("o", o, want_o, tol_o, of_seq)
    ragged.check("lse", lse, want_l, tol_l, of_seq)
    assert (o[~of_seq] == 7).all() and (lse[~of_seq] == 7).all()   # rows of no sequence are left alone


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = _batch(dev, name, padding=float("nan"))
    o, lse = _forward(attn, x)
    of_q, of_kv = x.sequence_rows()
    out = [torch.full_like(a, 7.0, memory_format=torch.contiguous_format) for a in (x.q, x.k, x.v)]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), d_q=out[0], d_k=out[1], d_v=out[2], dev_status=status)
    assert status.item() == 0
    want, tol = ragged.backward(_batch(dev, name), o, lse)
    for label, got, w, t, rows in zip(("dq", "dk", "dv"), out, want, tol, (of_q, of_kv, of_kv)):
        ragged.check(label, got, w, t, rows)
        assert (got[~rows] == 7).all()


def test_gradient_of_the_lse_and_strided_outputs():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [60, 130], [60, 130], 8, 2, 128, causal=True, seed=3)
    qkv = torch.cat([x.q, x.k, x.v], dim=1)   # one projection's output and its gradient
    x.q, x.k, x.v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())
    d_lse = torch.randn(190, 8, device=dev)
    grad = torch.empty_like(qkv)
    attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), d_lse=d_lse, d_q=grad[:, :8], d_k=grad[:, 8:10], d_v=grad[:, 10:])
    want, tol = ragged.backward(x, o, lse, d_lse=d_lse)
    for label, got, w, t in zip(("dq", "dk", "dv"), (grad[:, :8], grad[:, 8:10], grad[:, 10:]), want, tol):
        ragged.check(label, got, w, t)


@pytest.mark.parametrize("causal", [False, True])
def test_gradient_against_differences(causal):
    """sum(do * o) between two points of the float64 forward pass, along a random direction, against the gradient's product
    with it: the difference's own error (third derivatives) at h = 1e-4 is about 1e-8 of it."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [70, 9], [200, 40], 6, 2, 64, causal=causal, seed=5)
    o64, lse64, _, _ = ragged.forward(x)
    # the gradient at the exact point: o and lse in the precision the forward pass leaves them in
    o, lse = o64.to(torch.bfloat16), lse64.float()
    grads = attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args())[:3]
    _, tols = ragged.backward(x, o, lse)
    gen = torch.Generator(device=dev).manual_seed(1)
    for i, (g, t) in enumerate(zip(grads, tols)):
        along = torch.randn(g.shape, generator=gen, device=dev, dtype=torch.float64)
        moved = []
        for h in (1e-4, -1e-4):
            point = [a.double() for a in (x.q, x.k, x.v)]
            point[i] = point[i] + h * along
            moved.append((ragged.forward(x, *point)[0] * x.do.double()).sum())
        slope = (moved[0] - moved[1]) / 2e-4
        # o in bf16 moves delta by 2^-8 of each of its terms: dS by P times that, into dq and dk
        slack = 0.0
        if i < 2:
            for rows, h, keys, kh, hidden in x.heads():
                p = torch.where(hidden, 0.0, torch.exp(x.q[rows, h].double() @ x.k[keys, kh].double().T * x.scale - lse64[rows, h][:, None]))
                d = ragged.BF * (x.do[rows, h].double() * o64[rows, h]).abs().sum(dim=-1, keepdim=True)
                if i == 0:
                    slack += (x.scale * (p * d) @ x.k[keys, kh].double().abs() * along[rows, h].abs()).sum()
                else:
                    slack += (x.scale * (p * d).T @ x.q[rows, h].double().abs() * along[keys, kh].abs()).sum()
        assert (slope - (g.double() * along).sum()).abs() <= (t * along.abs()).sum() + slack + 1e-6 * slope.abs()


def test_results_do_not_depend_on_timing_or_stream():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [200, 3, 64], [700, 900, 50], 8, 2, 128, seed=9)
    first = None
    side = torch.cuda.Stream(dev)
    for stream in (None, side, None, side):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args(), stream=stream)
        out = (o, lse, *attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), stream=stream)[:3])
        torch.cuda.synchronize()
        if first is None:
            first = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_two_calls_at_once():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    xs = [ragged.Batch(dev, [30], [2000 + 100 * i], 8, 2, 128, seed=i) for i in range(2)]
    alone = []
    for x in xs:
        o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())
        alone.append((o, lse, *attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args())[:3]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in xs]
    got = [None, None]
    for _ in range(20):
        for i, (x, s) in enumerate(zip(xs, streams)):
            o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args(), stream=s)
            got[i] = (o, lse, *attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), stream=s)[:3])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_replay_from_a_graph_with_other_lengths():
    """The capture knows the totals; the offsets and lengths are read when it runs."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [100, 60], [400, 200], 8, 2, 128, room=[400, 400], seed=11)
    y = ragged.Batch(dev, [7, 153], [1, 399], 8, 2, 128, room=[400, 400], seed=12)
    ws = torch.empty(max(16, attn.attn_varlen_fwd_workspace_bytes(2, 160, 800, 8, 2)), dtype=torch.uint8, device=dev)
    bws = torch.empty(attn.attn_varlen_bwd_workspace_bytes(2, 160, 800, 8, 2), dtype=torch.uint8, device=dev)
    o, lse = torch.empty_like(x.q), torch.empty(160, 8, device=dev)
    grads = [torch.empty_like(t) for t in (x.q, x.k, x.v)]

    def step(stream):
        attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args(), workspace=ws, o=o, lse=lse, stream=stream)
        attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args(), workspace=bws, d_q=grads[0], d_k=grads[1], d_v=grads[2],
                             stream=stream)

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for a, b in ((x.q, y.q), (x.k, y.k), (x.v, y.v), (x.do, y.do), (x.qo, y.qo), (x.kvp, y.kvp), (x.lens, y.lens)):
        a.copy_(b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    want_o, want_l, tol_o, tol_l = ragged.forward(y)
    ragged.check("o", o, want_o, tol_o)
    ragged.check("lse", lse, want_l, tol_l)
    want, tol = ragged.backward(y, o, lse)
    for label, got, w, t in zip(("dq", "dk", "dv"), grads, want, tol):
        ragged.check(label, got, w, t)


def test_rows_past_32_bits():
    """Key rows 64 KB apart: the last ones lie more than 2^31 elements behind the first."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    stride, n = 1 << 16, 33000
    x = ragged.Batch(dev, [20, 50], [32600, 400], 4, 1, 128, seed=13, causal=True)
    assert x.total_kv == n
    k, v, q = (torch.empty(rows, stride, dtype=torch.bfloat16, device=dev)[:, :heads * 128].view(rows, heads, 128)
               for rows, heads in ((n, 1), (n, 1), (70, 4)))
    for a, b in ((k, x.k), (v, x.v), (q, x.q)):
        a.copy_(b)
    grads = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=dev) for t in (q, k, v)]
    o, lse, _ = attn.attn_varlen_fwd(q, k, v, **x.args())
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    ragged.check("o", o, want_o, tol_o)
    ragged.check("lse", lse, want_l, tol_l)
    attn.attn_varlen_bwd(x.do, q, k, v, o, lse, **x.args(), d_q=grads[0], d_k=grads[1], d_v=grads[2])
    want, tol = ragged.backward(x, o, lse)
    for label, got, w, t in zip(("dq", "dk", "dv"), grads, want, tol):
        ragged.check(label, got, w, t)


@pytest.mark.parametrize("d, group, causal", [(128, 4, False), (64, 3, True), (128, 5, True)])
def test_a_sequence_of_nan_stays_alone(d, group, causal):
    """Tiles hold rows of the sequences beside their own: what lies there reaches no output and no gradient."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    q, kv = [70, 45, 150, 3], [70, 130, 90, 33]
    x, y = (ragged.Batch(dev, q, kv, 2 * group, 2, d, causal=causal, lead=4, tail=30, seed=21) for _ in range(2))
    of_q, of_kv = x.sequence_rows()
    of_q[x.q_at[1]:x.q_at[2]] = False
    of_kv[x.kv_at[1]:x.kv_at[2]] = False
    for t, rows in ((x.q, of_q), (x.do, of_q), (x.k, of_kv), (x.v, of_kv)):
        t[~rows] = float("nan")
    o, lse = _forward(attn, x)
    want_o, want_l, tol_o, tol_l = ragged.forward(y)
    ragged.check("o", o, want_o, tol_o, of_q)
    ragged.check("lse", lse, want_l, tol_l, of_q)
    out = attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args())
    o = torch.where(of_q[:, None, None], o, want_o.to(o.dtype))
    lse = torch.where(of_q[:, None], lse, want_l.to(lse.dtype))
    want, tol = ragged.backward(y, o, lse)
    for label, got, w, t, rows in zip(("dq", "dk", "dv"), out, want, tol, (of_q, of_kv, of_kv)):
        ragged.check(label, got, w, t, rows)


def test_the_most_sequences():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    q, kv = [i % 4 for i in range(2048)], [i * 5 % 7 for i in range(2048)]
    x = ragged.Batch(dev, q, kv, 2, 1, 64, seed=22)
    o, lse = _forward(attn, x)
    want_o, want_l, tol_o, tol_l = ragged.forward(x)
    ragged.check("o", o, want_o, tol_o)
    ragged.check("lse", lse, want_l, tol_l)
    want, tol = ragged.backward(x, o, lse)
    for label, got, w, t in zip(("dq", "dk", "dv"), attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **x.args()), want, tol):
        ragged.check(label, got, w, t)


def test_offsets_outside_the_tensors_are_cut():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [40, 60], [100, 50], 4, 2, 128, seed=15)
    args = x.args()
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **args)
    grads = attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **args)[:3]
    args.update(qo_indptr=torch.tensor([-5, 40, 1000], dtype=torch.int32, device=dev),
                kv_indptr=torch.tensor([-1, 100, 1 << 30], dtype=torch.int32, device=dev),
                kv_lens=torch.tensor([1 << 30, 50], dtype=torch.int32, device=dev))
    o2, lse2, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(grads, attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **args)[:3]):
        assert torch.equal(a, b)
    # lengths below 0 are none; offsets that fall give sequences without rows, and those that overlap stay inside
    args.update(qo_indptr=torch.tensor([100, 0, 100], dtype=torch.int32, device=dev),
                kv_indptr=torch.tensor([0, 150, 0], dtype=torch.int32, device=dev),
                kv_lens=torch.tensor([-3, 10], dtype=torch.int32, device=dev))
    o2, lse2, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **args)
    assert (o2 == 0).all() and torch.isinf(lse2).all()
    attn.attn_varlen_bwd(x.do, x.q, x.k, x.v, o, lse, **args)
    torch.cuda.synchronize()


def test_refusals():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x = ragged.Batch(dev, [40], [100], 4, 2, 128)
    o, lse, _ = attn.attn_varlen_fwd(x.q, x.k, x.v, **x.args())

    def bwd(**kw):
        a = dict(d_o=x.do, q=x.q, k=x.k, v=x.v, o=o, lse=lse, **x.args())
        a.update(kw)
        return attn.attn_varlen_bwd(**a)

    for bad in (dict(q=x.q.float()), dict(k=x.k[:, :, :64]), dict(v=x.v[:50]), dict(d_o=x.do[:, :2]), dict(lse=lse[:, :2]),
                dict(lse=lse.double()), dict(qo_indptr=x.qo.long()), dict(kv_indptr=x.kvp[:1]), dict(kv_lens=x.qo),
                dict(d_lse=lse[:5]), dict(d_q=torch.empty_like(x.k)), dict(q=x.q.transpose(0, 1)), dict(o=o.cpu())):
        with pytest.raises(ValueError):
            bwd(**bad)
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(attn.AttnError):
            bwd(scale=scale)
        with pytest.raises(attn.AttnError):
            attn.attn_varlen_fwd(x.q, x.k, x.v, **{**x.args(), "scale": scale})
    with pytest.raises(attn.AttnError) as e:
        bwd(workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    assert e.value.status == -3
    odd = torch.empty(100 * 4 * 128 + 4, dtype=torch.bfloat16, device=dev)[4:].view(100, 4, 128)[:, :2]   # 8-byte aligned
    with pytest.raises(attn.AttnError):
        bwd(k=odd)
    assert attn.attn_varlen_fwd(x.q[:0], x.k, x.v, torch.zeros(2, dtype=torch.int32, device=dev), x.kvp)[0].shape == (0, 4, 128)

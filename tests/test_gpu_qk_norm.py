"""Norms of query and key heads with the rotation, and their gradient, against float64."""

import pytest
import torch

from parity import gpu_or_skip

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -23
# T, Hq, Hkv, D, rot, interleaved, weights' type (None: rotation alone), strided
CASES = [
    (1, 32, 8, 128, 128, False, torch.float32, True),
    (1, 1, 1, 64, 16, True, torch.bfloat16, False),
    (7, 5, 3, 64, 64, False, torch.float32, False),
    (33, 15, 3, 128, 64, False, torch.bfloat16, True),
    (33, 15, 3, 128, 64, True, torch.float32, True),
    (50, 4, 2, 128, 0, False, torch.float32, False),
    (50, 4, 2, 64, 48, False, None, True),
    (129, 0, 6, 128, 0, False, torch.float32, True),      # an encoder's keys alone
    (129, 6, 0, 64, 32, True, torch.float32, False),
    (3000, 9, 7, 128, 128, False, torch.float32, True),   # several heads to a unit, the last unit short
    (3000, 10, 2, 64, 16, True, torch.bfloat16, False),
]


def _inputs(dev, t, hq, hkv, d, rot, wtype, strided, seed):
    gen = torch.Generator(device=dev).manual_seed(seed)
    x = [torch.randn(t, h, d, generator=gen, device=dev).to(torch.bfloat16) if h else None for h in (hq, hkv)]
    dy = [torch.randn(t, h, d, generator=gen, device=dev).to(torch.bfloat16) if h else None for h in (hq, hkv)]
    if strided and hq and hkv:
        qkv = torch.cat([x[0], x[1], x[1]], dim=1)
        x = [qkv[:, :hq], qkv[:, hq:hq + hkv]]
    w = [(1 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(wtype) if h and wtype else None for h in (hq, hkv)]
    far = 500
    pos = torch.randint(0, far, (t,), generator=gen, device=dev).to(torch.int32)
    table = None
    if rot:
        a = torch.arange(far, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device=dev).double() / rot)
        table = torch.cat([a.cos(), a.sin()], 1).float()
    return x, dy, w, table, pos


def _turn(y, table, pos, interleaved, sign):
    """Rotated y, and |a| + |b| of every rotated pair (|y| elsewhere)."""
    size = y.abs()
    if table is None:
        return y, size
    rot = table.shape[1]
    c, s = (u[:, None, :] for u in table.double()[pos.long()].split(rot // 2, dim=1))
    s = s * sign
    y, size = y.clone(), size.clone()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., at[0]].clone(), y[..., at[1]].clone()
    y[..., at[0]], y[..., at[1]] = a * c - b * s, a * s + b * c
    size[..., at[0]] = size[..., at[1]] = a.abs() + b.abs()
    return y, size


def _forward(x, w, eps, table, pos, interleaved):
    x = x.double()
    y = x
    if w is not None:
        y = x * (x * x).mean(dim=-1, keepdim=True).add(eps).rsqrt() * w.double()
    y, size = _turn(y, table, pos, interleaved, 1)
    # the mean's sum (at most 12 roundings deep) and rsqrt count half, two products, the rotation's two and a sum
    return y, BF * y.abs() + 16 * F32 * size


def _backward(dy, x, w, eps, table, pos, interleaved):
    x = x.double()
    u, usize = _turn(dy.double(), table, pos, interleaved, -1)
    t_u = 4 * F32 * usize
    if w is None:
        return u, BF * u.abs() + t_u, None, None
    r = (x * x).mean(dim=-1, keepdim=True).add(eps).rsqrt()
    n, g = x * r, u * w.double()
    along = (g * n).mean(dim=-1, keepdim=True)
    dx = r * (g - n * along)
    gsize = usize * w.double().abs()
    t_dx = BF * dx.abs() + 24 * F32 * r * (gsize + n.abs() * (gsize * n.abs()).mean(dim=-1, keepdim=True))
    # chains of a lane (up to a few rows), a CTA (32 lanes' sums) and the CTAs (up to 32 slices of 20): under 128 roundings
    return dx, t_dx, (u * n).sum(dim=(0, 1)), 128 * F32 * (usize * n.abs()).sum(dim=(0, 1))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_and_gradient(case):
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    t, hq, hkv, d, rot, interleaved, wtype, strided = CASES[case]
    x, dy, w, table, pos = _inputs(dev, t, hq, hkv, d, rot, wtype, strided, case)
    eps = 1e-5
    more = dict(eps=eps, cos_sin=table, positions=pos, interleaved=interleaved)
    out = attn.attn_qk_norm_rope(x[0], x[1], w[0], w[1], **more)
    grads = attn.attn_qk_norm_rope_bwd(dy[0], dy[1], x[0], x[1], w[0], w[1], **more)
    for i in range(2):
        if x[i] is None:
            assert out[i] is None and grads[i] is None and grads[2 + i] is None
            continue
        y, tol = _forward(x[i], w[i], eps, table, pos, interleaved)
        assert ((out[i].double() - y).abs() <= tol).all()
        dx, tol, dw, tol_w = _backward(dy[i], x[i], w[i], eps, table, pos, interleaved)
        assert ((grads[i].double() - dx).abs() <= tol).all()
        if w[i] is None:
            assert grads[2 + i] is None
        else:
            assert ((grads[2 + i].double() - dw).abs() <= tol_w).all()


def test_gradient_against_differences():
    """Between two points of the float64 formula, along a direction: the difference's own error at h = 1e-5 is about 1e-9."""
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x, dy, w, table, pos = _inputs(dev, 20, 3, 2, 64, 32, torch.float32, False, 3)
    dq, dk, dwq, dwk, _ = attn.attn_qk_norm_rope_bwd(*dy, *x, *w, eps=1e-5, cos_sin=table, positions=pos)
    gen = torch.Generator(device=dev).manual_seed(9)
    for i, (g, gw) in enumerate(((dq, dwq), (dk, dwk))):
        _, t, _, tw = _backward(dy[i], x[i], w[i], 1e-5, table, pos, False)
        for grad, tol, at in ((g, t, 0), (gw, tw, 1)):
            along = torch.randn(grad.shape, generator=gen, device=dev, dtype=torch.float64)
            moved = []
            for h in (1e-5, -1e-5):
                point = [x[i].double(), w[i].double()]
                point[at] = point[at] + h * along
                moved.append((_forward(point[0], point[1], 1e-5, table, pos, False)[0] * dy[i].double()).sum())
            slope = (moved[0] - moved[1]) / 2e-5
            assert (slope - (grad.double() * along).sum()).abs() <= (tol * along.abs()).sum() + 1e-6 * slope.abs() + 1e-6


def test_in_place_and_into_a_projections_gradient():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x, dy, w, table, pos = _inputs(dev, 40, 8, 2, 128, 128, torch.float32, True, 5)
    want = attn.attn_qk_norm_rope(*x, *w, cos_sin=table, positions=pos)
    want_g = attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=pos)
    grad = torch.full((40, 12, 128), 7.0, dtype=torch.bfloat16, device=dev)
    attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=pos, d_q=grad[:, :8], d_k=grad[:, 8:10])
    assert torch.equal(grad[:, :8], want_g[0]) and torch.equal(grad[:, 8:10], want_g[1]) and (grad[:, 10:] == 7).all()
    got = attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=pos, d_q=dy[0], d_k=dy[1])
    assert got[0] is dy[0] and torch.equal(dy[0], want_g[0]) and torch.equal(dy[1], want_g[1])
    got = attn.attn_qk_norm_rope(*x, *w, cos_sin=table, positions=pos, q_out=x[0], k_out=x[1])
    assert got[0] is x[0] and torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])


def test_positions_outside_the_table_and_by_index():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x, dy, w, table, pos = _inputs(dev, 30, 4, 2, 128, 64, torch.float32, False, 6)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    good = attn.attn_qk_norm_rope(*x, *w, cos_sin=table, positions=pos, dev_status=status)
    assert status.item() == 0
    bad = pos.clone()
    bad[3], bad[20] = -1, 500
    keep = torch.ones(30, dtype=torch.bool, device=dev)
    keep[3] = keep[20] = False
    out = [torch.full_like(t, 7.0) for t in x]
    attn.attn_qk_norm_rope(*x, *w, cos_sin=table, positions=bad, q_out=out[0], k_out=out[1], dev_status=status)
    assert status.item() == attn.ATTN_DEV_POSITION_OUT_OF_RANGE
    for a, b in zip(out, good):
        assert torch.equal(a[keep], b[keep]) and (a[~keep] == 7).all()
    grads = attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=bad)
    for i in range(2):
        dx, tol, dw, tol_w = _backward(dy[i][keep], x[i][keep], w[i], 1e-6, table, pos[keep], False)
        assert ((grads[i][keep].double() - dx).abs() <= tol).all() and (grads[i][~keep] == 0).all()
        assert ((grads[2 + i].double() - dw).abs() <= tol_w).all()
    by_index = attn.attn_qk_norm_rope(*x, *w, cos_sin=table)
    same = attn.attn_qk_norm_rope(*x, *w, cos_sin=table, positions=torch.arange(30, dtype=torch.int32, device=dev))
    assert all(torch.equal(a, b) for a, b in zip(by_index, same))


def test_edges_and_refusals():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x, dy, w, table, pos = _inputs(dev, 12, 4, 2, 128, 64, torch.float32, False, 7)
    # rows of zeros stay zeros, and NaN stays in its row
    x[0][1] = 0
    x[0][2, 1, 5] = float("nan")
    q, _ = attn.attn_qk_norm_rope(*x, *w, cos_sin=table, positions=pos)
    assert (q[1] == 0).all() and torch.isnan(q[2, 1]).all() and torch.isfinite(q[2, 0]).all() and torch.isfinite(q[3:]).all()
    # no tokens: empty outputs, gradients of the weights 0
    none = attn.attn_qk_norm_rope_bwd(dy[0][:0], dy[1][:0], x[0][:0], x[1][:0], *w)
    assert none[0].shape == (0, 4, 128) and (none[2] == 0).all() and (none[3] == 0).all()
    for bad in (dict(q=x[0].float()), dict(k=x[1][:5]), dict(q_weight=w[0][:64]), dict(q_weight=w[0].double()),
                dict(q_weight=w[0].bfloat16()), dict(cos_sin=table.double()), dict(positions=pos[:3]), dict(q=None),
                dict(q=None, q_weight=None, k=None, k_weight=None), dict(q_out=torch.empty(12, 4, 64, device=dev).bfloat16()),
                dict(k=x[1][:, :, :64])):
        with pytest.raises(ValueError):
            attn.attn_qk_norm_rope(**{**dict(q=x[0], k=x[1], q_weight=w[0], k_weight=w[1], cos_sin=table, positions=pos), **bad})
    for eps in (0.0, -1.0, float("inf")):
        with pytest.raises(attn.AttnError):
            attn.attn_qk_norm_rope(*x, *w, eps=eps)
    with pytest.raises(attn.AttnError) as e:
        attn.attn_qk_norm_rope_bwd(*dy, *x, *w, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    assert e.value.status == -3


def test_sums_do_not_depend_on_timing_and_replay_from_a_graph():
    dev = gpu_or_skip()
    import causal_gqa_flashattention_attn_gb300 as attn
    x, dy, w, table, pos = _inputs(dev, 2500, 8, 2, 128, 128, torch.float32, False, 8)
    ws = torch.empty(attn.attn_qk_norm_rope_bwd_workspace_bytes(2500, 8, 2), dtype=torch.uint8, device=dev)
    first = [t.clone() for t in attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=pos, workspace=ws)[:4]]
    for _ in range(3):
        got = attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=pos, workspace=ws)[:4]
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        attn.attn_qk_norm_rope_bwd(*dy, *x, *w, cos_sin=table, positions=pos, workspace=ws, d_q=outs[0], d_k=outs[1],
                                   d_q_weight=outs[2], d_k_weight=outs[3], stream=side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))

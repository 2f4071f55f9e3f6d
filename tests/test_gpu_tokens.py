"""Tokens sorted by expert, copied out and brought back, and the router's
backward, against 64-bit references, and a run of them together with the router
and linear attention.  Copies are exact; sums of k products in fp32 are off by
at most k half steps of the sums of absolute values, plus half a step of the
result's type."""
import numpy as np
import pytest
import torch

import operator_refs as refs
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(t):
    return refs.U16 if t.dtype == torch.bfloat16 else refs.U32


def up(t):
    return t.double().cpu().numpy()


def make_idx(T, E, k, drop, seed):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32) if T else np.zeros((0, k), np.int32)
    if drop:
        idx[rng.random((T, k)) < drop] = -1
    return idx


SORTS = [(1, 1, 1, 0), (1, 64, 3, 0), (7, 3, 2, 0.3), (64, 8, 2, 0), (1000, 5, 5, 0.1), (1024, 64, 1, 0),
         (1025, 16, 2, 0.2), (5000, 16, 2, 0), (40000, 64, 3, 0.05), (300000, 8, 1, 0.5), (200, 4, 2, 1.1)]


@pytest.mark.parametrize("T,E,k,drop", SORTS)
def test_sort(T, E, k, drop):
    idx = make_idx(T, E, k, drop, T + E)
    if T > 10:
        idx[3, 0], idx[5, 0] = E, -7  # outside
        idx[9] = idx[9, 0]            # the same expert in every slot
    order, pos, offsets = swimba.sort_tokens(torch.from_numpy(idx).to(DEV), E)
    flat = idx.reshape(-1).astype(np.int64)
    valid = (flat >= 0) & (flat < E)
    want = np.argsort(np.where(valid, flat, E), kind="stable")
    place = np.empty_like(want)
    place[want] = np.arange(T * k)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.bincount(flat[valid], minlength=E).cumsum()]))
    assert np.array_equal(pos.cpu().numpy().reshape(-1), np.where(valid, place, -1))
    assert np.array_equal(order.cpu().numpy(), np.where(valid[want], want, -1))


def test_sort_empty_and_lead_dims():
    order, pos, offsets = swimba.sort_tokens(torch.zeros((0, 2), dtype=torch.int32, device=DEV), 4)
    assert order.numel() == 0 and pos.shape == (0, 2) and not offsets.any()
    idx = torch.randint(0, 8, (3, 50, 2), dtype=torch.int32, device=DEV)
    a, b = swimba.sort_tokens(idx, 8), swimba.sort_tokens(idx.view(150, 2), 8)
    assert a[1].shape == (3, 50, 2)
    assert all(torch.equal(x.reshape(-1), y.reshape(-1)) for x, y in zip(a, b))


MOVES = [(1, 1, 1, 1, 0), (3, 7, 4, 2, 0.3), (33, 64, 8, 2, 0), (50, 130, 4, 4, 0.2), (129, 1001, 16, 3, 0.1),
         (256, 5120, 8, 2, 0.1), (17, 2056, 64, 8, 0), (5, 4096, 2, 1, 0.5)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,E,k,drop", MOVES)
def test_moves(T, D, E, k, drop, dtype):
    rng = np.random.default_rng(T + D)

    def f(*shape, dt=DT[dtype]):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt).to(DEV)

    idx = make_idx(T, E, k, drop, D)
    if T > 2:
        idx[1] = -1  # a padded token
    _, pos, offsets = swimba.sort_tokens(torch.from_numpy(idx).to(DEV), E)
    hp = pos.cpu().numpy()
    used = int(offsets[-1])
    x, rows, dy = f(T, D), f(T * k, D), f(T, D)
    gate = f(T, k, dt=torch.float32)
    if T > 2:
        gate[1] = float("nan")  # the gates of slots without a row are not looked at
    if used < T * k:
        rows[used:] = float("inf")  # nor are rows behind the last

    out = torch.full((T * k, D), 7.0, dtype=DT[dtype], device=DEV)
    assert swimba.dispatch_tokens(x, pos, rows=out) is out
    want = torch.full((T * k, D), 7.0, dtype=DT[dtype])
    for t in range(T):
        for j in range(k):
            if hp[t, j] >= 0:
                want[hp[t, j]] = x[t].cpu()
    assert torch.equal(out.cpu(), want)

    r, g, d = up(rows), up(gate), up(dy)
    for ydt in ("f32", "bf16"):
        y = swimba.combine_tokens(rows, pos, gate, y_dtype=DT[ydt])
        ref = refs.combine(r, hp, g)
        size = refs.combine(np.abs(r), hp, np.abs(g))
        assert (np.abs(up(y) - ref) <= k * refs.U32 * size + half_step(y) * np.abs(ref)).all()
        drows = torch.full((T * k, D), 3.0, dtype=DT[ydt], device=DEV)
        got, dgate = swimba.combine_tokens_backward(rows, pos, gate, dy, drows=drows)
        wr, wg = refs.combine_backward(r, hp, g, d, np.full((T * k, D), 3.0))
        assert (np.abs(up(got) - wr) <= (half_step(got) + refs.U32) * np.abs(wr)).all()
        _, sg = refs.combine_backward(np.abs(r), hp, g, np.abs(d), np.zeros((T * k, D)))
        # a lane's D / 64 (or fewer) products in order, eight levels across lanes and waves
        assert (np.abs(up(dgate) - wg) <= (D / 64 + 24) * refs.U32 * sg + refs.U32 * np.abs(wg)).all()
    dx = swimba.dispatch_tokens_backward(rows, pos)
    ref = refs.combine(r, hp, None)
    assert (np.abs(up(dx) - ref) <= k * refs.U32 * refs.combine(np.abs(r), hp, None) + half_step(dx) * np.abs(ref)).all()


def test_moves_ignore_places_outside():
    # a caller's wrong places are slots without a row, not accesses
    T, k, D = 6, 2, 40
    pos = torch.tensor([[0, 1], [2, 12], [3, 1 << 30], [4, -5], [5, -2 ** 31], [6, 11]], dtype=torch.int32, device=DEV)
    x = torch.randn(T, D, device=DEV)
    rows = torch.zeros(T * k, D, device=DEV)
    swimba.dispatch_tokens(x, pos, rows=rows)
    assert torch.equal(rows[:7].cpu(), x[[0, 0, 1, 2, 3, 4, 5]].cpu()) and torch.equal(rows[11].cpu(), x[5].cpu())
    assert not rows[7:11].any()
    y = swimba.combine_tokens(rows, pos)
    assert torch.equal(y[:5].cpu(), torch.stack([2 * x[0], x[1], x[2], x[3], x[4]]).cpu())
    assert swimba.combine_tokens(x[:0].reshape(0, D), pos[:0]).shape == (0, D)


def test_moves_at_odd_addresses():
    T, k, D = 40, 2, 67
    idx = torch.from_numpy(make_idx(T, 4, k, 0, 1)).to(DEV)
    _, pos, _ = swimba.sort_tokens(idx, 4)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.randn(T * D + 1, device=DEV).to(dt)
        x = buf[1:].view(T, D)
        rows = torch.empty(T * k * D + 1, dtype=dt, device=DEV)[1:].view(T * k, D)
        swimba.dispatch_tokens(x, pos, rows=rows)
        assert torch.equal(rows[pos.long()].cpu(), x.unsqueeze(1).expand(T, k, D).cpu())
        assert torch.equal(swimba.dispatch_tokens_backward(rows, pos, grad_dtype=torch.float32).cpu(), 2 * x.float().cpu())


GRADS = [(1, 1, 1, 1), (1, 5, 4, 2), (64, 64, 16, 2), (65, 257, 16, 1), (200, 130, 33, 3), (500, 300, 64, 4),
         (4097, 70, 8, 2), (90, 1538, 64, 64), (1000, 1024, 17, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,E,k", GRADS)
def test_route_backward(T, D, E, k, dtype):
    rng = np.random.default_rng(T + D + E)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(DT[dtype]).to(DEV)
    Wr = torch.from_numpy((rng.standard_normal((D, E)) * D ** -0.5).astype(np.float32)).to(DEV)
    idx, gate = swimba.route(x, Wr, k)
    dgate = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(DEV)
    if T > 20 and k > 1:
        idx[4] = idx[4, 0]      # an expert listed twice
        idx[7, 1] = -1          # a slot without an expert
        idx[9], x[9] = E, float("nan")  # a token without any: not read
    clean = x.clone()
    if T > 20 and k > 1:
        clean[9] = 0
    wx, wW, sx, sW = refs.route_backward(up(clean), up(Wr), idx.cpu().numpy(), up(gate), up(dgate))
    for gdt in ("f32", "bf16"):
        dx, dW = swimba.route_backward(x, Wr, idx, gate, dgate, grad_dtype=DT[gdt])
        # the slope: k products and three operations more; dx: k products; dWr: T products
        s = (k + 4) * refs.U32
        assert (np.abs(up(dx) - wx) <= (s + k * refs.U32) * sx + half_step(dx) * np.abs(wx)).all()
        assert (np.abs(up(dW) - wW) <= (s + (T + 2) * refs.U32) * sW + refs.U32 * np.abs(wW)).all()
    if k == 1:
        assert not dx.any() and not dW.any()
    again = swimba.route_backward(x, Wr, idx, gate, dgate, grad_dtype=torch.bfloat16)
    assert torch.equal(dx, again[0]) and torch.equal(dW, again[1])


def test_route_backward_empty():
    Wr = torch.randn(16, 4, device=DEV)
    none = torch.zeros((0, 2), device=DEV)
    dx, dW = swimba.route_backward(torch.zeros((0, 16), device=DEV), Wr, none.int(), none, none)
    assert dx.shape == (0, 16) and not dW.any()


def test_route_backward_is_differences():
    # the loss sum(dgate * gate) of the router, along random directions; its
    # second-order term leaves (step^2) and the fp32 gates (2^-22 / step)
    T, D, E, k = 64, 48, 8, 2
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(DEV)
    Wr = torch.from_numpy((rng.standard_normal((D, E)) * D ** -0.5).astype(np.float32)).to(DEV)
    idx, gate = swimba.route(x, Wr, k)
    dgate = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(DEV)
    dx, dW = swimba.route_backward(x, Wr, idx, gate, dgate)

    def loss(x, W):
        l = (x.double() @ W.double()).gather(1, idx.long())
        return float((torch.softmax(l, 1) * dgate.double()).sum())

    step = 2.0 ** -10
    for n, g in ((0, dx), (1, dW)):
        d = torch.from_numpy(rng.standard_normal(g.shape).astype(np.float32)).to(DEV)
        a = (loss(x + step * d, Wr) - loss(x - step * d, Wr)) if n == 0 else (loss(x, Wr + step * d) - loss(x, Wr - step * d))
        want = a / (2 * step)
        scale = float((g.double() * d.double()).abs().sum())
        assert abs(float((g.double() * d.double()).sum()) - want) < (2.0 ** -12) * scale


def test_layer_together():
    """Router -> rows by expert -> a projection per expert -> back weighted ->
    linear attention, and all the way back, against the same layer in 64 bits
    (autograd through elementary operations)."""
    torch.manual_seed(0)
    B, L, D, E, k, H, P, N = 2, 70, 64, 6, 2, 4, 16, 32
    x = torch.randn(B, L, D, device=DEV)
    Wr = torch.randn(D, E, device=DEV) * D ** -0.5
    We = torch.randn(E, D, D, device=DEV) * D ** -0.5
    q, kk = (torch.randn(B, L, 2, N, device=DEV) * N ** -0.25 for _ in range(2))
    g = -torch.rand(B, L, H, device=DEV) * 0.2
    dy = torch.randn(B, L, H, P, device=DEV)

    idx, gate = swimba.route(x, Wr, k)
    order, pos, offsets = swimba.sort_tokens(idx, E)
    rows = swimba.dispatch_tokens(x, pos)
    cut = offsets.tolist()
    out = torch.cat([rows[a:b] @ We[e] for e, (a, b) in enumerate(zip(cut[:-1], cut[1:]))])
    v = swimba.combine_tokens(out, pos, gate).view(B, L, H, P)
    y, h = swimba.linear_attention(q, kk, v, g)
    grads = swimba.linear_attention_backward(q, kk, v, g, dy)
    dout, dgate = swimba.combine_tokens_backward(out, pos, gate, grads["dv"].view(B, L, D))
    drows = torch.cat([dout[a:b] @ We[e].t() for e, (a, b) in enumerate(zip(cut[:-1], cut[1:]))])
    dWe = torch.stack([rows[a:b].t() @ dout[a:b] for a, b in zip(cut[:-1], cut[1:])])
    dx, dWr = swimba.route_backward(x, Wr, idx, gate, dgate)
    dx = dx + swimba.dispatch_tokens_backward(drows, pos)

    r = {n: t.double().cpu().requires_grad_() for n, t in
         (("x", x), ("Wr", Wr), ("We", We), ("q", q), ("k", kk), ("g", g))}
    i = idx.cpu().long()
    rg = torch.softmax((r["x"] @ r["Wr"]).gather(2, i), 2)
    rv = sum(rg[..., j:j + 1] * torch.matmul(r["x"].unsqueeze(2), r["We"][i[..., j]]).squeeze(2) for j in range(k))
    rv = rv.view(B, L, H, P)
    st, ys = torch.zeros(B, H, N, P, dtype=torch.float64), []
    for t in range(L):
        kt, qt = (r[n][:, t].repeat_interleave(2, dim=1) for n in "kq")
        st = r["g"][:, t].exp()[..., None, None] * st + kt.unsqueeze(-1) * rv[:, t].unsqueeze(2)
        ys.append((qt.unsqueeze(-1) * st).sum(2))
    ry = torch.stack(ys, 1)
    (ry * dy.double().cpu()).sum().backward()
    pairs = {"y": (y, ry), "h": (h, st), "x": (dx, r["x"].grad), "Wr": (dWr, r["Wr"].grad), "We": (dWe, r["We"].grad),
             "q": (grads["dq"], r["q"].grad), "k": (grads["dk"], r["k"].grad), "g": (grads["dlog_decay"], r["g"].grad)}
    # fp32 throughout: relative to the norm, the longest chain of sums (rows of
    # 64, 70 tokens, states, 140 rows of a weight) stays under 1000 half steps
    for n, (a, b) in pairs.items():
        err = (a.double().cpu() - b.detach()).norm() / b.detach().norm()
        assert err < 1000 * refs.U32, (n, float(err))


def test_captured_replays():
    T, D, E, k = 3000, 256, 8, 2
    x = torch.randn(T, D, device=DEV).bfloat16()
    Wr = torch.randn(D, E, device=DEV) * D ** -0.5
    dgate = torch.randn(T, k, device=DEV)

    def run(stream=None):
        kw = {} if stream is None else {"stream": stream}
        idx, gate = swimba.route(x, Wr, k, **kw)
        order, pos, offsets = swimba.sort_tokens(idx, E, **kw)
        rows = swimba.dispatch_tokens(x, pos, **kw)
        y = swimba.combine_tokens(rows, pos, gate, **kw)
        drows, dg = swimba.combine_tokens_backward(rows, pos, gate, y, **kw)
        return [order, pos, offsets, rows, y, drows, dg] + list(swimba.route_backward(x, Wr, idx, gate, dgate, **kw))

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, held, again))


def test_binding_refuses():
    x = torch.randn(8, 16, device=DEV)
    pos = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        swimba.dispatch_tokens(x[:4], pos)
    with pytest.raises(ValueError):
        swimba.dispatch_tokens(x, pos.long())
    with pytest.raises(ValueError):
        swimba.combine_tokens(x, pos)  # 16 rows wanted
    with pytest.raises(ValueError):
        swimba.combine_tokens(torch.randn(16, 16, device=DEV), pos, torch.ones(8, 1, device=DEV))
    with pytest.raises(TypeError):
        swimba.dispatch_tokens(x.half(), pos)
    with pytest.raises(ValueError):
        swimba.sort_tokens(pos.t(), 4)
    with pytest.raises(swimba.SwimbaError):
        swimba.sort_tokens(pos, 1)  # k > E


@pytest.mark.parametrize("T,D", [(1, 1), (2, 3), (1, 7), (3, 1), (1, 3)])
def test_tensors_of_less_than_a_pack(T, D):
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(T, D, device=DEV).to(dt)
        _, pos, _ = swimba.sort_tokens(idx, 2)
        rows = swimba.dispatch_tokens(x, pos)
        assert torch.equal(rows.cpu(), x.cpu())
        gate = torch.full((T, 1), 0.5, device=DEV)
        assert torch.equal(swimba.combine_tokens(rows, pos, gate).cpu(), (0.5 * x.float()).to(dt).cpu())
        drows, dgate = swimba.combine_tokens_backward(rows, pos, gate, x)
        assert torch.equal(drows.cpu(), (0.5 * x.float()).to(dt).cpu())
        want = (up(x) ** 2).sum(1, keepdims=True)
        assert (np.abs(up(dgate) - want) <= (D + 8) * refs.U32 * want).all()
        two = torch.tensor([[0, 1]] * T, dtype=torch.int32, device=DEV)
        g2, dg2 = torch.full((T, 2), 0.5, device=DEV), torch.tensor([[1.0, -1.0]] * T, device=DEV)
        W = torch.randn(D, 2, device=DEV)
        dx, dW = swimba.route_backward(x, W, two, g2, dg2)
        wx, wW, sx, sW = refs.route_backward(up(x), up(W), two.cpu().numpy(), up(g2), up(dg2))
        assert (np.abs(up(dx) - wx) <= 10 * refs.U32 * sx).all()
        assert (np.abs(up(dW) - wW) <= (T + 10) * refs.U32 * sW).all()


@pytest.mark.parametrize("D", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("T", [9, 300])
def test_rows_narrower_than_a_pack(T, D):
    gen = torch.Generator().manual_seed(T + D)
    idx = torch.from_numpy(make_idx(T, 4, 2, 0.1, seed=D)).to(DEV)
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(T, D, generator=gen).to(dt).to(DEV)
        order, pos, off = swimba.sort_tokens(idx, 4)
        n = int(off[-1])
        rows = swimba.dispatch_tokens(x, pos)
        assert torch.equal(rows[:n], x[order[:n].long() // 2])
        rows[n:] = 0
        gate = torch.rand(T, 2, generator=gen).to(DEV)
        y = swimba.combine_tokens(rows, pos, gate, y_dtype=torch.float32)
        g = torch.where(pos >= 0, gate, torch.zeros_like(gate)).double()
        want = g.sum(1, keepdim=True) * x.double()
        size = want.abs() + 1e-30
        assert ((y.double() - want).abs() <= 4 * refs.U32 * size).all()
        drows, dgate = swimba.combine_tokens_backward(rows, pos, gate, x, grad_dtype=torch.float32)
        want = gate.flatten()[order[:n].long()][:, None].double() * x[order[:n].long() // 2].double()
        assert ((drows[:n].double() - want).abs() <= 2 * refs.U32 * want.abs()).all()
        want = torch.where(pos >= 0, (x.double() ** 2).sum(1, keepdim=True), 0.0)
        assert ((dgate.double() - want).abs() <= (D + 8) * refs.U32 * want).all()
        W, dg = torch.randn(D, 4, generator=gen).to(DEV), torch.randn(T, 2, generator=gen).to(DEV)
        dx, dW = swimba.route_backward(x, W, idx, gate, dg)
        wx, wW, sx, sW = refs.route_backward(up(x), up(W), idx.cpu().numpy(), up(gate), up(dg))
        assert (np.abs(up(dx) - wx) <= 12 * refs.U32 * sx).all()
        assert (np.abs(up(dW) - wW) <= (T + 12) * refs.U32 * sW).all()


def test_combine_backward_of_more_tokens_than_a_grid_row():
    T, D = (1 << 24) + 5, 3
    gen = torch.Generator(device=DEV).manual_seed(3)
    rows = torch.randn(T, D, generator=gen, device=DEV)
    dy = torch.randn(T, D, generator=gen, device=DEV)
    gate = torch.rand(T, 1, generator=gen, device=DEV)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)[:, None]
    drows, dgate = swimba.combine_tokens_backward(rows, pos, gate, dy)
    assert torch.equal(drows, (gate * dy).flip(0))  # one product, rounded once
    terms = dy.double() * rows.flip(0).double()
    assert ((dgate[:, 0].double() - terms.sum(1)).abs() <= (D + 8) * refs.U32 * terms.abs().sum(1)).all()

"""The gated delta rule against the 64-bit recurrence.  An output may be off by its
roundings' bound (delta_refs.bounds) plus half a step of its own type."""
import numpy as np
import pytest
import torch

import delta_refs as refs
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OPS = ("q", "k", "v", "g", "beta")


def make(B, L, H, G, N, P, dtype="bf16", form="token", h0=True, seed=0, reset=None):
    gen = torch.Generator().manual_seed(seed)

    def f(*shape):
        return torch.randn(*shape, generator=gen)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True).clamp(min=1e-3)

    t = {"q": unit(f(B, L, G, N)), "k": unit(f(B, L, G, N)), "v": f(B, L, H, P), "dy": f(B, L, H, P)}
    t = {n: x.to(DT[dtype]) for n, x in t.items()}
    if form == "head":
        t["g"] = torch.log1p(-torch.exp2(-torch.linspace(2, 8, H)))
    else:
        t["g"] = -0.3 * f(B, L, H).abs()
        if reset:
            t["g"][:, ::reset] = -float("inf")
    t["beta"] = torch.sigmoid(f(B, L, H))
    t["h0"] = f(B, H, N, P) if h0 else None
    t["dh"] = f(B, H, N, P) if h0 else None
    return t


def to_dev(t):
    return {n: None if x is None else x.to(DEV) for n, x in t.items()}


def wide(t, *names):
    return [None if t[n] is None else t[n].double() for n in names]


def close(got, want, allow, what):
    g = got.double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    most = allow + refs.HALF[got.dtype] * want.abs() * (1 + 2.0 ** -8) + 1e-30
    bad = ~((g - want).abs() <= most)
    assert not bad.any(), "%s: %d of %d off, worst %.3g times the bound" % (
        what, bad.sum(), bad.numel(), ((g - want).abs() / most).max())


def forward(d, **kw):
    return swimba.delta_rule(*(d[n] for n in OPS), h0=d["h0"], **kw)


def backward(d, **kw):
    return swimba.delta_rule_backward(*(d[n] for n in OPS), d["dy"], h0=d["h0"], dh_final=d["dh"], **kw)


def check_forward(t, dtype, ydt):
    y, h = forward(to_dev(t), y_dtype=DT[ydt])
    a = wide(t, *OPS, "h0")
    want, allow = refs.delta(*a), refs.bounds(dtype == "f32", *a, y_bf16=ydt == "bf16")
    close(h, want["h_final"], allow["h_final"], "h_final")
    close(y, want["y"], allow["y"], "y")


def check_backward(t, dtype, gdt):
    g = backward(to_dev(t), grad_dtype=DT[gdt])
    a = wide(t, *OPS, "h0", "dy", "dh")
    want, allow = refs.delta(*a), refs.bounds(dtype == "f32", *a)
    for name in ("dq", "dk", "dv", "dbeta", "dlog_decay", "dh0"):
        w = want[name]
        if name == "dlog_decay" and w.dim() == 3:  # documented: zero where nothing passes
            w = torch.where(a[3].exp() < 2.0 ** -150, torch.zeros_like(w), w)
        close(g[name], w, allow[name], name)


SHAPES = [  # B, L, H, G, N, P
    (1, 1, 1, 1, 1, 1), (2, 2, 2, 1, 16, 16), (1, 63, 2, 2, 32, 33), (1, 64, 3, 1, 33, 32),
    (2, 65, 4, 2, 64, 64), (1, 200, 6, 2, 80, 50), (1, 130, 2, 1, 128, 128), (1, 17, 2, 1, 9, 70),
    (1, 90, 1, 1, 24, 300), (3, 128, 5, 5, 100, 64), (1, 129, 3, 3, 127, 15)]
WIDE = [(1, 70, 1, 1, 129, 17), (1, 100, 2, 1, 256, 40), (1, 66, 2, 2, 200, 130)]  # bf16 only


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    check_forward(make(*shape, dtype=dtype, seed=sum(shape)), dtype, dtype)
    check_forward(make(*shape, dtype=dtype, form="head", h0=False, seed=1 + sum(shape)), dtype, "f32")


@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_wide_keys(shape):
    check_forward(make(*shape, seed=sum(shape)), "bf16", "bf16")
    check_forward(make(*shape, form="head", h0=False, seed=sum(shape)), "bf16", "f32")
    check_backward(make(*shape, seed=2 + sum(shape)), "bf16", "f32")
    d = to_dev(make(*shape, dtype="f32"))
    for call in (forward, backward):
        with pytest.raises(swimba.SwimbaError) as e:
            call(d)
        assert e.value.status == swimba.EUNSUPPORTED


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype):
    check_backward(make(*shape, dtype=dtype, seed=2 + sum(shape)), dtype, "f32")
    check_backward(make(*shape, dtype=dtype, form="head", h0=False, seed=3 + sum(shape)), dtype, dtype)


@pytest.mark.parametrize("dtype,shape,reset", [("bf16", (1, 700, 4, 1, 64, 64), 131), ("f32", (2, 300, 2, 1, 48, 33), 64),
                                               ("bf16", (1, 150, 2, 2, 128, 100), 7), ("f32", (1, 130, 1, 1, 20, 20), 1)])
def test_documents(dtype, shape, reset):
    check_forward(make(*shape, dtype=dtype, seed=11, reset=reset), dtype, "f32")
    check_backward(make(*shape, dtype=dtype, seed=12, reset=reset), dtype, "f32")


@pytest.mark.parametrize("dtype,shape", [("bf16", (1, 2100, 2, 1, 64, 64)), ("bf16", (2, 1500, 1, 1, 128, 33)),
                                         ("f32", (1, 1300, 3, 3, 40, 20))])
def test_long(dtype, shape):
    check_forward(make(*shape, dtype=dtype, seed=7, reset=411), dtype, "f32")
    check_backward(make(*shape, dtype=dtype, form="head", seed=8), dtype, "f32")


@pytest.mark.parametrize("B,L,H,G", [(5, 3900, 4, 1), (8, 4200, 6, 2)])  # two heads, three heads at a time
def test_heads_that_share_keys_are_summed(B, L, H, G):
    check_backward(make(B, L, H, G, 16, 16, seed=9, reset=900), "bf16", "f32")


def test_wide_keys_in_segments():
    t = make(1, 900, 1, 1, 200, 20, seed=10, reset=500)
    check_forward(t, "bf16", "f32")
    check_backward(t, "bf16", "f32")


def test_many_segments():
    # and a last one that is shorter
    t = make(1, 64 * 75 + 13, 1, 1, 32, 16, form="head", seed=16)
    check_forward(t, "bf16", "f32")
    check_backward(t, "bf16", "bf16")


def test_a_document_is_its_own():
    # behind a cleared state nothing of the first document is left, whatever its size
    t = make(1, 100, 2, 1, 32, 32, dtype="f32", seed=13)
    t["g"][:, 41] = -float("inf")
    d = to_dev(t)
    y, h = forward(d)
    g = backward(d)
    e = {n: None if x is None else x.clone() for n, x in d.items()}
    e["v"][:, :41] *= 1e4
    e["h0"] *= 1e4
    y2, h2 = forward(e)
    assert torch.equal(y[:, 41:], y2[:, 41:]) and torch.equal(h, h2)
    g2 = backward(e)
    for n in ("dq", "dk", "dv", "dbeta"):
        assert torch.equal(g[n][:, 41:], g2[n][:, 41:]), n
    # its decays' gradient shares 64-bit prefix sums with the first document's
    assert torch.allclose(g["dlog_decay"][:, 41:], g2["dlog_decay"][:, 41:], rtol=0, atol=1e-6)
    assert not g2["dlog_decay"][:, 41].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_decays_next_to_small_ones(dtype):
    t = make(1, 128, 2, 1, 32, 32, dtype=dtype, seed=3)
    t["g"] = torch.full((1, 128, 2), -0.01)
    t["g"][:, 5:60:3] = -80.0
    check_forward(t, dtype, "f32")
    check_backward(t, dtype, "f32")


def test_growing_decays_are_taken_as_they_are():
    t = make(1, 150, 1, 1, 16, 16, dtype="f32", seed=4)
    t["g"] = torch.full((1, 150, 1), 0.02)
    check_forward(t, "f32", "f32")
    check_backward(t, "f32", "f32")


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
def test_one_key_again_and_again(beta):
    # the hardest inverse: every key the same, nothing, all or twice of it erased
    t = make(1, 130, 2, 1, 32, 20, dtype="f32", seed=5)
    t["k"][:] = 0
    t["k"][..., 3] = 1.0
    t["beta"][:] = beta
    t["g"][:] = 0
    check_forward(t, "f32", "f32")
    check_backward(t, "f32", "f32")


def test_keys_of_zero_and_beta_of_zero():
    t = make(2, 80, 2, 1, 24, 24, dtype="f32", seed=6)
    t["k"][:, 10:20] = 0
    t["beta"][:, 15:30] = 0
    t["beta"][:, 40] = -0.5
    check_forward(t, "f32", "f32")
    check_backward(t, "f32", "f32")


def test_gradients_are_differences():
    # linear in q, v and h0: one difference is exact; the others by central differences of
    # the 64-bit reference's own outputs are tested on the CPU
    t = make(2, 100, 4, 2, 48, 40, dtype="f32", seed=21)
    d = to_dev(t)
    g = backward(d)
    allow = refs.bounds(True, *wide(t, *OPS, "h0"))

    def loss(x):
        y, h = forward(x)
        return float((d["dy"].double() * y.double()).sum() + (d["dh"].double() * h.double()).sum())

    # outputs off by their bounds, up to the largest of them; moved inputs are up to 5 times as large
    off = float((t["dy"].double().abs() * (allow["y"] + 2.0 ** -24)).sum() + (t["dh"].double().abs() * allow["h_final"]).sum())
    gen = torch.Generator().manual_seed(2)
    for name in ("q", "v", "h0"):
        m = torch.randn(t[name].shape, generator=gen).to(DEV)
        up, down = loss(dict(d, **{name: d[name] + m})), loss(dict(d, **{name: d[name] - m}))
        got = float((g["d" + name].double() * m.double()).sum())
        assert abs((up - down) / 2 - got) < 10 * off, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,N,P", [(1, 1, 1, 1, 1), (2, 6, 2, 80, 50), (3, 4, 4, 128, 128), (1, 24, 1, 64, 64),
                                       (2, 3, 1, 256, 17), (40, 16, 16, 33, 260), (1, 2, 1, 200, 64), (1, 1, 1, 5, 3)])
def test_step(B, H, G, N, P, dtype):
    for form in ("token", "head"):
        t = make(B, 1, H, G, N, P, dtype=dtype, form=form, seed=N + P)
        d = to_dev(t)
        a = [d[n][:, 0].contiguous() for n in ("q", "k", "v")]
        a += [d["g"][:, 0].contiguous() if form == "token" else d["g"], d["beta"][:, 0].contiguous()]
        out = torch.empty_like(d["h0"])
        y = swimba.delta_rule_step(*a, d["h0"], state_out=out)
        r = wide(t, *OPS, "h0")
        want = refs.delta(*r)
        # fp32 sums of N terms, three times (k.h, q.h, k.q), and a few single roundings; e^g within 4
        m = (3 * N + 16) * refs.U0
        e = r[3].expand(B, 1, H)[:, 0].exp()[..., None]
        qh, kh = (x[:, 0].repeat_interleave(H // G, 1).unsqueeze(-1).abs() for x in r[:2])
        ah = r[5].abs()
        u = r[4][:, 0, :, None] * (r[2][:, 0].abs() + e * (kh * ah).sum(2))
        close(out, want["h_final"], m * (e[..., None] * ah + kh * u[:, :, None]), "state")
        size = e * (qh * ah).sum(2) + (qh * kh).sum(2) * u
        close(y, want["y"][:, 0], m * size, "y")
        st = d["h0"].clone()
        y2 = swimba.delta_rule_step(*a, st, y_dtype=torch.float32)
        assert torch.equal(st, out)
        close(y2, want["y"][:, 0], m * size, "y in place")
        call = swimba.PreparedDeltaRuleStep(*a, d["h0"], state_out=out.zero_())
        assert torch.equal(call(), y) and torch.equal(out, st)


def test_step_misaligned_state():
    t = make(2, 1, 2, 1, 20, 32, dtype="f32", seed=9)
    d = to_dev(t)
    buf = torch.empty(d["h0"].numel() + 1, device=DEV)
    st = buf[1:].view(d["h0"].shape)
    st.copy_(d["h0"])
    a = [d[n][:, 0].contiguous() for n in OPS]
    y = swimba.delta_rule_step(*a, st)
    want = swimba.delta_rule_step(*a, d["h0"])
    # other columns per thread, the same sums in another order
    assert torch.allclose(y, want, rtol=0, atol=1e-5) and torch.allclose(st, d["h0"], rtol=0, atol=1e-5)


def test_rows_at_odd_addresses():
    for dtype in ("bf16", "f32"):
        t = make(1, 90, 3, 1, 37, 21, dtype=dtype, seed=31)
        d = to_dev(t)
        y, h = forward(d)
        g = backward(d)
        for n in ("q", "k", "v", "dy"):
            buf = torch.empty(d[n].numel() + 1, dtype=d[n].dtype, device=DEV)
            x = buf[1:].view(d[n].shape)
            x.copy_(d[n])
            d[n] = x
        y2, h2 = forward(d)
        assert torch.equal(y, y2) and torch.equal(h, h2)
        g2 = backward(d)
        assert all(torch.equal(g[n], g2[n]) for n in g)


def test_split_sequences_and_steps_agree():
    t = make(2, 150, 4, 2, 64, 32, dtype="f32", seed=5)
    d = to_dev(t)
    a = wide(t, *OPS, "h0")
    want, allow = refs.delta(*a), refs.bounds(True, *a)
    y1, h1 = swimba.delta_rule(*(d[n][:, :97].contiguous() for n in OPS), h0=d["h0"])
    y2, h2 = swimba.delta_rule(*(d[n][:, 97:].contiguous() for n in OPS), h0=h1)
    # other chunks, the same transitions: the parts' bounds are within twice the whole's
    close(torch.cat([y1, y2], 1), want["y"], 2 * allow["y"], "y")
    close(h2, want["h_final"], 2 * allow["h_final"], "h")
    st = d["h0"].clone()
    for i in range(20):
        y = swimba.delta_rule_step(*(d[n][:, i].contiguous() for n in OPS), st)
        close(y, want["y"][:, i], 2 * allow["y"][:, i], "step %d" % i)


def test_empty():
    d = to_dev(make(2, 0, 2, 1, 8, 8, dtype="f32", form="head"))
    y, h = forward(d)
    assert y.shape == (2, 0, 2, 8) and torch.equal(h, d["h0"])
    g = backward(d)
    assert torch.equal(g["dh0"], d["dh"]) and not g["dlog_decay"].any() and g["dbeta"].shape == (2, 0, 2)
    d = to_dev(make(0, 5, 2, 1, 8, 8, dtype="f32", form="head", h0=False))
    y, h = forward(d)
    assert y.shape == (0, 5, 2, 8) and h.shape == (0, 2, 8, 8)
    assert not backward(d)["dlog_decay"].any()


def both(d, stream=None):
    y, h = forward(d, stream=stream)
    return [y, h] + list(backward(d, stream=stream).values())


@pytest.mark.parametrize("form", ["token", "head"])
def test_deterministic(form):
    d = to_dev(make(2, 700, 8, 2, 64, 64, form=form, seed=8))
    runs = [both(d) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


@pytest.mark.parametrize("form", ["token", "head"])
def test_captured_and_side_stream(form):
    d = to_dev(make(1, 1000, 4, 2, 64, 64, form=form, seed=12))
    want = both(d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(d, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(d)
    for i in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        again = both(d)  # eager work between the replays
        torch.cuda.synchronize()
        for a, b, c in zip(want, held, again):
            assert torch.equal(a, b) and torch.equal(a, c), i
    d["v"].mul_(0.5)
    graph.replay()
    want = both(d)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_captured_step():
    d = to_dev(make(3, 1, 4, 2, 64, 64, seed=14))
    a = [d[n][:, 0].contiguous() for n in OPS]
    call = swimba.PreparedDeltaRuleStep(*a, d["h0"])
    st = d["h0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    d["h0"].copy_(st)
    for _ in range(3):
        want = swimba.delta_rule_step(*a, st)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.y, want) and torch.equal(st, d["h0"])


def test_own_workspace_and_outputs():
    d = to_dev(make(2, 200, 4, 2, 32, 48, seed=15))
    y, h = forward(d)
    need = swimba.delta_rule_workspace_bytes(*(d[n] for n in OPS))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read unwritten
    out = torch.empty_like(y)
    y2, h2 = forward(d, workspace=ws, y=out)
    assert y2 is out and torch.equal(y, y2) and torch.equal(h, h2)
    with pytest.raises(swimba.SwimbaError) as e:
        forward(d, workspace=ws[:need - 256])
    assert e.value.status == swimba.EWORKSPACE
    y3, none = forward(d, want_state=False)
    assert none is None and torch.equal(y, y3)
    g = backward(d, want_dh0=False)
    assert "dh0" not in g and all(torch.equal(g[n], x) for n, x in backward(d).items() if n != "dh0")


def test_wrong_arguments():
    d = to_dev(make(1, 8, 4, 2, 16, 16))
    q, k, v, g, beta = (d[n] for n in OPS)
    with pytest.raises(ValueError):
        swimba.delta_rule(q, k[:, :4].contiguous(), v, g, beta)
    with pytest.raises(ValueError):
        swimba.delta_rule(q, k, v, g.bfloat16(), beta)
    with pytest.raises(ValueError):
        swimba.delta_rule(q, k, v, g, beta.bfloat16())
    with pytest.raises(ValueError):
        swimba.delta_rule(q, k, v, g, beta[:, :, :2].contiguous())
    with pytest.raises(ValueError):
        swimba.delta_rule(q.float(), k, v, g, beta)
    with pytest.raises(ValueError):
        swimba.delta_rule(q, k, v.transpose(1, 2), g, beta)
    with pytest.raises(ValueError):
        swimba.delta_rule(q, k, v, g, beta, h0=torch.zeros(1, 4, 16, 8, device=DEV))
    with pytest.raises(swimba.SwimbaError):
        three = torch.zeros(1, 8, 3, 16, dtype=q.dtype, device=DEV)
        swimba.delta_rule(three, three, v, g, beta)
    with pytest.raises(TypeError):
        swimba.delta_rule(q.half(), k.half(), v.half(), g, beta)
    with pytest.raises(ValueError):
        swimba.delta_rule_backward(q, k, v, g, beta, torch.zeros(1, 8, 4, 16, device=DEV))


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 3, 200), (1, 1, 1, 1, 100, 2), (1, 2, 1, 1, 3, 2), (1, 1, 3, 1, 5, 1)], ids=str)
def test_operands_of_less_than_a_pack(shape):
    for dtype in ("bf16", "f32"):
        check_forward(make(*shape, dtype=dtype, seed=41), dtype, "f32")
        check_backward(make(*shape, dtype=dtype, seed=42), dtype, "f32")


@pytest.mark.parametrize("dtype,N,P,L", [("bf16", 64, 64, 150), ("f32", 33, 20, 150), ("bf16", 128, 96, 1500)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_never_reach_earlier_tokens(dtype, N, P, L, bad):
    # a padded batch may hold anything behind its last token, and the token before
    # it lies in the same chunk
    s = L // 2 + 2
    t = make(1, L, 2, 1, N, P, dtype=dtype, seed=51)
    d = to_dev(t)
    y, h = forward(d)
    a = wide(t, *OPS, "h0")
    want, allow = refs.delta(*a), refs.bounds(dtype == "f32", *a, y_bf16=dtype == "bf16")
    for name in OPS:
        if name == "g" and bad < 0:
            continue  # clears the state
        e = {n: x.clone() for n, x in d.items()}
        e[name][0, s].view(-1)[1] = bad  # key 1, value (head 0, column 1), head 1
        y2, h2 = forward(e)
        if name in ("k", "g", "beta"):
            # the chunk is walked without its last tokens: other products, the same bounds
            close(y2[:, :s], want["y"][:, :s], allow["y"][:, :s], name)
        else:
            assert torch.equal(y2[:, :s], y[:, :s]), name
        if name == "q":
            keep = torch.arange(L, device=DEV) != s
            assert torch.equal(y2[:, keep], y[:, keep]) and torch.equal(h2, h)
            assert not torch.isfinite(y2[:, s]).any()
        elif name == "v":
            assert torch.isnan(y2[0, s:, 0, 1]).all() and torch.isnan(h2[0, 0, :, 1]).all()
            other = torch.arange(P, device=DEV) != 1
            assert torch.equal(y2[0, :, 0, other], y[0, :, 0, other]) and torch.equal(y2[0, :, 1], y[0, :, 1])
            assert torch.equal(h2[0, 0, :, other], h[0, 0, :, other]) and torch.equal(h2[0, 1], h[0, 1])
        elif name == "k":
            assert torch.isnan(y2[:, s:]).all() and torch.isnan(h2).all()
        else:
            assert torch.isnan(y2[0, s:, 1]).all() and torch.equal(y2[0, :, 0], y[0, :, 0])
            assert torch.isnan(h2[0, 1]).all() and torch.equal(h2[0, 0], h[0, 0])


def test_fp32_inputs_bf16_results():
    check_forward(make(2, 90, 4, 2, 40, 24, dtype="f32", seed=61), "f32", "bf16")
    check_backward(make(2, 90, 4, 2, 40, 24, dtype="f32", seed=62), "f32", "bf16")


@pytest.mark.parametrize("scale", [1e5, 1e-6])
def test_large_and_small_magnitudes(scale):
    t = make(1, 140, 2, 1, 32, 32, dtype="f32", seed=71)
    for n in ("q", "v", "h0", "dy", "dh"):
        t[n] = t[n] * scale
    check_forward(t, "f32", "f32")
    check_backward(t, "f32", "f32")


def test_states_in_place():
    d = to_dev(make(1, 500, 4, 2, 64, 64, seed=21))
    y, h = forward(d)
    want = backward(d)
    st = d["h0"].clone()
    y2, h2 = swimba.delta_rule(*(d[n] for n in OPS), h0=st, h_final=st)
    assert torch.equal(y, y2) and torch.equal(h, h2) and h2 is st
    adj = d["dh"].clone()
    got = swimba.delta_rule_backward(*(d[n] for n in OPS), d["dy"], h0=d["h0"], dh_final=adj, out={"dh0": adj})
    assert all(torch.equal(want[n], got[n]) for n in want)


def test_a_layer_trains_and_decodes():
    # queries and keys normed and turned, the rule over a prompt, the way back to the projections,
    # and the same tokens decoded one by one
    B, L, H, G, N, P = 2, 100, 4, 2, 32, 24
    t = make(B, L, H, G, N, P, dtype="f32", seed=81)
    gen = torch.Generator().manual_seed(82)
    proj = torch.randn(B, L, 2 * G * N + 7, generator=gen)  # q and k side by side, and something else
    x = proj.to(DEV)
    q, k = (x[..., i * G * N:(i + 1) * G * N].unflatten(-1, (G, N)) for i in (0, 1))
    w = [1 + 0.1 * torch.randn(N, generator=gen) for _ in range(2)]
    pos = torch.arange(L, dtype=torch.int32).expand(B, L).contiguous()
    rates = torch.pow(100.0, -torch.arange(0, 16, 2) / 16.0)
    how = dict(wq=w[0].to(DEV), wk=w[1].to(DEV), positions=pos.to(DEV), rates=rates.to(DEV), norm="l2")
    d = to_dev(t)
    qn, kn = swimba.norm_rotate(q, k, **how)
    rest = [d[n] for n in ("v", "g", "beta")]
    y, h = swimba.delta_rule(qn, kn, *rest, h0=d["h0"])
    g = swimba.delta_rule_backward(qn, kn, *rest, d["dy"], h0=d["h0"], dh_final=d["dh"])
    back = swimba.norm_rotate_backward(q, k, g["dq"], g["dk"], **how)

    def plain(x):
        return x.double().reshape(B * L, G, N).cpu().numpy()

    ref, _ = refs.norm_rotate(plain(q), plain(k), w[0].double().numpy(), w[1].double().numpy(), pos.reshape(-1).numpy(),
                              rates.numpy(), "l2", "halves", 1e-6, 1.0)
    rq, rk = (torch.from_numpy(ref[n]).reshape(B, L, G, N) for n in "qk")
    a = [rq, rk] + wide(t, "v", "g", "beta", "h0", "dy", "dh")
    want, allow = refs.delta(*a), refs.bounds(True, *a)
    # q and k are off by 24 half steps at most (test_gpu_norm_rotate.py), which the rule passes on like
    # a rounding of its own inputs; its bounds hold 64 of them for every sum
    close(y, want["y"], 2 * allow["y"], "y")
    close(h, want["h_final"], 2 * allow["h_final"], "h")
    grad, size = refs.norm_rotate(plain(q), plain(k), w[0].double().numpy(), w[1].double().numpy(), pos.reshape(-1).numpy(),
                                  rates.numpy(), "l2", "halves", 1e-6, 1.0,
                                  want["dq"].reshape(B * L, G, N).numpy(), want["dk"].reshape(B * L, G, N).numpy())
    _, off = refs.norm_rotate(plain(q), plain(k), w[0].double().numpy(), w[1].double().numpy(), pos.reshape(-1).numpy(),
                              rates.numpy(), "l2", "halves", 1e-6, 1.0,
                              2 * allow["dq"].reshape(B * L, G, N).numpy(), 2 * allow["dk"].reshape(B * L, G, N).numpy())
    for n in ("dq", "dk", "dwq", "dwk"):
        got = back[n].double().cpu().reshape(grad[n].shape).numpy()
        assert (np.abs(got - grad[n]) <= off[n] + (400 * refs.U0) * size[n] + 1e-30).all(), n
    st = d["h0"].clone()
    for i in range(L):
        qi, ki = swimba.norm_rotate(q[:, i], k[:, i], **dict(how, positions=how["positions"][:, i].contiguous()))
        assert torch.equal(qi, qn[:, i]) and torch.equal(ki, kn[:, i])
        yi = swimba.delta_rule_step(qi, ki, *(x[:, i].contiguous() for x in rest), st)
        close(yi, want["y"][:, i], 2 * allow["y"][:, i], "token %d" % i)
    close(st, want["h_final"], 2 * allow["h_final"], "state")

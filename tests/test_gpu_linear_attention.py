"""Linear attention with a decay per head against the 64-bit recurrence.  An
output may be off by its roundings' bound (operator_refs.roundings: half steps
times the same sums over absolute values), plus half a step of its own type."""
import numpy as np
import pytest
import torch

import operator_refs as refs
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, L, H, G, N, P, dtype="bf16", form="token", h0=True, grad=False, seed=0, reset=None):
    rng = np.random.default_rng(seed)

    def f(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32))

    t = {"q": f(B, L, G, N) * N ** -0.25, "k": f(B, L, G, N) * N ** -0.25, "v": f(B, L, H, P)}
    t = {n: x.to(DT[dtype]) for n, x in t.items()}
    if form == "head":
        t["log_decay"] = torch.log1p(-torch.exp2(-torch.linspace(2, 8, H)))
    else:
        t["log_decay"] = -0.3 * f(B, L, H).abs()
        if reset:
            t["log_decay"][:, ::reset] = -float("inf")
    t["h0"] = f(B, H, N, P) if h0 else None
    if grad:
        t["dy"] = f(B, L, H, P).to(DT[dtype])
        t["dh"] = f(B, H, N, P) if h0 else None
    dev = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    ref = {n: None if x is None else x.double().numpy() for n, x in t.items()}
    return dev, ref


def close(got, want, size, bound, what):
    half = refs.U16 if got.dtype == torch.bfloat16 else refs.U32
    g = got.double().cpu().numpy()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    allow = bound * size + half * np.abs(want) + 1e-30
    bad = ~(np.abs(g - want) <= allow)
    assert not bad.any(), "%s: %d of %d off, worst %.3g times the bound" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(g - want) / allow))


def forward(dev, **kw):
    return swimba.linear_attention(dev["q"], dev["k"], dev["v"], dev["log_decay"], h0=dev["h0"], **kw)


def args(ref, grad=False):
    a = [ref["q"], ref["k"], ref["v"], ref["log_decay"], ref["h0"]]
    return a + [ref["dy"], ref["dh"]] if grad else a


SHAPES = [  # B, L, H, G, N, P
    (1, 1, 1, 1, 1, 1), (2, 2, 2, 1, 16, 16), (1, 63, 2, 2, 32, 33), (1, 64, 3, 1, 33, 32),
    (2, 65, 4, 2, 64, 64), (1, 200, 6, 2, 80, 50), (1, 130, 2, 1, 128, 128), (1, 70, 1, 1, 129, 17),
    (1, 100, 2, 1, 256, 40), (1, 90, 1, 1, 24, 300), (3, 128, 5, 5, 100, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    B, L, H, G, N, P = shape
    for form, h0, ydt in (("token", True, dtype), ("head", False, "f32")):
        dev, ref = make(*shape, dtype=dtype, form=form, h0=h0, seed=sum(shape))
        y, h = forward(dev, y_dtype=DT[ydt])
        want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
        b3 = refs.roundings(N, P, L)
        close(h, want["h_final"], size["h_final"], b3, "h_final")
        close(y, want["y"], size["y"], refs.roundings(N, P, L, ydt == "f32"), "y")


@pytest.mark.parametrize("dtype,shape", [("bf16", (1, 2100, 2, 1, 64, 64)), ("bf16", (2, 1500, 1, 1, 128, 33)),
                                         ("f32", (1, 1300, 3, 3, 40, 20)), ("f32", (1, 800, 1, 1, 200, 70))])
def test_forward_in_segments(dtype, shape):
    B, L, H, G, N, P = shape
    dev, ref = make(*shape, dtype=dtype, form="token", seed=7, reset=411)
    assert swimba.linear_attention_workspace_bytes(dev["q"], dev["k"], dev["v"], dev["log_decay"]) > 0
    y, h = forward(dev, y_dtype=torch.float32)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    b = refs.roundings(N, P, L)
    close(h, want["h_final"], size["h_final"], b, "h_final")
    close(y, want["y"], size["y"], b, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype):
    B, L, H, G, N, P = shape
    if P > 256:
        dev, _ = make(*shape, dtype=dtype, grad=True)
        with pytest.raises(swimba.SwimbaError) as e:
            swimba.linear_attention_backward(dev["q"], dev["k"], dev["v"], dev["log_decay"], dev["dy"])
        assert e.value.status == swimba.EUNSUPPORTED
        return
    for form, h0, gdt in (("token", True, "f32"), ("head", False, dtype)):
        dev, ref = make(*shape, dtype=dtype, form=form, h0=h0, grad=True, seed=1 + sum(shape))
        check_backward(dev, ref, shape, gdt)


def check_backward(dev, ref, shape, gdt):
    B, L, H, G, N, P = shape
    g = swimba.linear_attention_backward(dev["q"], dev["k"], dev["v"], dev["log_decay"], dev["dy"],
                                         h0=dev["h0"], dh_final=dev["dh"], grad_dtype=DT[gdt])
    want, size = refs.attention(*args(ref, True)), refs.attention_sizes(*args(ref, True))
    for name in ("dq", "dk", "dv", "dlog_decay", "dh0"):
        b = refs.roundings(N, P, L, not (name == "dv" and gdt == "bf16")) + H // G * refs.U32
        w, s = want[name], size[name]
        if name == "dlog_decay" and w.ndim == 3:  # documented: zero where nothing passes
            w = np.where(np.exp(ref["log_decay"]) == 0, 0.0, w)
        close(g[name], w, s, b, name)


@pytest.mark.parametrize("dtype,shape", [("bf16", (1, 1400, 4, 1, 64, 64)), ("bf16", (1, 1100, 2, 2, 100, 128)),
                                         ("f32", (1, 900, 2, 1, 48, 33))])
def test_backward_in_segments_with_documents(dtype, shape):
    dev, ref = make(*shape, dtype=dtype, form="token", grad=True, seed=11, reset=331)
    check_backward(dev, ref, shape, "f32")


def test_large_decays_next_to_small_ones():
    # after a decay of e^-80 per token the small decays must keep their size:
    # differences of running sums of thousands
    shape = (1, 128, 2, 1, 32, 32)
    dev, ref = make(*shape, dtype="f32", grad=True, seed=3)
    g = np.full((1, 128, 2), -0.01)
    g[:, 5:60:3] = -80.0
    ref["log_decay"] = g
    dev["log_decay"] = torch.from_numpy(g.astype(np.float32)).to(DEV)
    ref["log_decay"] = dev["log_decay"].double().cpu().numpy()
    y, h = forward(dev)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    b = refs.roundings(32, 32, 128)
    close(y, want["y"], size["y"], b, "y")
    close(h, want["h_final"], size["h_final"], b, "h_final")
    check_backward(dev, ref, shape, "f32")


def test_growing_decays_are_taken_as_they_are():
    shape = (1, 150, 1, 1, 16, 16)
    dev, ref = make(*shape, dtype="f32", seed=4)
    dev["log_decay"] = torch.full((1, 150, 1), 0.05, device=DEV)
    ref["log_decay"] = dev["log_decay"].double().cpu().numpy()
    y, h = forward(dev)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    close(y, want["y"], size["y"], refs.roundings(16, 16, 150), "y")


def test_gradients_are_differences():
    # the loss is linear in q, in k, in v and in h0: one difference is exact
    shape = (2, 100, 4, 2, 48, 40)
    dev, _ = make(*shape, dtype="f32", grad=True, seed=21)
    g = swimba.linear_attention_backward(dev["q"], dev["k"], dev["v"], dev["log_decay"], dev["dy"],
                                         h0=dev["h0"], dh_final=dev["dh"])

    def loss(d):
        y, h = forward(d)
        ly, lh = dev["dy"].double() * y.double(), dev["dh"].double() * h.double()
        return float(ly.sum() + lh.sum()), float(ly.abs().sum() + lh.abs().sum())

    rng = np.random.default_rng(2)
    for name in ("q", "k", "v", "h0"):
        d = torch.from_numpy(rng.standard_normal(dev[name].shape).astype(np.float32)).to(DEV)
        (up, su), (down, sd) = loss(dict(dev, **{name: dev[name] + d})), loss(dict(dev, **{name: dev[name] - d}))
        got = float((g["d" + name].double() * d.double()).sum())
        # outputs of order one off by at most roundings() each
        assert abs((up - down) / 2 - got) < refs.roundings(48, 40, 100) * (su + sd), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,N,P", [(1, 1, 1, 1, 1), (2, 6, 2, 80, 50), (3, 4, 4, 128, 128), (1, 24, 1, 64, 64),
                                       (2, 3, 1, 256, 17), (40, 16, 16, 33, 260)])
def test_step(B, H, G, N, P, dtype):
    for form in ("token", "head"):
        dev, ref = make(B, 1, H, G, N, P, dtype=dtype, form=form, seed=N + P)
        g = dev["log_decay"][:, 0].contiguous() if form == "token" else dev["log_decay"]
        a = (dev["q"][:, 0].contiguous(), dev["k"][:, 0].contiguous(), dev["v"][:, 0].contiguous(), g)
        out = torch.empty_like(dev["h0"])
        y = swimba.linear_attention_step(*a, dev["h0"], state_out=out)
        want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
        b = refs.roundings(N, P, 1)
        close(y, want["y"][:, 0], size["y"][:, 0], b, "y")
        close(out, want["h_final"], size["h_final"], b, "state")
        st = dev["h0"].clone()
        y2 = swimba.linear_attention_step(*a, st, y_dtype=torch.float32)
        assert torch.equal(st, out)
        close(y2, want["y"][:, 0], size["y"][:, 0], b, "y in place")
        call = swimba.PreparedLinearAttentionStep(*a, dev["h0"], state_out=out.zero_())
        assert torch.equal(call(), y) and torch.equal(out, st)


def test_step_misaligned_state():
    dev, ref = make(2, 1, 2, 1, 20, 32, dtype="f32", seed=9)
    buf = torch.empty(dev["h0"].numel() + 1, device=DEV)
    st = buf[1:].view(dev["h0"].shape)
    st.copy_(dev["h0"])
    y = swimba.linear_attention_step(dev["q"][:, 0].contiguous(), dev["k"][:, 0].contiguous(),
                                     dev["v"][:, 0].contiguous(), dev["log_decay"][:, 0].contiguous(), st)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    close(st, want["h_final"], size["h_final"], refs.roundings(20, 32, 1), "state")
    close(y, want["y"][:, 0], size["y"][:, 0], refs.roundings(20, 32, 1), "y")


def test_rows_at_odd_addresses():
    # every operand one element behind an aligned address, odd row widths
    shape = (1, 90, 3, 1, 37, 21)
    for dtype in ("bf16", "f32"):
        dev, ref = make(*shape, dtype=dtype, grad=True, seed=31)
        for n in ("q", "k", "v", "dy"):
            buf = torch.empty(dev[n].numel() + 1, dtype=dev[n].dtype, device=DEV)
            x = buf[1:].view(dev[n].shape)
            x.copy_(dev[n])
            dev[n] = x
        y, h = forward(dev, y_dtype=torch.float32)
        want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
        close(y, want["y"], size["y"], refs.roundings(37, 21, 90), "y")
        check_backward(dev, ref, shape, "f32")


def test_split_sequences_and_steps_agree():
    dev, ref = make(2, 150, 4, 2, 64, 32, dtype="f32", seed=5)
    y, h = forward(dev)
    cut = {n: (x[:, :97].contiguous(), x[:, 97:].contiguous()) for n, x in dev.items() if n != "h0" and x is not None}
    y1, h1 = swimba.linear_attention(*(cut[n][0] for n in ("q", "k", "v", "log_decay")), h0=dev["h0"])
    y2, h2 = swimba.linear_attention(*(cut[n][1] for n in ("q", "k", "v", "log_decay")), h0=h1)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    b = refs.roundings(64, 32, 150 + 64)
    close(torch.cat([y1, y2], 1), want["y"], size["y"], b, "y")
    close(h2, want["h_final"], size["h_final"], b, "h")
    st = dev["h0"].clone()
    for t in range(20):
        yt = swimba.linear_attention_step(*(dev[n][:, t].contiguous() for n in ("q", "k", "v", "log_decay")), st)
        close(yt, want["y"][:, t], size["y"][:, t], refs.roundings(64, 32, 64 * 21), "step %d" % t)


def test_empty():
    dev, _ = make(2, 0, 2, 1, 8, 8, dtype="f32", form="head", grad=True)
    y, h = forward(dev)
    assert y.shape == (2, 0, 2, 8) and torch.equal(h, dev["h0"])
    g = swimba.linear_attention_backward(dev["q"], dev["k"], dev["v"], dev["log_decay"], dev["dy"],
                                         h0=dev["h0"], dh_final=dev["dh"])
    assert torch.equal(g["dh0"], dev["dh"]) and not g["dlog_decay"].any()
    dev, _ = make(0, 5, 2, 1, 8, 8, dtype="f32", form="head", h0=False, grad=True)
    y, h = forward(dev)
    assert y.shape == (0, 5, 2, 8) and h.shape == (0, 2, 8, 8)


def test_deterministic():
    dev, _ = make(2, 700, 8, 2, 64, 64, grad=True, seed=8)
    runs = []
    for _ in range(3):
        y, h = forward(dev)
        g = swimba.linear_attention_backward(dev["q"], dev["k"], dev["v"], dev["log_decay"], dev["dy"],
                                             h0=dev["h0"], dh_final=dev["dh"])
        runs.append([y, h] + list(g.values()))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_captured_and_side_stream():
    dev, _ = make(1, 1000, 4, 2, 64, 64, grad=True, seed=12)

    def both(stream=None):
        y, h = forward(dev, stream=stream)
        g = swimba.linear_attention_backward(dev["q"], dev["k"], dev["v"], dev["log_decay"], dev["dy"],
                                             h0=dev["h0"], dh_final=dev["dh"], stream=stream)
        return [y, h] + list(g.values())

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        again = both()  # eager work between the replays
        torch.cuda.synchronize()
        for a, b, c in zip(want, held, again):
            assert torch.equal(a, b) and torch.equal(a, c), i
    # new inputs in the same buffers
    dev["v"].mul_(0.5)
    graph.replay()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_wrong_arguments():
    dev, _ = make(1, 8, 4, 2, 16, 16)
    q, k, v, g = dev["q"], dev["k"], dev["v"], dev["log_decay"]
    with pytest.raises(ValueError):
        swimba.linear_attention(q, k[:, :4].contiguous(), v, g)
    with pytest.raises(ValueError):
        swimba.linear_attention(q, k, v, g.bfloat16())
    with pytest.raises(ValueError):
        swimba.linear_attention(q.float(), k, v, g)
    with pytest.raises(ValueError):
        swimba.linear_attention(q, k, v.transpose(1, 2), g)
    with pytest.raises(ValueError):
        swimba.linear_attention(q, k, v, g, h0=torch.zeros(1, 4, 16, 8, device=DEV))
    with pytest.raises(swimba.SwimbaError):
        three = torch.zeros(1, 8, 3, 16, dtype=q.dtype, device=DEV)
        swimba.linear_attention(three, three, v, g)
    with pytest.raises(TypeError):
        swimba.linear_attention(q.half(), k.half(), v.half(), g)
    with pytest.raises(ValueError):
        swimba.linear_attention_backward(q, k, v, g, torch.zeros(1, 8, 4, 16, device=DEV))


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 3, 200), (1, 1, 1, 1, 256, 2), (1, 2, 1, 1, 3, 2), (1, 1, 3, 1, 5, 1)], ids=str)
def test_operands_of_less_than_a_pack(shape):
    B, L, H, G, N, P = shape
    for dtype in ("bf16", "f32"):
        dev, ref = make(*shape, dtype=dtype, grad=True, seed=41)
        y, h = forward(dev, y_dtype=torch.float32)
        want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
        close(y, want["y"], size["y"], refs.roundings(N, P, L), "y")
        close(h, want["h_final"], size["h_final"], refs.roundings(N, P, L), "h")
        check_backward(dev, ref, shape, "f32")


@pytest.mark.parametrize("dtype,N,P", [("bf16", 64, 64), ("f32", 33, 20), ("bf16", 128, 96)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_never_reach_earlier_tokens(dtype, N, P, bad):
    # a padded batch may hold anything behind its last token, and the token before
    # it lies in the same chunk
    L, s = 150, 77
    dev, ref = make(1, L, 2, 1, N, P, dtype=dtype, form="token", h0=True, seed=51)
    y, h = forward(dev)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    for name in ("q", "k", "v", "log_decay"):
        if name == "log_decay" and bad < 0:
            continue  # clears the state
        d = {n: x.clone() for n, x in dev.items() if x is not None}
        d[name][0, s].view(-1)[1] = bad  # key 1, value (head 0, column 1) or head 1
        y2, h2 = forward(d)
        if name == "log_decay":
            # that chunk of that head takes the decays pair by pair instead of as two
            # factors: other roundings, each result within the same bound of the exact
            # one as any output
            close(y2[:, :s], want["y"][:, :s], size["y"][:, :s], refs.roundings(N, P, L, dtype == "f32"), name)
        else:
            assert torch.equal(y2[:, :s], y[:, :s]), name
        if name == "q":
            keep = torch.arange(L, device=DEV) != s
            assert torch.equal(y2[:, keep], y[:, keep]) and torch.equal(h2, h)
            assert not torch.isfinite(y2[:, s]).any()
        elif name == "v":
            assert not torch.isfinite(y2[0, s:, 0, 1]).any() and not torch.isfinite(h2[0, 0, :, 1]).any()
            # the columns next to it go with it, 32 together; others and other heads do not
            assert torch.equal(y2[0, :, 0, 32:], y[0, :, 0, 32:]) and torch.equal(y2[0, :, 1], y[0, :, 1])
            assert torch.equal(h2[0, 0, :, 32:], h[0, 0, :, 32:]) and torch.equal(h2[0, 1], h[0, 1])
        elif name == "k":
            assert not torch.isfinite(y2[:, s:]).any() and not torch.isfinite(h2[0, :, 1]).any()
        else:
            assert not torch.isfinite(y2[0, s:, 1]).any() and torch.equal(y2[0, :, 0], y[0, :, 0])


def test_non_finite_gradients_stay_behind():
    # dy of a token with rubbish reaches dq of that token and what came before it,
    # not dq of other tokens; dk and dv of later tokens stay as they are
    L, s = 100, 41
    dev, _ = make(1, L, 2, 2, 32, 32, dtype="bf16", grad=True, seed=52)
    a = [dev[n] for n in ("q", "k", "v", "log_decay")]
    g = swimba.linear_attention_backward(*a, dev["dy"], h0=dev["h0"], dh_final=dev["dh"])
    dy = dev["dy"].clone()
    dy[0, s, 0, 3] = float("nan")
    b = swimba.linear_attention_backward(*a, dy, h0=dev["h0"], dh_final=dev["dh"])
    keep = torch.arange(L, device=DEV) != s
    assert torch.equal(g["dq"][:, keep], b["dq"][:, keep]) and not torch.isfinite(b["dq"][0, s, 0]).any()
    for n in ("dk", "dv"):
        assert torch.equal(g[n][:, s + 1:], b[n][:, s + 1:]) and torch.equal(g[n][:, :, 1], b[n][:, :, 1]), n


def test_fp32_inputs_bf16_results():
    dev, ref = make(2, 90, 4, 2, 40, 24, dtype="f32", seed=61)
    y, h = forward(dev, y_dtype=torch.bfloat16)
    want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
    close(y, want["y"], size["y"], refs.roundings(40, 24, 90, False), "y")


def test_large_and_small_magnitudes():
    for scale in (1e5, 1e-6):
        dev, ref = make(1, 140, 2, 1, 32, 32, dtype="f32", seed=71)
        for n in ("q", "k", "v", "h0"):
            f = scale * scale if n == "h0" else scale
            dev[n] = dev[n] * f
            ref[n] = dev[n].double().cpu().numpy()
        y, h = forward(dev)
        want, size = refs.attention(*args(ref)), refs.attention_sizes(*args(ref))
        close(y, want["y"], size["y"], refs.roundings(32, 32, 140), "y")
        close(h, want["h_final"], size["h_final"], refs.roundings(32, 32, 140), "h")


@pytest.mark.parametrize("L", [100, 1500])  # whole walks and segments
def test_states_in_place(L):
    dev, _ = make(1, L, 4, 2, 64, 64, grad=True, seed=21)
    grads = dict(h0=dev["h0"], dh_final=dev["dh"])
    ops = [dev[n] for n in ("q", "k", "v", "log_decay")]
    y, h = forward(dev)
    want = swimba.linear_attention_backward(*ops, dev["dy"], **grads)
    st = dev["h0"].clone()
    y2, h2 = swimba.linear_attention(*ops, h0=st, h_final=st)
    assert torch.equal(y, y2) and torch.equal(h, h2) and h2 is st
    adj = dev["dh"].clone()
    got = swimba.linear_attention_backward(*ops, dev["dy"], h0=dev["h0"], dh_final=adj, out={"dh0": adj})
    assert all(torch.equal(want[n], got[n]) for n in want)

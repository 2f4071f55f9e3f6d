"""Norms of queries and keys with their rotation against 64 bits.  An output may be off by half
a step of its type and, relative to the sums over absolute values, by fp32 half steps: N / 8
for the lane's part of a row's sum of squares and 5 for the lanes (halved by the root), 16
for root, cosines and sines (2 each) and the products."""
import numpy as np
import pytest
import torch

import delta_refs as refs
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(T, Hq, Hk, N, R, dtype, weights, seed=0, far=0):
    gen = torch.Generator().manual_seed(seed)

    def f(*s):
        return torch.randn(*s, generator=gen)

    t = {"q": f(T, Hq, N), "k": f(T, Hk, N), "dq": f(T, Hq, N), "dk": f(T, Hk, N)}
    t = {n: x.to(DT[dtype]) for n, x in t.items()}
    t["wq"], t["wk"] = (1 + 0.2 * f(N) if weights else None for _ in range(2))
    t["pos"] = (far + torch.arange(T) * 3).to(torch.int32) if R else None
    t["rates"] = torch.pow(10000.0, -torch.arange(0, R, 2, dtype=torch.float64) / R).float() if R else None
    return t


def plain(x):
    return None if x is None else x.double().numpy() if x.dtype != torch.int32 else x.numpy()


def call(t, how, back=False, **kw):
    d = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    args = dict(wq=d["wq"], wk=d["wk"], positions=d["pos"], rates=d["rates"], **how)
    if back:
        return swimba.norm_rotate_backward(d["q"], d["k"], d["dq"], d["dk"], **args, **kw)
    return swimba.norm_rotate(d["q"], d["k"], **args, **kw)


def reference(t, norm, pairs, eps=1e-6, q_scale=1.0):
    return refs.norm_rotate(*(plain(t[n]) for n in ("q", "k", "wq", "wk", "pos", "rates")), norm, pairs, eps, q_scale,
                            plain(t["dq"]), plain(t["dk"]))


def close(got, want, size, steps, what):
    g = got.double().cpu().numpy().reshape(want.shape)
    allow = steps * refs.U0 * size + refs.HALF[got.dtype] * (1 + 2.0 ** -8) * np.abs(want) + 1e-30
    bad = ~(np.abs(g - want) <= allow)
    assert not bad.any(), "%s: %d of %d off, worst %.3g times the bound" % (what, bad.sum(), bad.size, np.nanmax(np.abs(g - want) / allow))


def steps(N):
    return N / 16 + 2.5 + 16


SHAPES = [  # T, Hq, Hk, N, R
    (1, 1, 1, 1, 0), (1, 2, 1, 2, 2), (3, 4, 2, 16, 16), (5, 3, 3, 64, 64), (7, 8, 1, 128, 32), (4, 6, 2, 80, 48),
    (9, 2, 2, 37, 10), (2, 1, 5, 512, 512), (70, 5, 3, 24, 24), (33, 1, 1, 256, 0), (6, 7, 2, 50, 50), (300, 40, 8, 64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_both_ways(shape, dtype):
    T, Hq, Hk, N, R = shape
    for i, (norm, pairs) in enumerate((n, p) for n in ("rms", "l2") for p in ("halves", "neighbours")):
        t = make(*shape, dtype, i % 2 == 0, seed=i + N)
        how = dict(norm=norm, pairs=pairs, q_scale=0.25)
        want, size = reference(t, norm, pairs, q_scale=0.25)
        odt = "f32" if i == 1 else dtype
        q, k = call(t, how, out_dtype=DT[odt])
        close(q, want["q"], size["q"], steps(N), "q")
        close(k, want["k"], size["k"], steps(N), "k")
        g = call(t, how, back=True, grad_dtype=DT[odt])
        # the row's second sum, and the first one's root again
        for n in ("dq", "dk"):
            close(g[n], want[n], size[n], 2 * steps(N) + N / 8, n)
        for n, heads in (("dwq", Hq), ("dwk", Hk)):
            if t["w" + n[-1]] is None:
                assert g[n] is None
            else:  # a thread's rows in fp32, the workgroup's, then 64 bits
                close(g[n], want[n], size[n], steps(N) + T * heads / 16 + 20, n)


def test_in_place_and_parts_of_one_projection():
    for pairs in ("halves", "neighbours"):
        for N, R in ((64, 64), (50, 20)):
            t = make(40, 4, 2, N, R, "bf16", True, seed=1)
            how = dict(norm="rms", pairs=pairs)
            want = call(t, how)
            q, k = t["q"].to(DEV), t["k"].to(DEV)
            args = dict(wq=t["wq"].to(DEV), wk=t["wk"].to(DEV), positions=t["pos"].to(DEV), rates=t["rates"].to(DEV), **how)
            got = swimba.norm_rotate(q, k, q_out=q, k_out=k, **args)
            assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
            # rows of one buffer, at an odd address
            flat = torch.full((40 * (6 * N + 3) + 1,), float("nan"), dtype=torch.bfloat16, device=DEV)[1:].view(40, 6 * N + 3)
            flat[:, :4 * N] = t["q"].to(DEV).flatten(1)
            flat[:, 4 * N:6 * N] = t["k"].to(DEV).flatten(1)
            q, k = flat[:, :4 * N].unflatten(-1, (4, N)), flat[:, 4 * N:6 * N].unflatten(-1, (2, N))
            got = swimba.norm_rotate(q, k, **args)
            assert got[0].is_contiguous() and all(torch.equal(a, b) for a, b in zip(got, want))
            dq, dk = t["dq"].to(DEV), t["dk"].to(DEV)
            g = swimba.norm_rotate_backward(q, k, dq, dk, **args, grad_dtype=torch.bfloat16)
            g2 = call(t, how, back=True, grad_dtype=torch.bfloat16)
            assert all(torch.equal(g[n], g2[n]) for n in g)
            g3 = swimba.norm_rotate_backward(q, k, dq, dk, **args, grad_dtype=torch.bfloat16, out={"dq": dq, "dk": dk})
            assert g3["dq"] is dq and all(torch.equal(g3[n], g2[n]) for n in g2)


def test_leading_dimensions():
    t = make(12, 3, 2, 32, 16, "f32", True, seed=2)
    how = dict(norm="l2", pairs="halves")
    want = call(t, how)
    shaped = {n: x.reshape(3, 4, *x.shape[1:]) if n in ("q", "k", "pos", "dq", "dk") else x for n, x in t.items()}
    got = call(shaped, how)
    assert got[0].shape == (3, 4, 3, 32) and all(torch.equal(a.flatten(0, 1), b) for a, b in zip(got, want))
    one = {n: x[0] if n in ("q", "k", "pos", "dq", "dk") else x for n, x in t.items()}  # no leading dimension
    got = call(one, how)
    assert torch.equal(got[0], want[0][0])
    # rows of a sliced sequence
    q, k = (x.to(DEV).reshape(3, 4, *x.shape[1:])[:, 1:3] for x in (t["q"], t["k"]))
    with pytest.raises(ValueError):
        swimba.norm_rotate(q, k)  # tokens not equally far apart


@pytest.mark.parametrize("far", [0, 1000000, 2000000000])
def test_far_positions(far):
    t = make(20, 2, 1, 32, 32, "f32", False, seed=3, far=far)
    want, size = reference(t, "rms", "halves")
    q, k = call(t, dict(norm="rms", pairs="halves"))
    # an angle of 2e9 in 64 bits is off by 2^-53 of it, three times
    close(q, want["q"], size["q"], steps(32) + 3 * far * 2.0 ** -53 / refs.U0, "q")
    close(k, want["k"], size["k"], steps(32) + 3 * far * 2.0 ** -53 / refs.U0, "k")
    t["pos"] = -t["pos"]  # backwards
    want, size = reference(t, "rms", "halves")
    q, _ = call(t, dict(norm="rms", pairs="halves"))
    close(q, want["q"], size["q"], steps(32) + 3 * far * 2.0 ** -53 / refs.U0, "q")


def test_rows_of_zero_small_and_large_values():
    t = make(4, 2, 1, 64, 64, "f32", True, seed=4)
    t["q"][0] = 0
    t["q"][1] *= 1e-20
    t["q"][2] *= 1e15
    want, size = reference(t, "l2", "halves")
    how = dict(norm="l2", pairs="halves")
    q, k = call(t, how)
    assert not q[0].any()
    close(q, want["q"], size["q"], steps(64), "q")
    g = call(t, how, back=True)
    close(g["dq"], want["dq"], size["dq"], 2 * steps(64) + 8, "dq")


def test_non_finite_values_stay_in_their_row():
    t = make(6, 3, 2, 48, 16, "bf16", True, seed=5)
    how = dict(norm="rms", pairs="neighbours")
    q, k = call(t, how)
    for bad in (float("nan"), float("inf")):
        b = {n: None if x is None else x.clone() for n, x in t.items()}
        b["q"][2, 1, 7] = bad
        q2, k2 = call(b, how)
        assert torch.isnan(q2[2, 1, 6:8]).any() and torch.equal(k2, k)
        keep = torch.ones(6, 3, dtype=torch.bool)
        keep[2, 1] = False
        assert torch.equal(q2[keep.to(DEV)], q[keep.to(DEV)])


def test_empty_and_wrong_arguments():
    t = make(0, 2, 1, 16, 8, "bf16", True)
    how = dict(norm="rms", pairs="halves")
    q, k = call(t, how)
    assert q.shape == (0, 2, 16) and k.shape == (0, 1, 16)
    g = call(t, how, back=True)
    assert not g["dwq"].any() and not g["dwk"].any()
    t = make(4, 2, 1, 16, 8, "bf16", True)
    q, k = t["q"].to(DEV), t["k"].to(DEV)
    pos, rates = t["pos"].to(DEV), t["rates"].to(DEV)
    for bad in (dict(norm="max"), dict(pairs="thirds"), dict(positions=pos), dict(rates=rates),
                dict(positions=pos[:3], rates=rates), dict(positions=pos.long(), rates=rates),
                dict(wq=torch.ones(8, device=DEV)), dict(wk=torch.ones(16, device=DEV, dtype=torch.bfloat16)),
                dict(q_out=torch.empty(4, 2, 8, device=DEV))):
        with pytest.raises(ValueError):
            swimba.norm_rotate(q, k, **bad)
    with pytest.raises(ValueError):
        swimba.norm_rotate(q, k[:3])
    with pytest.raises(ValueError):
        swimba.norm_rotate(q, k.float())
    with pytest.raises(ValueError):
        swimba.norm_rotate(q.transpose(1, 2), k)
    with pytest.raises(TypeError):
        swimba.norm_rotate(q.half(), k.half())
    with pytest.raises(swimba.SwimbaError):
        swimba.norm_rotate(q, k, eps=0.0)
    with pytest.raises(swimba.SwimbaError):
        swimba.norm_rotate(q, k, positions=pos, rates=torch.ones(9, device=DEV))  # more than a head has
    with pytest.raises(ValueError):
        swimba.norm_rotate_backward(q, k, q.float(), k)


def test_deterministic_captured_and_side_stream():
    t = make(3000, 6, 2, 64, 64, "bf16", True, seed=6)
    d = {n: x.to(DEV) for n, x in t.items()}
    args = dict(wq=d["wq"], wk=d["wk"], positions=d["pos"], rates=d["rates"])

    def both(stream=None):
        out = swimba.norm_rotate(d["q"], d["k"], **args, stream=stream)
        return list(out) + list(swimba.norm_rotate_backward(d["q"], d["k"], d["dq"], d["dk"], **args, stream=stream).values())

    want = both()
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
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
        for x in held:
            x.zero_()
        graph.replay()
        again = both()
        torch.cuda.synchronize()
        for a, b, c in zip(want, held, again):
            assert torch.equal(a, b) and torch.equal(a, c), i

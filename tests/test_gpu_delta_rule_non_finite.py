"""Where an infinity or a NaN of an input goes in the delta rule's gradients: never lost where the
forward pass carries it, and not in what it has no part in."""
import pytest
import torch

import delta_refs as refs
from parameter_space_moe_amd import swimba
from test_gpu_delta_rule import OPS, backward, close, forward, make, to_dev, wide

pytestmark = pytest.mark.gpu

CASES = [("bf16", 64, 64, 150), ("f32", 33, 20, 150), ("bf16", 128, 96, 1500), ("f32", 48, 70, 1100), ("bf16", 200, 24, 2000)]
BAD = [float("nan"), float("inf"), -float("inf")]


def none_finite(x, what):
    assert not torch.isfinite(x).any(), what


def same(a, b, what):
    assert torch.equal(a, b), what


@pytest.mark.parametrize("dtype,N,P,L", CASES)
@pytest.mark.parametrize("bad", BAD)
def test_key_beta_or_decay(dtype, N, P, L, bad):
    s = L // 2 + 2
    t = make(1, L, 2, 1, N, P, dtype=dtype, seed=91)
    d = to_dev(t)
    g = backward(d)
    a = wide(t, *OPS, "h0", "dy", "dh")
    want, allow = refs.delta(*a), refs.bounds(dtype == "f32", *a)
    behind = (s // 64 + 1) * 64  # of the value's chunk
    for name in ("k", "g", "beta"):
        if name == "g" and bad < 0:
            continue  # clears the state
        e = {n: x.clone() for n, x in d.items()}
        e[name][0, s].view(-1)[1] = bad  # key 1 of both heads, or head 1
        got = backward(e)
        heads = [0, 1] if name == "k" else [1]
        assert torch.isnan(got["dq"][:, s:]).all() and torch.isnan(got["dk"]).all(), name
        close(got["dq"][:, :s], want["dq"][:, :s], allow["dq"][:, :s], name)
        for n in ("dbeta", "dlog_decay"):
            assert torch.isnan(got[n][:, :, heads]).all(), (name, n)
        assert torch.isnan(got["dv"][:, :s + 1, heads]).all() and torch.isnan(got["dh0"][:, heads]).all(), name
        same(got["dv"][:, behind:], g["dv"][:, behind:], name)
        if heads == [1]:
            for n in ("dv", "dbeta", "dlog_decay"):
                same(got[n][:, :, 0], g[n][:, :, 0], (name, n))
            same(got["dh0"][:, 0], g["dh0"][:, 0], name)


@pytest.mark.parametrize("dtype,N,P,L", CASES)
@pytest.mark.parametrize("bad", BAD)
def test_value_query_or_slope(dtype, N, P, L, bad):
    s = L // 2 + 2
    d = to_dev(make(1, L, 2, 1, N, P, dtype=dtype, seed=92))
    g = backward(d)
    behind, other = (s // 64 + 1) * 64, torch.arange(P, device="cuda") != 1
    keep = torch.arange(L, device="cuda") != s
    for name in ("v", "q", "dy"):
        e = {n: x.clone() for n, x in d.items()}
        e[name][0, s].view(-1)[1] = bad  # head 0, column 1; query 1
        got = backward(e)
        if name == "v":
            for n in ("dq", "dk"):
                none_finite(got[n][:, s:], n)
                same(got[n][:, :s], g[n][:, :s], n)
            for n in ("dbeta", "dlog_decay"):
                none_finite(got[n][:, s:, 0], n)
                same(got[n][:, :s, 0], g[n][:, :s, 0], n)
                same(got[n][:, :, 1], g[n][:, :, 1], n)
            same(got["dv"], g["dv"], "dv")
            same(got["dh0"], g["dh0"], "dh0")
            continue
        heads = [0, 1] if name == "q" else [0]
        columns = slice(None) if name == "q" else 1
        for n in ("dbeta", "dlog_decay"):
            none_finite(got[n][:, :s + 1, heads], n)
        for n in ("dk", "dbeta", "dlog_decay", "dv"):
            same(got[n][:, behind:], g[n][:, behind:], n)
        none_finite(got["dk"][:, :s + 1], name)
        none_finite(got["dv"][:, :s + 1, heads][..., columns], name)
        none_finite(got["dh0"][:, heads][..., columns], name)
        same(got["dq"][:, keep], g["dq"][:, keep], name)
        if name == "dy":
            none_finite(got["dq"][:, s], name)
            same(got["dv"][:, :, 0][..., other], g["dv"][:, :, 0][..., other], name)
            same(got["dh0"][:, 0][..., other], g["dh0"][:, 0][..., other], name)
            for n in ("dv", "dbeta", "dlog_decay"):
                same(got[n][:, :, 1], g[n][:, :, 1], n)
            same(got["dh0"][:, 1], g["dh0"][:, 1], name)


@pytest.mark.parametrize("bad", BAD[:2])
def test_a_decay_per_head(bad):
    d = to_dev(make(2, 300, 4, 2, 64, 40, form="head", seed=95))
    g = backward(d)
    d["g"][1] = bad
    got = backward(d)
    assert torch.isnan(got["dlog_decay"][1]) and torch.isnan(got["dh0"][:, 1]).all()
    for n in ("dv", "dbeta"):
        assert torch.isnan(got[n][:, :, 1]).all(), n
        same(got[n][:, :, [0, 2, 3]], g[n][:, :, [0, 2, 3]], n)
    same(got["dlog_decay"][[0, 2, 3]], g["dlog_decay"][[0, 2, 3]], "dlog_decay")
    for n in ("dq", "dk"):
        assert torch.isnan(got[n][:, :, 0]).all(), n
        same(got[n][:, :, 1], g[n][:, :, 1], n)


@pytest.mark.parametrize("dtype,N,P,L,s", [("bf16", 64, 64, 150, 70), ("f32", 33, 20, 150, 128), ("bf16", 128, 96, 1500, 801),
                                           ("f32", 48, 70, 1100, 1), ("bf16", 200, 24, 2000, 640)])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_anything_behind_the_last_token(dtype, N, P, L, s, fill):
    # dy and dL/dh_final are zero there: the gradients are those of the tokens before
    t = make(1, L, 4, 2, N, P, dtype=dtype, seed=93)
    d = to_dev(t)
    for n in ("k", "v", "g", "beta"):
        d[n][:, s:] = fill
    d["dy"][:, s:] = 0
    got = backward(dict(d, dh=None))
    a = [None if x is None else x if n == "h0" else x[:, :s] for n, x in zip(OPS + ("h0", "dy"), wide(t, *OPS, "h0", "dy"))]
    want, allow = refs.delta(*a), refs.bounds(dtype == "f32", *a)
    for n in ("dq", "dk", "dv", "dbeta", "dlog_decay"):
        close(got[n][:, :s], want[n], allow[n], n)
    close(got["dh0"], want["dh0"], allow["dh0"], "dh0")
    for n in ("dq", "dk", "dbeta", "dlog_decay"):
        assert torch.isnan(got[n][:, s:]).all(), n
    # one head's rubbish is not the others'
    d = to_dev(t)
    d["beta"][:, s:, 1] = fill
    d["dy"][:, s:, 1] = 0
    b = backward(dict(d, dh=None))
    close(b["dv"][:, :s, 1], want["dv"][:, :, 1], allow["dv"][:, :, 1], "dv")
    close(b["dbeta"][:, :s, 1], want["dbeta"][:, :, 1], allow["dbeta"][:, :, 1], "dbeta")
    d["beta"] = t["beta"].to("cuda")
    c = backward(dict(d, dh=None))
    for n in ("dv", "dbeta", "dlog_decay"):
        same(b[n][:, :, [0, 2, 3]], c[n][:, :, [0, 2, 3]], n)


def test_nothing_grows_out_of_nothing():
    # a state of zeros through segments whose transitions are beyond fp32
    t = make(1, 2000, 1, 1, 32, 16, dtype="f32", h0=False, seed=94)
    t["g"][:, :1600] = 1.0
    t["v"][:, :1600] = 0
    y, h = forward(to_dev(t), y_dtype=torch.float32)
    assert not y[:, :1600].any()
    a = [x[:, 1600:] for x in wide(t, *OPS)]
    want, allow = refs.delta(*a), refs.bounds(True, *a)
    close(y[:, 1600:], want["y"], allow["y"], "y")
    close(h, want["h_final"], allow["h_final"], "h_final")

"""The delta rule and the norms of queries and keys without a GPU: struct layout, refusals
before anything is launched, workspace sizes, and the 64-bit references against
differences."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import delta_refs as refs
from parameter_space_moe_amd import swimba as sw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x100000  # never read: every call below is refused on the host


@pytest.fixture(scope="module")
def lib():
    return sw.load()


STRUCTS = (("swimba_delta_rule_args", sw.DeltaRuleArgs), ("swimba_delta_rule_grad_args", sw.DeltaRuleGradArgs),
           ("swimba_delta_rule_step_args", sw.DeltaRuleStepArgs), ("swimba_norm_rotate_args", sw.NormRotateArgs),
           ("swimba_norm_rotate_grad_args", sw.NormRotateGradArgs))


def test_structs_match_header(tmp_path):
    src = ['#include <cstddef>', '#include <cstdio>', '#include "swimba.h"', 'int main() {']
    for c, cls in STRUCTS:
        src.append('std::printf("%s sizeof %%zu\\n", sizeof(%s));' % (c, c))
        for f, _ in cls._fields_:
            src.append('std::printf("%s %s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f))
    src.append("return 0; }")
    f = tmp_path / "layout.cpp"
    f.write_text("\n".join(src))
    exe = tmp_path / "layout"
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), str(f), "-o", str(exe)], check=True)
    got = {tuple(l.split()[:2]): int(l.split()[2]) for l in
           subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()}
    for c, cls in STRUCTS:
        assert got[(c, "sizeof")] == ctypes.sizeof(cls)
        for name, _ in cls._fields_:
            assert got[(c, name)] == getattr(cls, name).offset, (c, name)


OPERANDS = ("q", "k", "v", "log_decay", "beta")


def delta_args(**kw):
    a = sw.DeltaRuleArgs()
    a.B, a.L, a.H, a.G, a.N, a.P = 1, 8192, 2, 1, 64, 64
    a.in_dtype, a.y_dtype, a.decay_form = sw.BF16, sw.BF16, sw.DECAY_TOKEN
    for f in OPERANDS + ("y",):
        setattr(a, f, FAKE)
    for f, v in kw.items():
        setattr(a, f, v)
    return a


def grad_args(fwd=None, **kw):
    g = sw.DeltaRuleGradArgs()
    g.fwd = delta_args(**(fwd or {}))
    g.grad_dtype = sw.BF16
    for f in ("dy", "dq", "dk", "dv", "dlog_decay", "dbeta"):
        setattr(g, f, FAKE)
    for f, v in kw.items():
        setattr(g, f, v)
    return g


BAD = ([(f, -1, sw.EINVAL) for f in "BL"] + [(f, 0, sw.EINVAL) for f in "HGNP"] +
       [("G", 3, sw.EINVAL), ("in_dtype", 7, sw.EINVAL), ("y_dtype", 7, sw.EINVAL), ("decay_form", 2, sw.EINVAL),
        ("N", 257, sw.EUNSUPPORTED), ("L", (1 << 30) + 1, sw.EUNSUPPORTED), ("B", 1 << 24, sw.EUNSUPPORTED),
        ("L", 1 << 30, sw.EUNSUPPORTED), ("P", 1 << 23, sw.EUNSUPPORTED)] +
       [(f, None, sw.EINVAL) for f in OPERANDS] + [(f, FAKE + 1, sw.EINVAL) for f in "qkv"])


@pytest.mark.parametrize("field,value,status", BAD)
def test_delta_rule_refuses(lib, field, value, status):
    a = delta_args(**{field: value})
    assert lib.swimba_delta_rule(ctypes.byref(a), None, 0, None) == status
    g = grad_args({field: value})
    assert lib.swimba_delta_rule_backward(ctypes.byref(g), None, 0, None) == status


def test_delta_rule_refuses_wide_fp32_keys(lib):
    for N, ok in ((128, True), (129, False)):
        a = delta_args(in_dtype=sw.F32, N=N)
        want = sw.EWORKSPACE if ok else sw.EUNSUPPORTED
        assert lib.swimba_delta_rule(ctypes.byref(a), None, 0, None) == want
        assert (lib.swimba_delta_rule_workspace_size(ctypes.byref(a)) > 0) == ok


@pytest.mark.parametrize("L", (0, 1, 2, 64, 65))
def test_delta_rule_refuses_wide_fp32_keys_at_any_length(lib, L):
    for N, ok in ((128, True), (129, False), (256, False)):
        a = delta_args(in_dtype=sw.F32, N=N, L=L)
        want = (sw.OK if L == 0 else sw.EWORKSPACE) if ok else sw.EUNSUPPORTED
        assert lib.swimba_delta_rule(ctypes.byref(a), None, 0, None) == want, N
        if ok and L == 0:
            continue  # (writes a zero dlog_decay where there is one per head)
        g = grad_args({"in_dtype": sw.F32, "N": N, "L": L})
        assert lib.swimba_delta_rule_backward(ctypes.byref(g), None, 0, None) == want, N


def test_delta_rule_backward_refuses_more_chunks_than_a_launch_holds(lib):
    """512 threads per chunk and head: the forward takes twice as many."""
    for B, ok in (((1 << 22) - 1, True), (1 << 22, False)):
        fwd = {"B": B, "L": 64, "H": 2, "N": 8, "P": 8}
        assert lib.swimba_delta_rule(ctypes.byref(delta_args(**fwd)), None, 0, None) == sw.EWORKSPACE
        want = sw.EWORKSPACE if ok else sw.EUNSUPPORTED
        assert lib.swimba_delta_rule_backward(ctypes.byref(grad_args(fwd)), None, 0, None) == want, B


def test_delta_rule_refuses_workspace(lib):
    a = delta_args()
    need = lib.swimba_delta_rule_workspace_size(ctypes.byref(a))
    assert need > 0
    for ws, n in ((None, 0), (FAKE, need - 1), (FAKE + 128, need)):
        assert lib.swimba_delta_rule(ctypes.byref(a), ws, n, None) == sw.EWORKSPACE
    assert lib.swimba_delta_rule(None, None, 0, None) == sw.EINVAL
    assert lib.swimba_delta_rule_workspace_size(None) == 0
    assert lib.swimba_delta_rule(ctypes.byref(delta_args(y=None)), FAKE, need, None) == sw.EINVAL
    for f in ("dy", "dq", "dk", "dv", "dlog_decay", "dbeta"):
        g = grad_args(**{f: None})
        assert lib.swimba_delta_rule_backward(ctypes.byref(g), None, 0, None) == sw.EINVAL, f
    assert lib.swimba_delta_rule_backward(ctypes.byref(grad_args(grad_dtype=3)), None, 0, None) == sw.EINVAL
    assert lib.swimba_delta_rule_backward(ctypes.byref(grad_args(dq=FAKE + 1)), None, 0, None) == sw.EINVAL
    assert lib.swimba_delta_rule_backward(None, None, 0, None) == sw.EINVAL
    g = grad_args()
    need = lib.swimba_delta_rule_backward_workspace_size(ctypes.byref(g))
    for ws, n in ((None, 0), (FAKE, need - 1), (FAKE + 128, need)):
        assert lib.swimba_delta_rule_backward(ctypes.byref(g), ws, n, None) == sw.EWORKSPACE
    # without tokens nothing is needed
    assert lib.swimba_delta_rule_workspace_size(ctypes.byref(delta_args(L=0))) == 0
    assert lib.swimba_delta_rule_backward_workspace_size(ctypes.byref(grad_args({"B": 0}))) == 0


def test_delta_rule_step_refuses(lib):
    def step(**kw):
        a = sw.DeltaRuleStepArgs()
        a.B, a.H, a.G, a.N, a.P = 2, 4, 2, 16, 16
        a.in_dtype, a.y_dtype, a.decay_form = sw.BF16, sw.F32, sw.DECAY_HEAD
        for f in OPERANDS + ("state", "y"):
            setattr(a, f, FAKE)
        for f, v in kw.items():
            setattr(a, f, v)
        return lib.swimba_delta_rule_step(ctypes.byref(a), None)

    for f in OPERANDS + ("state", "y"):
        assert step(**{f: None}) == sw.EINVAL, f
    for kw in ({"B": -1}, {"H": 0}, {"G": 3}, {"N": 0}, {"P": 0}, {"in_dtype": 5}, {"decay_form": 9}, {"q": FAKE + 1}):
        assert step(**kw) == sw.EINVAL, kw
    assert step(N=300) == sw.EUNSUPPORTED
    assert step(B=1 << 20, H=4, P=64) == sw.EUNSUPPORTED  # threads of a launch
    assert lib.swimba_delta_rule_step(None, None) == sw.EINVAL
    assert step(B=0) == sw.OK


def norm_args(**kw):
    a = sw.NormRotateArgs()
    a.T, a.Hq, a.Hk, a.N, a.R = 8, 4, 2, 16, 8
    a.in_dtype, a.out_dtype, a.norm, a.pairs, a.eps, a.q_scale = sw.BF16, sw.F32, 0, 1, 1e-6, 1.0
    for f in ("q", "k", "positions", "rates", "q_out", "k_out"):
        setattr(a, f, FAKE)
    for f, v in kw.items():
        setattr(a, f, v)
    return a


NORM_BAD = ([(f, 0, sw.EINVAL) for f in ("Hq", "Hk", "N")] + [(f, None, sw.EINVAL) for f in ("q", "k", "positions", "rates")] +
            [("T", -1, sw.EINVAL), ("R", -2, sw.EINVAL), ("R", 7, sw.EINVAL), ("R", 18, sw.EINVAL), ("in_dtype", 4, sw.EINVAL),
             ("norm", 2, sw.EINVAL), ("pairs", -1, sw.EINVAL), ("eps", 0.0, sw.EINVAL), ("eps", -1.0, sw.EINVAL),
             ("eps", float("nan"), sw.EINVAL), ("eps", float("inf"), sw.EINVAL), ("q_stride", 63, sw.EINVAL),
             ("k_stride", -32, sw.EINVAL), ("N", 513, sw.EUNSUPPORTED), ("Hq", 1 << 16, sw.EUNSUPPORTED),
             ("T", (1 << 31) + 1, sw.EUNSUPPORTED), ("q", FAKE + 1, sw.EINVAL)])


@pytest.mark.parametrize("field,value,status", NORM_BAD)
def test_norm_rotate_refuses(lib, field, value, status):
    a = norm_args(**{field: value})
    assert lib.swimba_norm_rotate(ctypes.byref(a), None) == status
    g = sw.NormRotateGradArgs()
    g.fwd = a
    g.grad_dtype = sw.F32
    for f in ("dq_out", "dk_out", "dq", "dk", "dwq"):
        setattr(g, f, FAKE)
    assert lib.swimba_norm_rotate_backward(ctypes.byref(g), None, 0, None) == status


def test_norm_rotate_refuses_results_and_workspace(lib):
    for f in ("q_out", "k_out"):
        assert lib.swimba_norm_rotate(ctypes.byref(norm_args(**{f: None})), None) == sw.EINVAL
        assert lib.swimba_norm_rotate(ctypes.byref(norm_args(**{f: FAKE + 2})), None) == sw.EINVAL
    assert lib.swimba_norm_rotate(ctypes.byref(norm_args(out_dtype=9)), None) == sw.EINVAL
    assert lib.swimba_norm_rotate(None, None) == sw.EINVAL
    assert lib.swimba_norm_rotate(ctypes.byref(norm_args(T=0)), None) == sw.OK

    def grad(**kw):
        g = sw.NormRotateGradArgs()
        g.fwd = norm_args()
        g.grad_dtype = sw.BF16
        for f in ("dq_out", "dk_out", "dq", "dk", "dwq", "dwk"):
            setattr(g, f, FAKE)
        for f, v in kw.items():
            setattr(g, f, v)
        return g

    for f in ("dq_out", "dk_out", "dq", "dk"):
        assert lib.swimba_norm_rotate_backward(ctypes.byref(grad(**{f: None})), None, 0, None) == sw.EINVAL, f
    assert lib.swimba_norm_rotate_backward(ctypes.byref(grad(grad_dtype=2)), None, 0, None) == sw.EINVAL
    assert lib.swimba_norm_rotate_backward(None, None, 0, None) == sw.EINVAL
    need = lib.swimba_norm_rotate_backward_workspace_size(ctypes.byref(grad()))
    assert need > 0
    for ws, n in ((None, 0), (FAKE, need - 1), (FAKE + 8, need)):
        assert lib.swimba_norm_rotate_backward(ctypes.byref(grad()), ws, n, None) == sw.EWORKSPACE
    assert lib.swimba_norm_rotate_backward_workspace_size(ctypes.byref(grad(dwq=None, dwk=None))) == 0


def test_host_tensors_are_refused():
    q = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError):
        sw.delta_rule(q, q, q, torch.zeros(2), torch.zeros(1, 4, 2))
    with pytest.raises(ValueError):
        sw.delta_rule_step(q[:, 0], q[:, 0], q[:, 0], torch.zeros(2), torch.zeros(1, 2), torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError):
        sw.norm_rotate(q, q)


def test_reference_gradients_are_differences():
    gen = torch.Generator().manual_seed(3)

    def f(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    ops = {"q": f(1, 9, 2, 4), "k": 0.6 * f(1, 9, 2, 4), "v": f(1, 9, 4, 3), "g": -0.3 * f(1, 9, 4).abs(),
           "beta": torch.sigmoid(f(1, 9, 4)), "h0": f(1, 4, 4, 3)}
    dy, dh = f(1, 9, 4, 3), f(1, 4, 4, 3)
    out = refs.delta(*ops.values(), dy, dh)

    def loss(o):
        r = refs.delta(*o.values())
        return float((r["y"] * dy).sum() + (r["h_final"] * dh).sum())

    grads = {"q": "dq", "k": "dk", "v": "dv", "g": "dlog_decay", "beta": "dbeta", "h0": "dh0"}
    for name, grad in grads.items():
        d = f(*ops[name].shape)
        step = 1e-5
        got = (loss(dict(ops, **{name: ops[name] + step * d})) - loss(dict(ops, **{name: ops[name] - step * d}))) / (2 * step)
        want = float((out[grad] * d).sum())
        # the third derivative's step^2 and the loss's rounding over the step
        assert abs(got - want) < 1e-7 * (1 + abs(want)), name


def test_reference_norm_gradients_are_differences():
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((5, 3, 10)), rng.standard_normal((5, 2, 10))
    wq, wk = rng.standard_normal(10), rng.standard_normal(10)
    dq, dk = rng.standard_normal(q.shape), rng.standard_normal(k.shape)
    pos, rates = np.arange(5) * 7, np.array([1.0, 0.3, 0.01])
    for norm in ("rms", "l2"):
        for pairs in ("halves", "neighbours"):
            how = (pos, rates, norm, pairs, 1e-3, 0.7)
            out, _ = refs.norm_rotate(q, k, wq, wk, *how, dq=dq, dk=dk)

            def loss(q, k, wq, wk):
                o, _ = refs.norm_rotate(q, k, wq, wk, *how)
                return (o["q"] * dq).sum() + (o["k"] * dk).sum()

            ops = {"q": q, "k": k, "wq": wq, "wk": wk}
            for name in ops:
                d = rng.standard_normal(ops[name].shape)
                got = (loss(**dict(ops, **{name: ops[name] + 1e-5 * d})) - loss(**dict(ops, **{name: ops[name] - 1e-5 * d}))) / 2e-5
                want = (out["d" + name] * d).sum()
                assert abs(got - want) < 1e-7 * (1 + abs(want)), (norm, pairs, name)

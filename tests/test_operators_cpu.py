"""Linear attention, the token moves and the router's backward without a GPU:
struct layout, refusals before anything is launched, workspace sizes, and the
64-bit references against differences."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import operator_refs as refs
from parameter_space_moe_amd import swimba as sw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x100000  # never read: every call below is refused on the host


@pytest.fixture(scope="module")
def lib():
    return sw.load()


STRUCTS = (("swimba_linear_attention_args", sw.LinearAttentionArgs),
           ("swimba_linear_attention_grad_args", sw.LinearAttentionGradArgs),
           ("swimba_linear_attention_step_args", sw.LinearAttentionStepArgs))


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


def attention_args(**kw):
    a = sw.LinearAttentionArgs()
    a.B, a.L, a.H, a.G, a.N, a.P = 1, 8192, 2, 1, 64, 64
    a.in_dtype, a.y_dtype, a.decay_form = sw.BF16, sw.BF16, sw.DECAY_TOKEN
    for f in ("q", "k", "v", "log_decay", "y"):
        setattr(a, f, FAKE)
    for f, v in kw.items():
        setattr(a, f, v)
    return a


BAD = [("B", -1, sw.EINVAL), ("L", -1, sw.EINVAL), ("H", 0, sw.EINVAL), ("G", 0, sw.EINVAL),
       ("N", 0, sw.EINVAL), ("P", 0, sw.EINVAL), ("H", 3, sw.OK), ("G", 3, sw.EINVAL),
       ("in_dtype", 7, sw.EINVAL), ("y_dtype", 7, sw.EINVAL), ("decay_form", 2, sw.EINVAL),
       ("N", 257, sw.EUNSUPPORTED), ("q", None, sw.EINVAL), ("k", None, sw.EINVAL),
       ("v", None, sw.EINVAL), ("log_decay", None, sw.EINVAL), ("q", FAKE + 1, sw.EINVAL)]


@pytest.mark.parametrize("field,value,status", [b for b in BAD if b[2] != sw.OK])
def test_linear_attention_refuses(lib, field, value, status):
    a = attention_args(**{field: value})
    assert lib.swimba_linear_attention(ctypes.byref(a), None, 0, None) == status
    g = sw.LinearAttentionGradArgs()
    g.fwd = a
    g.grad_dtype = sw.BF16
    for f in ("dy", "dq", "dk", "dv", "dlog_decay"):
        setattr(g, f, FAKE)
    assert lib.swimba_linear_attention_backward(ctypes.byref(g), None, 0, None) == status


def test_linear_attention_refuses_workspace(lib):
    a = attention_args()
    need = lib.swimba_linear_attention_workspace_size(ctypes.byref(a))
    assert need > 0  # two heads do not fill the device: segments
    assert lib.swimba_linear_attention(ctypes.byref(a), None, 0, None) == sw.EWORKSPACE
    assert lib.swimba_linear_attention(ctypes.byref(a), FAKE, need - 1, None) == sw.EWORKSPACE
    assert lib.swimba_linear_attention(ctypes.byref(a), FAKE + 128, need, None) == sw.EWORKSPACE
    assert lib.swimba_linear_attention(None, None, 0, None) == sw.EINVAL
    assert lib.swimba_linear_attention_workspace_size(None) == 0
    a = attention_args(y=None)
    assert lib.swimba_linear_attention(ctypes.byref(a), FAKE, need, None) == sw.EINVAL


def test_linear_attention_backward_refuses(lib):
    def grad(**kw):
        g = sw.LinearAttentionGradArgs()
        g.fwd = attention_args(**kw.pop("fwd", {}))
        g.grad_dtype = sw.BF16
        for f in ("dy", "dq", "dk", "dv", "dlog_decay"):
            setattr(g, f, FAKE)
        for f, v in kw.items():
            setattr(g, f, v)
        return g

    def call(g, ws=None, n=0):
        return lib.swimba_linear_attention_backward(ctypes.byref(g), ws, n, None)

    for f in ("dy", "dq", "dk", "dv", "dlog_decay"):
        assert call(grad(**{f: None})) == sw.EINVAL, f
    assert call(grad(grad_dtype=3)) == sw.EINVAL
    assert call(grad(fwd={"P": 257})) == sw.EUNSUPPORTED
    assert call(grad()) == sw.EWORKSPACE
    assert call(grad(dq=FAKE + 1)) == sw.EINVAL
    assert lib.swimba_linear_attention_backward(None, None, 0, None) == sw.EINVAL


def test_linear_attention_step_refuses(lib):
    def step(**kw):
        a = sw.LinearAttentionStepArgs()
        a.B, a.H, a.G, a.N, a.P = 2, 4, 2, 16, 16
        a.in_dtype, a.y_dtype, a.decay_form = sw.BF16, sw.F32, sw.DECAY_HEAD
        for f in ("q", "k", "v", "log_decay", "state", "y"):
            setattr(a, f, FAKE)
        for f, v in kw.items():
            setattr(a, f, v)
        return lib.swimba_linear_attention_step(ctypes.byref(a), None)

    for f in ("q", "k", "v", "log_decay", "state", "y"):
        assert step(**{f: None}) == sw.EINVAL, f
    assert step(B=-1) == step(G=3) == step(N=0) == step(in_dtype=9) == step(y=FAKE + 1) == sw.EINVAL
    assert step(decay_form=-1) == sw.EINVAL
    assert step(N=300) == sw.EUNSUPPORTED
    assert step(B=0) == sw.OK  # nothing to do, nothing launched
    assert lib.swimba_linear_attention_step(None, None) == sw.EINVAL


def test_tokens_refuse(lib):
    sort, F = lib.swimba_sort_tokens, FAKE
    assert sort(F, -1, 4, 2, F, F, F, None, 0, None) == sw.EINVAL
    assert sort(F, 8, 0, 1, F, F, F, None, 0, None) == sw.EINVAL
    assert sort(F, 8, 4, 5, F, F, F, None, 0, None) == sw.EINVAL
    assert sort(F, 8, 65, 2, F, F, F, None, 0, None) == sw.EUNSUPPORTED
    assert sort(F, (1 << 29) + 1, 4, 2, F, F, F, None, 0, None) == sw.EUNSUPPORTED
    assert sort(None, 8, 4, 2, F, F, F, None, 0, None) == sw.EINVAL
    assert sort(F, 8, 4, 2, F, None, F, None, 0, None) == sw.EINVAL
    assert sort(F, 8, 4, 2, F, F, None, None, 0, None) == sw.EINVAL
    need = lib.swimba_sort_tokens_workspace_size(65536, 4, 2)
    assert need > 0 and lib.swimba_sort_tokens_workspace_size(8, 4, 2) == 0
    assert sort(F, 65536, 4, 2, F, F, F, F, need - 1, None) == sw.EWORKSPACE
    d = lib.swimba_dispatch_tokens
    assert d(F, 9, F, 8, 16, 2, F, None) == sw.EINVAL
    assert d(F, sw.F32, F, 8, 0, 2, F, None) == sw.EINVAL
    assert d(None, sw.F32, F, 8, 16, 2, F, None) == sw.EINVAL
    assert d(F + 2, sw.F32, F, 8, 16, 2, F, None) == sw.EINVAL
    assert d(None, sw.F32, None, 0, 16, 2, None, None) == sw.OK  # no tokens, nothing launched
    c = lib.swimba_combine_tokens
    assert c(F, sw.F32, None, F, 8, 16, 2, F, sw.F32, None) == sw.EINVAL
    assert c(F, sw.F32, F, F, 8, 16, 0, F, sw.F32, None) == sw.EINVAL
    assert c(F, sw.F32, F, F, 8, 16, 2, F, 4, None) == sw.EINVAL
    b = lib.swimba_combine_tokens_backward
    assert b(F, sw.F32, F, None, F, sw.F32, 8, 16, 2, F, sw.F32, F, None) == sw.EINVAL
    assert b(F, sw.F32, F, F, F, sw.F32, 8, 16, 2, F, sw.F32, None, None) == sw.EINVAL


def test_route_backward_refuses(lib):
    r, F = lib.swimba_route_backward, FAKE
    assert r(F, sw.F32, F, F, F, F, 8, 16, 4, 5, F, sw.F32, F, None, 0, None) == sw.EINVAL
    assert r(F, sw.F32, F, F, F, F, 8, 16, 65, 5, F, sw.F32, F, None, 0, None) == sw.EUNSUPPORTED
    assert r(F, sw.F32, F, F, F, F, 8, 16, 4, 2, F, 8, F, None, 0, None) == sw.EINVAL
    assert r(None, sw.F32, F, F, F, F, 8, 16, 4, 2, F, sw.F32, F, None, 0, None) == sw.EINVAL
    assert r(F, sw.F32, F, F, F, F, 8, 16, 4, 2, F, sw.F32, None, None, 0, None) == sw.EINVAL
    need = lib.swimba_route_backward_workspace_size(4096, 64, 4)
    assert need > 0
    assert r(F, sw.F32, F, F, F, F, 4096, 64, 4, 2, F, sw.F32, F, None, 0, None) == sw.EWORKSPACE


def test_binding_refuses_host_tensors():
    t = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError):
        sw.linear_attention(t, t, t, torch.zeros(2))
    with pytest.raises(ValueError):
        sw.sort_tokens(torch.zeros(4, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        sw.combine_tokens(torch.zeros(8, 16), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sw.route_backward(torch.zeros(4, 16), torch.zeros(16, 4), None, None, None)


@pytest.mark.parametrize("form", [1, 3])
def test_attention_reference_gradients_are_differences(form):
    rng = np.random.default_rng(5)
    B, L, H, G, N, P = 2, 7, 4, 2, 3, 5
    a = {"q": rng.standard_normal((B, L, G, N)), "k": rng.standard_normal((B, L, G, N)),
         "v": rng.standard_normal((B, L, H, P)), "h0": rng.standard_normal((B, H, N, P)),
         "log_decay": -rng.random(H if form == 1 else (B, L, H))}
    dy, dh = rng.standard_normal((B, L, H, P)), rng.standard_normal((B, H, N, P))

    def loss(x):
        r = refs.attention(x["q"], x["k"], x["v"], x["log_decay"], x["h0"])
        return (dy * r["y"]).sum() + (dh * r["h_final"]).sum()

    g = refs.attention(a["q"], a["k"], a["v"], a["log_decay"], a["h0"], dy, dh)
    for name in a:
        d = rng.standard_normal(a[name].shape)
        step = 1e-5
        up, down = dict(a), dict(a)
        up[name], down[name] = a[name] + step * d, a[name] - step * d
        want = (loss(up) - loss(down)) / (2 * step)
        got = (g["d" + name] * d).sum()
        assert abs(got - want) < 1e-6 * max(1.0, abs(want)), (name, got, want)


def test_route_and_combine_reference_gradients_are_differences():
    rng = np.random.default_rng(6)
    T, D, E, k = 9, 6, 5, 2
    x, Wr = rng.standard_normal((T, D)), rng.standard_normal((D, E))
    logits = x @ Wr
    idx = np.argsort(-logits, axis=1)[:, :k]
    dgate = rng.standard_normal((T, k))

    def gates(x, Wr):
        l = np.take_along_axis(x @ Wr, idx, 1)
        e = np.exp(l - l.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)

    dx, dW, _, _ = refs.route_backward(x, Wr, idx, gates(x, Wr), dgate)
    for which, g in ((0, dx), (1, dW)):
        d = rng.standard_normal(g.shape)
        s = 1e-6
        up = (x + s * d, Wr) if which == 0 else (x, Wr + s * d)
        down = (x - s * d, Wr) if which == 0 else (x, Wr - s * d)
        want = ((gates(*up) - gates(*down)) * dgate).sum() / (2 * s)
        assert abs((g * d).sum() - want) < 1e-7
    _, pos, _ = refs.sort_tokens(idx, E)
    rows, gate, dy = rng.standard_normal((T * k, D)), rng.random((T, k)), rng.standard_normal((T, D))
    drows, dg = refs.combine_backward(rows, pos, gate, dy, np.zeros_like(rows))
    d, e = rng.standard_normal(rows.shape), rng.standard_normal(gate.shape)  # bilinear: exact
    assert abs((drows * d).sum() - (dy * refs.combine(d, pos, gate)).sum()) < 1e-12
    assert abs((dg * e).sum() - (dy * refs.combine(rows, pos, e)).sum()) < 1e-12


def test_refuses_more_than_a_launch_counts(lib):
    """Threads of a launch are counted in 32 bits."""
    many = {"B": 1 << 24, "L": 1, "H": 1, "G": 1, "N": 1, "P": 1}
    wide = {"B": 1 << 20, "L": 1, "H": 1, "G": 1, "N": 1, "P": 512}
    for kw in (many, wide, dict(many, L=0)):
        a = attention_args(**kw)
        assert lib.swimba_linear_attention(ctypes.byref(a), FAKE, 1 << 40, None) == sw.EUNSUPPORTED
        assert lib.swimba_linear_attention_workspace_size(ctypes.byref(a)) == 0
    for kw in (many, dict(many, B=1 << 22), dict(many, B=1 << 21, N=256),
               dict(many, B=16, L=(1 << 28) - 64), dict(many, B=1 << 10, L=1 << 18, H=2, G=1, N=128)):
        g = sw.LinearAttentionGradArgs()
        g.fwd = attention_args(**kw)
        g.grad_dtype = sw.BF16
        for f in ("dy", "dq", "dk", "dv", "dlog_decay"):
            setattr(g, f, FAKE)
        assert lib.swimba_linear_attention_backward(ctypes.byref(g), FAKE, 1 << 40, None) == sw.EUNSUPPORTED
    st = sw.LinearAttentionStepArgs()
    st.B, st.H, st.G, st.N, st.P = 1 << 14, 1 << 10, 1, 1, 1
    assert lib.swimba_linear_attention_step(ctypes.byref(st), None) == sw.EUNSUPPORTED
    assert lib.swimba_dispatch_tokens(FAKE, sw.F32, FAKE, 1 << 30, 128, 1, FAKE, None) == sw.EUNSUPPORTED
    assert lib.swimba_combine_tokens(FAKE, sw.F32, FAKE, None, 1 << 30, 128, 1, FAKE, sw.F32,
                                     None) == sw.EUNSUPPORTED


PACKS = r'''
#include <cstdio>
#include "pack.hpp"
using namespace swimba;
// Every whole load of every row has to lie inside the tensor, and to hold the
// row's elements from its `back`-th on.
template <int N>
int check() {
  int bad = 0;
  for (int rows = 1; rows <= 24; ++rows)
    for (int width = 1; width <= 2 * N + 3; ++width) {
      if (rows * width < N) continue;  // taken element by element
      for (int r = 0; r < rows; ++r)
        for (int c = 0; c < width; c += N) {
          const int left = width - c, back = back_of<N>(rows - 1 - r, width, left);
          const int first = r * width + c - back, used = left < N ? left : N;
          if (back < 0 || first < 0 || first + N > rows * width || back + used > N) {
            if (bad++ < 5) std::printf("%d: %d x %d, row %d column %d\n", N, rows, width, r, c);
          }
        }
    }
  return bad;
}
int main() { return check<4>() + check<8>() != 0; }
'''


def test_whole_loads_stay_inside_the_tensor(tmp_path):
    f = tmp_path / "packs.hip"
    f.write_text(PACKS)
    exe = tmp_path / "packs"
    subprocess.run(["/opt/rocm/bin/hipcc", "--offload-host-only", "-std=c++17",
                    "-I" + os.path.join(ROOT, "parameter_space_moe_amd", "csrc"), str(f), "-o",
                    str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("B,L", [(2, 0), (0, 5)])
def test_backward_without_tokens_takes_empty_gradients(lib, B, L):
    """An empty tensor has no address: the decays' gradient per token may be null there,
    the one per head may not."""
    g = sw.LinearAttentionGradArgs()
    g.fwd = attention_args(B=B, L=L, q=None, k=None, v=None, log_decay=None, y=None)
    g.grad_dtype = sw.BF16
    assert lib.swimba_linear_attention_backward(ctypes.byref(g), None, 0, None) == sw.OK
    g.fwd.decay_form = sw.DECAY_HEAD
    assert lib.swimba_linear_attention_backward(ctypes.byref(g), None, 0, None) == sw.EINVAL


def test_binding_takes_the_first_argument_by_keyword():
    t = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError):
        sw.linear_attention(q=t, k=t, v=t, log_decay=torch.zeros(2))
    with pytest.raises(ValueError):
        sw.sort_tokens(idx=torch.zeros(4, 2, dtype=torch.int32), E=4)
    with pytest.raises(ValueError):
        sw.sort_tokens(E=4)

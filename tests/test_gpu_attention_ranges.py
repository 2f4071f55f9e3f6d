"""Linear attention over the sizes of its numbers and of its walks: magnitudes up
to the documented limit, walks and segments of many chunks, rows of more than 128."""
import pytest
import torch

import operator_refs as refs
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"


def off(got, want, size, bound):
    """The worst error in terms of what it may be."""
    half = refs.U16 if got.dtype == torch.bfloat16 else refs.U32
    return float(((got.double() - want).abs() / (bound * size + half * want.abs() + 1e-30)).nan_to_num(nan=9e9).max())


def signs(gen, *shape):
    """Magnitudes of 1/2 to 1, either sign."""
    m = 0.5 + 0.5 * torch.rand(shape, generator=gen, device=DEV)
    return torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.5, -m, m)


# a decay per token: sums over 64 tokens of -23.9, -4.6 and -39.7 in base 2, and a decay of one
@pytest.mark.parametrize("decay", [-0.2588, -0.05, -0.43, 0.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("H", [320, 1])  # a whole walk per head; segments
def test_states_up_to_the_limit(H, dtype, decay):
    B, L, N, P = 1, 330, 16, 16
    gen = torch.Generator(device=DEV).manual_seed(H)
    g = torch.full((H,), decay, device=DEV)
    most = 5e25 / min(L, 1 / (1 - 2.718281828 ** decay) if decay < 0 else L)  # |k| |v|
    big = most ** 0.5
    q, k, v, dy = (signs(gen, B, L, H, n) * s for n, s in ((N, 1e-10), (N, big), (P, big), (P, 1e-3)))
    h0 = signs(gen, B, H, N, P) * 1e25
    dh = signs(gen, B, H, N, P) * 1e-12
    for swap in (False, True):  # the adjoint's state at the limit instead
        if swap:
            q, k, v, dy, h0, dh = k, q, dy, v, dh, h0
        ops = [t.to(dtype) for t in (q, k, v)]
        y, h = swimba.linear_attention(*ops, g, h0=h0, y_dtype=torch.float32)
        got = swimba.linear_attention_backward(*ops, g, dy.to(dtype), h0=h0, dh_final=dh)
        want, size = refs.attention_on_device(*ops, g, h0, dy.to(dtype), dh)
        assert max(float(t.max()) for n, t in size.items() if n != "terms") < 1e26
        for name, t in dict(got, y=y, h_final=h).items():
            assert off(t, want[name], size[name], refs.roundings(N, P, L)) <= 1, (swap, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("H,L,N,P", [(320, 150, 16, 40), (2, 700, 40, 33), (2, 200, 128, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_columns_of_non_finite_values_are_apart(H, L, N, P, dtype, bad):
    # one value of one head: its column is lost from that token on, and nothing else
    gen = torch.Generator(device=DEV).manual_seed(L)
    q, k, v = (torch.randn(1, L, H, n, generator=gen, device=DEV).to(dtype) for n in (N, N, P))
    g = -0.1 * torch.rand(1, L, H, generator=gen, device=DEV)
    g[:, 100] = -float("inf")
    h0 = torch.randn(1, H, N, P, generator=gen, device=DEV)
    dy = torch.randn(1, L, H, P, generator=gen, device=DEV).to(dtype)
    s, last, col = 77, L - 2, 5
    y, h = swimba.linear_attention(q, k, v, g, h0=h0)
    grads = swimba.linear_attention_backward(q, k, v, g, dy, h0=h0)
    w = v.clone()
    w[0, s, 1, col] = bad
    w[0, last, 0, P - 1] = bad
    y2, h2 = swimba.linear_attention(q, k, w, g, h0=h0)
    lost = torch.zeros_like(y, dtype=torch.bool)
    lost[0, s:, 1, col] = lost[0, last:, 0, P - 1] = True
    assert not torch.isfinite(y2[lost]).any() and torch.equal(y2[~lost], y[~lost])
    gone = torch.zeros_like(h, dtype=torch.bool)
    gone[0, 1, :, col] = gone[0, 0, :, P - 1] = True
    assert not torch.isfinite(h2[gone]).any() and torch.equal(h2[~gone], h[~gone])
    # the backward's values are k (for dq) and q (for dk, from the last token back)
    for name, n in (("k", "dq"), ("q", "dk")):
        ops = {"q": q, "k": k}
        ops[name] = ops[name].clone()
        ops[name][0, s, 1, col] = bad
        got = swimba.linear_attention_backward(ops["q"], ops["k"], v, g, dy, h0=h0)[n]
        lost = torch.zeros_like(got, dtype=torch.bool)
        lost[0, (slice(s, None) if n == "dq" else slice(0, s + 1)), 1, col] = True
        assert not torch.isfinite(got[lost]).any() and torch.equal(got[~lost], grads[n][~lost]), n


def segments(q, v, g):
    """Segments of the forward walk, from the workspace that holds their states."""
    B, L, H, P = v.shape
    state = B * H * q.shape[-1] * P * 4
    return max(1, swimba.linear_attention_workspace_bytes(q, q, v, g) // state)


def check(shape, dtype, form, gdt, h0=True, reset=0, seed=0):
    B, L, H, G, N, P = shape
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    q, k = (normal(B, L, G, N) * N ** -0.25 for _ in range(2))
    v, dy = normal(B, L, H, P), normal(B, L, H, P)
    if form == "head":  # from 1 - 1/4 to 1 - 1/1024
        g = torch.log1p(-torch.exp2(-torch.linspace(2, 10, H, device=DEV)))
    else:
        g = -0.2 * normal(B, L, H).abs() * torch.rand(H, generator=gen, device=DEV)
        if reset:
            g[torch.rand(B, L, generator=gen, device=DEV) < 1 / reset] = -float("inf")
    q, k, v, dy = (t.to(dtype) for t in (q, k, v, dy))
    st, dh = (normal(B, H, N, P), normal(B, H, N, P)) if h0 else (None, None)
    y, h = swimba.linear_attention(q, k, v, g, h0=st, y_dtype=gdt)
    got = swimba.linear_attention_backward(q, k, v, g, dy, h0=st, dh_final=dh, grad_dtype=gdt)
    want, size = refs.attention_on_device(q, k, v, g, st, dy, dh)
    for name, t in dict(got, y=y, h_final=h).items():
        b = refs.roundings(N, P, L, gdt == torch.float32 or name not in ("y", "dv")) + H // G * refs.U32
        worst = off(t, want[name], size[name], b)
        assert worst <= 1, (name, worst)
    return segments(q, v, g), -(-L // 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("form", ["head", "token", "documents"])
@pytest.mark.parametrize("shape", [(4, 1300, 80, 80, 16, 16), (3, 1000, 120, 30, 24, 40)], ids=str)
def test_whole_walks_of_many_chunks(shape, form, dtype):
    nseg, chunks = check(shape, dtype, form, torch.float32, h0=form != "head", reset=300 * (form == "documents"))
    assert nseg == 1 and chunks >= 16


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("form", ["head", "token", "documents"])
@pytest.mark.parametrize("shape", [(2, 1400, 40, 40, 16, 16), (4, 1500, 32, 8, 128, 128), (4, 1100, 24, 24, 64, 64),
                                   (2, 900, 30, 10, 33, 50), (2, 1100, 20, 20, 40, 256)], ids=str)
def test_segments_of_several_chunks(shape, form, dtype):
    gdt = dtype if form == "head" else torch.float32
    nseg, chunks = check(shape, dtype, form, gdt, h0=form != "head", reset=250 * (form == "documents"), seed=1)
    # fp32 rows of 128 leave one workgroup per CU: whole walks of 24 chunks there
    assert chunks > nseg and (nseg > 1) == (dtype == torch.bfloat16 or shape[4] < 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("shape", [(1, 200, 2, 1, 96, 256), (1, 130, 1, 1, 40, 200), (2, 70, 3, 3, 256, 256),
                                   (1, 1100, 2, 2, 256, 256), (1, 65, 2, 1, 7, 131), (1, 700, 4, 2, 200, 136)], ids=str)
def test_rows_of_more_than_128(shape, dtype):
    for form, gdt in (("head", torch.float32), ("token", dtype)):
        check(shape, dtype, form, gdt, reset=100 * (form == "token"), seed=2)

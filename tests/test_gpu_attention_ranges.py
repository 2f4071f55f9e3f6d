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

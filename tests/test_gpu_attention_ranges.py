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

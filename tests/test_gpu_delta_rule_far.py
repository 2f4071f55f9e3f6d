"""Offsets of more than 32 bits: the end of a sequence of 2^31 values and more against a call of its
own, for the delta rule and for the norms."""
import pytest
import torch

from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"


def off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("L,H,G,N,P", [(600011, 64, 1, 16, 64), (300007, 64, 32, 128, 16)])
def test_delta_rule(L, H, G, N, P):
    gen = torch.Generator(device=DEV).manual_seed(7)

    def f(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    tail = 131
    q, k = (f(1, L, G, N).mul_(N ** -0.5) for _ in range(2))
    v, dy = f(1, L, H, P), f(1, L, H, P)
    assert max(v.numel(), q.numel()) * 2 > 1 << 31
    g = -0.2 * torch.rand(1, L, H, generator=gen, device=DEV)
    beta = torch.rand(1, L, H, generator=gen, device=DEV)
    ops = [q, k, v, g, beta]
    y, h = swimba.delta_rule(*ops, y_dtype=torch.float32)
    # what a sequence of 64 chunks has made of its state no longer depends on what was before
    start = L - 64 * 64 - tail
    _, mid = swimba.delta_rule(*(x[:, start:L - tail].contiguous() for x in ops))
    end = [x[:, L - tail:].contiguous() for x in ops]
    y2, h2 = swimba.delta_rule(*end, h0=mid, y_dtype=torch.float32)
    # three roundings of 2^-22 each at most in the 2-norm
    assert off(y[:, L - tail:], y2) < 1e-6 and off(h, h2) < 1e-6
    del y
    got = swimba.delta_rule_backward(*ops, dy)
    want = swimba.delta_rule_backward(*end, dy[:, L - tail:].contiguous(), h0=mid)
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        assert off(got[n][:, L - tail:], want[n]) < 2e-6, n


@pytest.mark.parametrize("T,Hq,Hk,N,R", [(700001, 40, 8, 64, 64), (400003, 3, 70, 75, 30)])
def test_norms(T, Hq, Hk, N, R):
    gen = torch.Generator(device=DEV).manual_seed(8)
    q, k, dq, dk = (torch.randn(T, h, N, generator=gen, device=DEV, dtype=torch.bfloat16) for h in (Hq, Hk, Hq, Hk))
    assert (q.numel() + k.numel()) > 1 << 31
    w = torch.rand(N, generator=gen, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    rates = torch.rand(R // 2, generator=gen, device=DEV)
    how = dict(wq=w, wk=w, rates=rates)
    a = swimba.norm_rotate(q, k, positions=pos, **how)
    da = swimba.norm_rotate_backward(q, k, dq, dk, positions=pos, **how, grad_dtype=torch.bfloat16)
    n = 77
    for part in (slice(0, n), slice(T - n, T)):
        end = [x[part].contiguous() for x in (q, k, dq, dk)]
        b = swimba.norm_rotate(*end[:2], positions=pos[part].contiguous(), **how)
        db = swimba.norm_rotate_backward(*end, positions=pos[part].contiguous(), **how, grad_dtype=torch.bfloat16)
        assert all(torch.equal(x[part], z) for x, z in zip(a, b))
        assert all(torch.equal(da[x][part], db[x]) for x in ("dq", "dk"))

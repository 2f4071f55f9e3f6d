"""Calls of the operators around the scan that their documentation allows: without
tokens, by keyword, on other streams and in captured graphs."""
import pytest
import torch

from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_backward_without_tokens_and_a_decay_per_token():
    H, N, P = 2, 8, 8
    q, v = torch.zeros(2, 0, 1, N, device=DEV), torch.zeros(2, 0, H, P, device=DEV)
    dh = torch.randn(2, H, N, P, device=DEV)
    g = swimba.linear_attention_backward(q, q, v, torch.zeros(2, 0, H, device=DEV), v, dh_final=dh)
    assert torch.equal(g["dh0"], dh) and g["dlog_decay"].shape == (2, 0, H) and g["dq"].shape == q.shape


def test_arguments_by_keyword():
    q, v = torch.randn(1, 9, 2, 16, device=DEV), torch.randn(1, 9, 4, 8, device=DEV)
    g, st = -torch.rand(4, device=DEV), torch.randn(1, 4, 16, 8, device=DEV)
    y, h = swimba.linear_attention(q, q, v, g)
    y2, h2 = swimba.linear_attention(log_decay=g, v=v, k=q, q=q)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    a = swimba.linear_attention_backward(q, q, v, g, v)
    b = swimba.linear_attention_backward(q=q, k=q, v=v, log_decay=g, dy=v)
    assert all(torch.equal(a[n], b[n]) for n in a)
    one = [t[:, 0].contiguous() for t in (q, v)]
    assert torch.equal(swimba.linear_attention_step(one[0], one[0], one[1], g, st.clone()),
                       swimba.linear_attention_step(q=one[0], k=one[0], v=one[1], log_decay=g, state=st.clone()))
    idx = torch.randint(0, 4, (9, 2), dtype=torch.int32, device=DEV)
    order, pos, offsets = swimba.sort_tokens(idx=idx, E=4)
    assert torch.equal(pos, swimba.sort_tokens(idx, 4)[1])
    x, gate = torch.randn(9, 32, device=DEV), torch.rand(9, 2, device=DEV)
    rows = swimba.dispatch_tokens(x=x, pos=pos)
    assert torch.equal(swimba.combine_tokens(rows=rows, pos=pos, gate=gate), swimba.combine_tokens(rows, pos, gate))
    assert torch.equal(swimba.dispatch_tokens_backward(drows=rows, pos=pos), swimba.combine_tokens(rows, pos))
    c = swimba.combine_tokens_backward(rows=rows, pos=pos, gate=gate, dy=x)
    assert torch.equal(c[1], swimba.combine_tokens_backward(rows, pos, gate, x)[1])
    W = torch.randn(32, 4, device=DEV)
    d = swimba.route_backward(x=x, Wr=W, idx=idx, gate=gate, dgate=c[1])
    assert all(torch.equal(m, n) for m, n in zip(d, swimba.route_backward(x, W, idx, gate, c[1])))

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


def step_inputs(B=3, H=4, G=2, N=64, P=32, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    return [normal(B, G, N), normal(B, G, N), normal(B, H, P), -normal(B, H).abs()], normal(B, H, N, P)


@pytest.mark.parametrize("prepared", [False, True])
def test_step_on_another_stream(prepared):
    # the state is there only behind a wait on that stream
    ops, st = step_inputs()
    y = swimba.linear_attention_step(*ops, st, state_out=(out := torch.empty_like(st)))
    late, got = torch.zeros_like(st), torch.empty_like(st)
    call = swimba.PreparedLinearAttentionStep(*ops, late, state_out=got)
    assert torch.isfinite(call()).all()  # also after a call on the stream that it was made on
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(st)
        y2 = call() if prepared else swimba.linear_attention_step(*ops, late, state_out=got)
    side.synchronize()
    assert torch.equal(y2, y) and torch.equal(got, out)
    # a stream of the caller's
    late.zero_()
    torch.cuda.synchronize()
    if prepared:
        call = swimba.PreparedLinearAttentionStep(*ops, late, state_out=got, stream=side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(st)
    y2 = call() if prepared else swimba.linear_attention_step(*ops, late, state_out=got, stream=side)
    side.synchronize()
    assert torch.equal(y2, y) and torch.equal(got, out)


@pytest.mark.parametrize("prepared", [False, True])
def test_step_captured(prepared):
    # a decode loop: the state in place, a token per replay
    ops, first = step_inputs(seed=1)
    tokens = [step_inputs(seed=2 + i)[0] for i in range(4)]
    want, st = [], first.clone()
    for t in tokens:
        want.append(swimba.linear_attention_step(*t, st))
    held, y = first.clone(), torch.empty_like(want[0])
    call = swimba.PreparedLinearAttentionStep(*ops, held, y=y)
    if not prepared:
        def call():
            return swimba.linear_attention_step(*ops, held, y=y)
    call()  # warm-up
    held.copy_(first)
    y.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    assert torch.equal(held, first) and not y.any()  # recorded, not run
    for t, w in zip(tokens, want):
        for dst, src in zip(ops, t):
            dst.copy_(src)
        graph.replay()
        other = swimba.linear_attention_step(*t, first.clone())  # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(y, w) and torch.isfinite(other).all()
    assert torch.equal(held, st)

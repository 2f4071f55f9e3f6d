"""Three bf16 terms in every product of the gated delta rule: errors in the 2-norm, which two terms
or a pair of terms left out would exceed (delta_terms.py has the limits and where they come
from).  Two of the shapes are walked in segments."""
import pytest
import torch

import delta_refs as refs
import delta_terms as terms
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OPS = ("q", "k", "v", "g", "beta")
CASES = [(d, s) for s in terms.SHAPES for d in DT] + [("bf16", terms.WIDE)]


def prepared(dtype, shape):
    t = terms.inputs(*shape, DT[dtype], sum(shape))
    return {n: x.to(DEV) for n, x in t.items()}, refs.delta(*(t[n].double() for n in OPS + ("h0", "dy", "dh")))


@pytest.mark.parametrize("dtype,shape", CASES, ids=str)
def test_results_in_bf16(dtype, shape):
    d, want = prepared(dtype, shape)
    y, h = swimba.delta_rule(*(d[n] for n in OPS), h0=d["h0"], y_dtype=torch.bfloat16)
    assert terms.moved(y, want["y"]) < terms.MOVED
    assert terms.off(h, want["h_final"]) < terms.LIMIT["h_final"]


@pytest.mark.parametrize("dtype,shape", CASES, ids=str)
def test_results_and_gradients_in_fp32(dtype, shape):
    d, want = prepared(dtype, shape)
    y, h = swimba.delta_rule(*(d[n] for n in OPS), h0=d["h0"], y_dtype=torch.float32)
    got = dict(swimba.delta_rule_backward(*(d[n] for n in OPS), d["dy"], h0=d["h0"], dh_final=d["dh"]), y=y, h_final=h)
    for n, limit in terms.LIMIT.items():
        assert terms.off(got[n], want[n]) < limit, n
    if shape in terms.SUMMED:
        d["g"] = d["g"][0, 0].contiguous()  # the same decays, one per head
        got = swimba.delta_rule_backward(*(d[n] for n in OPS), d["dy"], h0=d["h0"], dh_final=d["dh"])["dlog_decay"]
        size = want["dlog_decay"].square().sum((0, 1)).sqrt()
        off = (got.double().cpu() - want["dlog_decay"].sum((0, 1))).abs() / size
        assert off.max() < terms.LIMIT_SUM


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bf16_results_that_cancel(dtype):
    # y = x - x (1 + r 2^-13), exactly representable operands apart from the state, which two terms
    # hold within 2^-18.  y's own rounding to bf16 is 2^-22 of x; three terms are off by 2^-27 of each of the
    # two states and six fp32 additions by less than 2^-22.
    P = 4096
    gen = torch.Generator().manual_seed(3)
    x = 1 + torch.rand(P, generator=gen)
    r = 2 * torch.rand(P, generator=gen) - 1
    h0 = torch.stack([x, x * (1 + r * 2.0 ** -13)]).reshape(1, 1, 2, P)
    q = torch.tensor([1.0, -1.0]).expand(1, 3, 1, 2).to(DT[dtype]).contiguous().to(DEV)
    zero = torch.zeros(1, 3, 1, P, dtype=DT[dtype], device=DEV)
    y, h = swimba.delta_rule(q, q, zero, torch.zeros(1, 3, 1, device=DEV), torch.zeros(1, 3, 1, device=DEV), h0=h0.to(DEV),
                             y_dtype=torch.bfloat16)
    assert torch.equal(h.cpu(), h0)
    want = h0[0, 0, 0].double() - h0[0, 0, 1].double()
    most = refs.HALF[torch.bfloat16] * want.abs() * (1 + 2.0 ** -8) + 2 * (2.0 ** -27 + 2.0 ** -23) * x.double()
    assert ((y[0].double().cpu().squeeze(1) - want).abs() <= most).all()

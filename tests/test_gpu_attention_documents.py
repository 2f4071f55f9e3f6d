"""The decays' gradient of linear attention next to other packed documents: what
one document's numbers are must not show in another's."""
import pytest
import torch

import operator_refs as refs
from parameter_space_moe_amd import swimba

pytestmark = pytest.mark.gpu

DEV = "cuda"


def inputs(B, L, H, N, P, starts, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    t = {"q": normal(B, L, H, N) * N ** -0.25, "k": normal(B, L, H, N) * N ** -0.25, "v": normal(B, L, H, P),
         "log_decay": -0.1 * normal(B, L, H).abs(), "h0": normal(B, H, N, P), "dy": normal(B, L, H, P),
         "dh": normal(B, H, N, P)}
    t["log_decay"][:, starts] = -float("inf")
    return t


def backward(t, **kw):
    return swimba.linear_attention_backward(t["q"], t["k"], t["v"], t["log_decay"], t["dy"], h0=t["h0"],
                                            dh_final=t["dh"], **kw)


# heads: a whole walk per head, and segments
@pytest.mark.parametrize("B,H,L", [(4, 80, 300), (1, 1, 300), (2, 40, 700)])
@pytest.mark.parametrize("starts", [[37], [64], [63, 130], [20, 30, 40, 191, 192]], ids=str)
def test_decay_gradients_stay_inside_documents(B, H, L, starts):
    N, P = 16, 24
    t = inputs(B, L, H, N, P, starts, seed=L + len(starts))
    t["dy"][:, starts[-1]:] *= 1e6
    t["dh"] *= 1e6
    got = backward(t)["dlog_decay"].double()
    want, size = refs.attention_on_device(**t)
    want, size = want["dlog_decay"], size["dlog_decay"]
    # the walks' roundings, and the conversion of the result
    allow = refs.roundings(N, P, L) * size + refs.U32 * want.abs() + 1e-30
    off = (got - want).abs() / allow
    assert bool((off <= 1).all()), "worst %.3g times the bound, at token %d" % (
        float(off.max()), int(off.amax((0, 2)).argmax()))

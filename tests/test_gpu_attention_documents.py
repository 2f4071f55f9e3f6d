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


# as above, and with a first state whose gradient is not asked for
@pytest.mark.parametrize("B,H,L,h0", [(4, 80, 300, "given"), (2, 130, 300, "kept"), (1, 1, 200, None),
                                      (2, 40, 700, "kept"), (1, 2, 900, "given")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decay_gradients_before_non_finite_keys_and_values(B, H, L, h0, dtype, bad):
    # a padded batch: rubbish in k and v behind the last token, zeros in dy.  No
    # gradient of the last token's decay and of earlier ones depends on that rubbish
    N, P = 16, 24
    t = inputs(B, L, H, N, P, [], seed=L)
    for n in ("q", "k", "v", "dy"):
        t[n] = t[n].to(dtype)
    s = L - 70
    t["dy"][:, s:] = 0
    t["k"][:, s], t["v"][:, s] = 0, 0
    if h0 is None:
        t["h0"] = t["dh"] = None
    want, size = refs.attention_on_device(**t)
    allow = refs.roundings(N, P, L) * size["dlog_decay"][:, :1]  # a sum from either end
    allow = allow + refs.U32 * want["dlog_decay"].abs() + 1e-30
    for name in ("k", "v", "both"):
        r = dict(t)
        for n in ("k", "v"):
            if name in (n, "both"):
                r[n] = t[n].clone()
                r[n][:, s, :, 3] = bad
                r[n][0, s + 9] = float("nan")
        got = backward(r, want_dh0=h0 == "given")["dlog_decay"].double()
        off = ((got - want["dlog_decay"]).abs() / allow)[:, :s + 1]
        assert bool((off <= 1).all()), (name, float(off.max()))

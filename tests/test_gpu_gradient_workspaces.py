"""Callers' own workspaces for the gradients of the delta rule and of the norms: sized by a query,
read nowhere before it is written, refused when too small."""
import pytest
import torch

from parameter_space_moe_amd import swimba
from test_gpu_delta_rule import OPS, backward, make, to_dev

pytestmark = pytest.mark.gpu

DEV = "cuda"


def spoiled(need):
    return torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read unwritten


@pytest.mark.parametrize("shape", [(2, 200, 4, 2, 32, 48), (1, 1500, 2, 1, 128, 96), (3, 1, 2, 2, 5, 1)], ids=str)
@pytest.mark.parametrize("dtype,form", [("bf16", "token"), ("f32", "head")])
def test_delta_rule(shape, dtype, form):
    d = to_dev(make(*shape, dtype=dtype, form=form, seed=17))
    want = backward(d)
    need = swimba.delta_rule_backward_workspace_bytes(*(d[n] for n in OPS))
    got = backward(d, workspace=spoiled(need))
    assert need > 0 and all(torch.equal(want[n], got[n]) for n in want)
    with pytest.raises(swimba.SwimbaError) as e:
        backward(d, workspace=spoiled(need)[:need - 256])
    assert e.value.status == swimba.EWORKSPACE


@pytest.mark.parametrize("T", [1, 700, 5000])
def test_norms(T):
    gen = torch.Generator().manual_seed(18)
    q, k, dq, dk = (torch.randn(T, h, 64, generator=gen).bfloat16().to(DEV) for h in (6, 2, 6, 2))
    w, rates = torch.ones(64, device=DEV), torch.ones(16, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    assert swimba.norm_rotate_backward_workspace_bytes(q, k) == 0
    for how in (dict(wq=w), dict(wk=w), dict(wq=w, wk=w), dict(wq=w, wk=w, positions=pos, rates=rates)):
        want = swimba.norm_rotate_backward(q, k, dq, dk, **how)
        need = swimba.norm_rotate_backward_workspace_bytes(q, k, **how)
        got = swimba.norm_rotate_backward(q, k, dq, dk, **how, workspace=spoiled(need))
        for n, x in want.items():
            assert x is None and got[n] is None or torch.equal(x, got[n]), n
        with pytest.raises(swimba.SwimbaError) as e:
            swimba.norm_rotate_backward(q, k, dq, dk, **how, workspace=spoiled(need)[:need - 256])
        assert e.value.status == swimba.EWORKSPACE

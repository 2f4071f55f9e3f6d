"""The limits of test_gpu_delta_rule_terms.py lie between what two bf16 terms per operand leave and
what three terms and fp32 sums do."""
import pytest
import torch

import delta_refs as refs
import delta_terms as terms

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype,shape", [(d, s) for s in terms.SHAPES for d in DT] + [("bf16", terms.WIDE)], ids=str)
def test_limits_tell_three_terms_from_two(dtype, shape):
    t = terms.inputs(*shape, DT[dtype], sum(shape))
    a = [t[n].double() for n in ("q", "k", "v", "g", "beta", "h0", "dy", "dh")]
    want, f32 = refs.delta(*a), dtype == "f32"
    whole = terms.emulate(None, f32, *a)
    two, three = (terms.emulate(n, f32, *a) for n in (2, 3))
    sums = terms.emulate(None, f32, *a, dtype=torch.float32)
    for n, limit in terms.LIMIT.items():
        assert terms.off(whole[n], want[n]) < 1e-12, n
        assert terms.off(two[n], want[n]) > 1.5 * limit, n
        assert terms.off(three[n], want[n]) + terms.off(sums[n], want[n]) < limit / 1.5, n
    if shape in terms.SUMMED:
        assert terms.off_summed(two["dlog_decay"], want["dlog_decay"]) > 1.5 * terms.LIMIT_SUM
        assert (terms.off_summed(three["dlog_decay"], want["dlog_decay"])
                + terms.off_summed(sums["dlog_decay"], want["dlog_decay"])) < terms.LIMIT_SUM / 1.5
    # what only y is made from in two terms moves it as far
    y = terms.emulate(3, f32, *a, y_terms=2)["y"]
    assert terms.moved(y.bfloat16(), want["y"]) > 1.5 * terms.MOVED
    assert terms.moved(three["y"].bfloat16(), want["y"]) + terms.moved(sums["y"].bfloat16(), want["y"]) < terms.MOVED / 1.5


def test_cut():
    x = torch.tensor([1.0, 1 + 2.0 ** -9, 1 + 2.0 ** -17 + 2.0 ** -23, 3.14159274], dtype=torch.float64)
    assert terms.cut(x, 1).tolist()[:2] == [1.0, 1.0]
    for n in (1, 2, 3):
        assert ((terms.cut(x, n) - x).abs() <= 2.0 ** (-9 * n) * x).all()

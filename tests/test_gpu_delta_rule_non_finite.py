"""What is beyond fp32 and where it goes in the delta rule."""
import pytest
import torch

import delta_refs as refs
from test_gpu_delta_rule import OPS, close, forward, make, to_dev, wide

pytestmark = pytest.mark.gpu


def test_nothing_grows_out_of_nothing():
    # a state of zeros through segments whose transitions are beyond fp32
    t = make(1, 2000, 1, 1, 32, 16, dtype="f32", h0=False, seed=94)
    t["g"][:, :1600] = 1.0
    t["v"][:, :1600] = 0
    y, h = forward(to_dev(t), y_dtype=torch.float32)
    assert not y[:, :1600].any()
    a = [x[:, 1600:] for x in wide(t, *OPS)]
    want, allow = refs.delta(*a), refs.bounds(True, *a)
    close(y[:, 1600:], want["y"], allow["y"], "y")
    close(h, want["h_final"], allow["h_final"], "h_final")

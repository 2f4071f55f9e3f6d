"""The delta rule over segments whose states have several tiles of columns, in both directions,
and in fp32 with more than 64 keys, against the 64-bit recurrence."""
import pytest
import torch

from parameter_space_moe_amd import swimba
from test_gpu_delta_rule import OPS, check_backward, check_forward, make, to_dev

pytestmark = pytest.mark.gpu

CASES = [  # the last segment is shorter than the others, and a document ends inside a chunk
    ("bf16", (1, 1500, 2, 1, 128, 96), 411), ("bf16", (1, 1100, 2, 2, 128, 130), 300), ("f32", (1, 1300, 2, 1, 100, 70), 500),
    ("bf16", (1, 1300, 4, 1, 64, 200), 0), ("f32", (2, 1000, 2, 2, 128, 128), 333), ("bf16", (1, 2003, 1, 1, 256, 72), 700)]


def segments(t):
    """Whether the forward and the backward walk in segments: their states are in the workspace."""
    d = to_dev(t)
    B, L, H, P = t["v"].shape
    ops = [d[n] for n in OPS]
    units = B * H * ((L + 63) // 64)
    one = units * (6 * 512 * 4 + 6 * 64 * 4) + 1024  # inverses and gates, each rounded up to 256
    rows = 32 << max(0, (t["q"].shape[3] - 1).bit_length() - 5)
    cols = (P + 63) // 64 * 64
    share = H // t["q"].shape[2]
    parts = 2 * share * t["q"].numel() * 4 if share > 1 else 0  # rows of dq and dk, at most
    back = units * (2 * 6 * 512 * 4 + 6 * 64 * 4 + 8 * (rows + 64) * cols) + parts + 8 * units + 4096
    return (swimba.delta_rule_workspace_bytes(*ops) > one, swimba.delta_rule_backward_workspace_bytes(*ops) > back)


@pytest.mark.parametrize("dtype,shape,reset", CASES, ids=str)
def test_documents(dtype, shape, reset):
    t = make(*shape, dtype=dtype, seed=sum(shape), reset=reset)
    assert segments(t) == (True, True)
    check_forward(t, dtype, "f32")
    check_forward(t, dtype, dtype)
    check_backward(t, dtype, "f32")


@pytest.mark.parametrize("dtype,shape,reset", CASES[:3], ids=str)
def test_a_decay_per_head(dtype, shape, reset):
    t = make(*shape, dtype=dtype, form="head", h0=False, seed=1 + sum(shape))
    check_forward(t, dtype, dtype)
    check_backward(t, dtype, dtype)


def test_short_sequences_are_one_walk():
    assert segments(make(1, 100, 2, 1, 64, 64)) == (False, False)

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

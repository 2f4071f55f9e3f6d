"""The number of segments that the delta rule's walks are cut into, read off the workspace that it
asks for, against what measures well on 256 CUs."""
import ctypes

import pytest

from parameter_space_moe_amd import swimba as sw


def padded(N):
    return 32 if N <= 32 else 64 if N <= 64 else 128 if N <= 128 else 256


def segments(B, L, H, G, N, P, dtype, back):
    """From the difference to the same call without segments' states."""
    lib = sw.load()
    g = sw.DeltaRuleGradArgs()
    a = g.fwd
    a.B, a.L, a.H, a.G, a.N, a.P = B, L, H, G, N, P
    a.in_dtype = a.y_dtype = g.grad_dtype = dtype
    a.decay_form = sw.DECAY_TOKEN
    up = lambda n: (n + 255) // 256 * 256
    units, rows, cols = B * H * ((L + 63) // 64), padded(N), (P + 63) // 64 * 64
    tri, gates = up(units * 6 * 512 * 4), up(units * 6 * 64 * 4)
    if back:
        assert H == G  # no rows of dq and dk for parts of shared heads
        base = 2 * tri + gates + 2 * up(units * rows * cols * 4) + 2 * up(units * 64 * cols * 4)
        need = lib.swimba_delta_rule_backward_workspace_size(ctypes.byref(g))
    else:
        base = tri + gates
        need = lib.swimba_delta_rule_workspace_size(ctypes.byref(a))
    each = B * H * rows * (cols + rows) * 4
    assert (need - base) % each == 0
    return max(1, (need - base) // each)


@pytest.mark.parametrize("shape,dtype,back,low,high", [
    # within 6 % of the best of a sweep
    ((1, 65536, 40, 1, 128, 64), sw.BF16, False, 11, 32), ((8, 4096, 32, 32, 128, 128), sw.BF16, False, 1, 1),
    ((1, 32768, 8, 8, 64, 64), sw.BF16, False, 32, 48), ((1, 32768, 8, 8, 64, 64), sw.BF16, True, 32, 64),
    ((1, 65536, 1, 1, 128, 128), sw.BF16, True, 48, 64), ((16, 1024, 8, 8, 128, 128), sw.BF16, True, 1, 1),
    # the join of 256 keys is its longest part, above all walking back
    ((1, 8192, 8, 8, 256, 128), sw.BF16, True, 4, 9), ((1, 8192, 8, 2, 256, 128), sw.BF16, False, 6, 11),
    ((1, 8192, 16, 4, 64, 128), sw.F32, False, 8, 16), ((2, 4096, 16, 4, 128, 128), sw.F32, False, 3, 4)])
def test_segments(shape, dtype, back, low, high):
    assert low <= segments(*shape, dtype, back) <= high

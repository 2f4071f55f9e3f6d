"""The norms where a workgroup takes several tokens, several groups of them one after the other,
and where the heads of a token are cut into several workgroups, against 64 bits."""
import pytest

from test_gpu_norm_rotate import DT, call, close, make, reference, steps

pytestmark = pytest.mark.gpu

CASES = [  # T, Hq, Hk, N, R
    (2503, 6, 2, 64, 64),      # four tokens in a workgroup, three in the last
    (2501, 6, 2, 50, 20),      # the same, element by element
    (4200, 1, 1, 512, 512), (132003, 1, 1, 16, 16),  # the table of cosines is full
    (2203, 40, 8, 128, 128),   # more groups of tokens than workgroups run at once (backward)
    (130, 40, 40, 128, 0),     # heads cut in two or more
    (101, 40, 39, 128, 64),    # the last cut is shorter
    (100, 13, 6, 512, 256), (37, 30, 3, 80, 48)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_both_ways(shape, dtype):
    T, Hq, Hk, N, R = shape
    for i, (norm, pairs) in enumerate((("rms", "halves"), ("l2", "neighbours"))):
        t = make(*shape, dtype, True, seed=i + N + T)
        how = dict(norm=norm, pairs=pairs, q_scale=0.25)
        want, size = reference(t, norm, pairs, q_scale=0.25)
        q, k = call(t, how)
        close(q, want["q"], size["q"], steps(N), "q")
        close(k, want["k"], size["k"], steps(N), "k")
        g = call(t, how, back=True, grad_dtype=DT[dtype])
        # the row's second sum, and the first one's root again
        for n in ("dq", "dk"):
            close(g[n], want[n], size[n], 2 * steps(N) + N / 8, n)
        # in fp32 a thread's rows (three of a group of tokens, two groups at most), six lanes and four waves;
        # then 64 bits
        for n in ("dwq", "dwk"):
            close(g[n], want[n], size[n], steps(N) + 16, n)

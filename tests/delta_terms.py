"""The gated delta rule's chunked products with their operands in a given number of bf16 terms,
emulated in 64 bits: what a number of terms leaves in every output, apart from the
rounding of fp32 sums.  Nothing here is shared with the library."""
from __future__ import annotations

import torch

CHUNK = 64

# What tells three terms from two; test_delta_rule_terms_cpu.py computes both on the inputs of
# the tests.  Relative 2-norms of what two terms leave are 2.8e-6 and more (4.2e-6 and more in the
# decays' gradients), those of three terms and of fp32 sums together 4e-7 and less (9e-7).
LIMIT = {"y": 1e-6, "h_final": 1e-6, "dq": 1e-6, "dk": 1e-6, "dv": 1e-6, "dbeta": 1e-6, "dh0": 1e-6, "dlog_decay": 2e-6}
# The decays' gradients summed over the tokens, relative to their 2-norm: 2.7e-5 and more, 6.5e-6 and less
# (of the SUMMED shapes: in others the terms' errors happen to cancel as well).
LIMIT_SUM = 1e-5
# A y in bf16 is another number than the nearest to the exact one where this is closer to the middle
# of two numbers than y is off.  The share of such values: 3.2e-3 and more, 5e-4 and less.
MOVED = 1.2e-3

# B, L, H, G, N, P
SHAPES = [(1, 300, 2, 1, 64, 48), (1, 1300, 2, 1, 128, 96), (2, 700, 4, 2, 64, 64), (1, 1500, 4, 2, 32, 70)]
WIDE = (1, 200, 2, 1, 200, 40)  # bf16 only
SUMMED = SHAPES[2:]


def cut(x, terms):
    """x as the sum of `terms` bf16 terms, each the nearest to what the ones before leave."""
    out, rest = torch.zeros_like(x), x
    for _ in range(terms):
        t = rest.float().bfloat16().to(x.dtype)
        out, rest = out + t, rest - t
    return out


def emulate(terms, f32, q, k, v, g, beta, h0, dy, dh, dtype=torch.float64, y_terms=None):
    """All outputs of the rule and its backward (a dict), from fp64 inputs.  Operands that are
    computed, and fp32 inputs, enter products in `terms` terms (None: as they are), those
    that only y is made from in y_terms; everything else is in dtype."""
    def c(x, n=None):
        return x if terms is None else cut(x, n or terms)

    def i(x):
        return c(x) if f32 else x

    B, L, H, P = v.shape
    G, N = q.shape[2:]
    g = g.expand(B, L, H)
    Q, K = (t.repeat_interleave(H // G, 2).transpose(1, 2) for t in (q, k))  # [B, H, L, N]
    V, dY = v.transpose(1, 2), dy.transpose(1, 2)
    gates, b = g.transpose(1, 2), beta.transpose(1, 2).unsqueeze(-1).to(dtype)
    Q, K, V, dY = (t.to(dtype) for t in (Q, K, V, dY))
    h = h0.to(dtype)
    y, kept = [], []
    spans = [slice(s, min(L, s + CHUNK)) for s in range(0, L, CHUNK)]
    for s in spans:
        Gs = gates[:, :, s].clamp(min=-2000.0).cumsum(-1)
        n = Gs.shape[-1]
        low = torch.ones(n, n, dtype=torch.bool).tril()
        D = (Gs.unsqueeze(-1) - Gs.unsqueeze(-2)).masked_fill(~low, -2000.0).exp().to(dtype)
        e, w = Gs.exp().unsqueeze(-1).to(dtype), (Gs[..., -1:] - Gs).exp().unsqueeze(-1).to(dtype)
        q1, k1, b1 = i(Q[:, :, s]), i(K[:, :, s]), b[:, :, s]
        A = (k1 @ k1.mT * D).tril(-1) * b1.mT
        T = torch.linalg.solve_triangular(torch.eye(n, dtype=dtype) + A, torch.eye(n, dtype=dtype).expand_as(A), upper=False, unitriangular=True)
        S = q1 @ k1.mT * D
        O = c(T) @ c(V[:, :, s] - e * (k1 @ c(h)))
        y.append(e * (q1 @ c(h, y_terms)) + c(S, y_terms) @ c(b1 * O, y_terms))
        kept.append((D, e, w, T, S, O, h, A))
        h = e[:, :, -1:] * h + k1.mT @ c(w * b1 * O)
    out = {"y": torch.cat(y, 2), "h_final": h}
    a = dh.to(dtype)
    dq, dk, dv, db, dg = ([None] * len(spans) for _ in range(5))
    for m in range(len(spans) - 1, -1, -1):
        s = spans[m]
        D, e, w, T, S, O, h, A = kept[m]
        q1, k1, b1, d1 = i(Q[:, :, s]), i(K[:, :, s]), b[:, :, s], i(dY[:, :, s])
        dU = c(S).mT @ d1 + w * (k1 @ c(a))
        dV = c(T).mT @ c(b1 * dU)
        F, E = d1 @ c(O).mT * D, (c(dV) @ c(O).mT * D).tril(-1)
        FD, ED = F * b1.mT, E * b1.mT
        reads, erased, written = d1 @ c(h).mT, c(dV) @ c(h).mT, c(O) @ c(a).mT
        dq[m] = e * reads + c(FD) @ k1
        dk[m] = b1 * w * written - e * erased + c(FD).mT @ q1 - c(ED + ED.mT) @ k1
        dv[m] = dV
        pairs = (q1 @ k1.mT) * F - (k1 @ k1.mT).tril(-1) * E
        wrote = w[..., 0] * (k1 * written).sum(-1)
        db[m] = pairs.sum(-2) + wrote
        pairs = pairs.tril(-1).double() * b1.mT.double()
        rect = pairs.sum(-2) - pairs.sum(-1)
        seen = (e[..., 0] * (q1 * reads - k1 * erased).sum(-1)).double()
        wb = (b1[..., 0] * wrote).double()
        thru = e[:, :, -1, 0].double() * (h * a).sum((-1, -2)).double()
        dg[m] = rect.cumsum(-1) - rect + seen.flip(-1).cumsum(-1).flip(-1) + wb.cumsum(-1) - wb + thru.unsqueeze(-1)
        a = e[:, :, -1:] * a + q1.mT @ c(e * d1) - k1.mT @ c(e * dV)
    out["dq"], out["dk"] = (torch.cat(x, 2).transpose(1, 2).reshape(B, L, G, H // G, N).sum(3) for x in (dq, dk))
    out["dv"], out["dh0"] = torch.cat(dv, 2).transpose(1, 2), a
    out["y"] = out["y"].transpose(1, 2)
    out["dbeta"] = torch.cat(db, 2).transpose(1, 2)
    out["dlog_decay"] = torch.cat(dg, 2).transpose(1, 2)
    return out


def off(got, want):
    """The relative 2-norm of got - want."""
    return float((got.double().cpu() - want).norm() / want.norm())


def off_summed(got, want):
    """The largest error of a head's sum over batch and tokens, relative to its values' 2-norm."""
    return float(((got.double().cpu() - want).sum((0, 1)).abs() / want.square().sum((0, 1)).sqrt()).max())


def moved(got, want):
    """The share of bf16 values that are not the nearest to the exact ones."""
    return float((got.cpu() != want.bfloat16()).double().mean())


def inputs(B, L, H, G, N, P, dtype, seed):
    """Unit keys, a decay per token (the same for all tokens of a head), states in and out: fp32
    tensors, q, k, v and dy in dtype."""
    gen = torch.Generator().manual_seed(seed)

    def f(*shape):
        return torch.randn(*shape, generator=gen)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    t = {"q": unit(f(B, L, G, N)), "k": unit(f(B, L, G, N)), "v": f(B, L, H, P), "g": torch.log1p(-torch.exp2(-torch.linspace(3, 8, H))).repeat(B, L, 1),
         "beta": torch.sigmoid(f(B, L, H)), "h0": f(B, H, N, P), "dy": f(B, L, H, P), "dh": f(B, H, N, P)}
    return {n: x.to(dtype) if n in ("q", "k", "v", "dy") else x for n, x in t.items()}

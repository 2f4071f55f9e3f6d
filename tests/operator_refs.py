"""64-bit references of linear attention, the token moves and the router's
backward, straight from their definitions, with the size that rounding errors
are measured against: the same sums over absolute values.  Nothing here is
shared with the library."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24   # half a step of fp32
U16 = 2.0 ** -8    # half a step of bf16


def attention(q, k, v, log_decay, h0=None, dy=None, dh=None):
    """fp64 arrays: q, k [B,L,G,N], v [B,L,H,P], log_decay [H] or [B,L,H].  Returns
    a dict of y, h_final and, with dy, the gradients."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    share = H // G
    form = np.asarray(log_decay).ndim
    e = np.exp(np.broadcast_to(np.asarray(log_decay, np.float64), (B, L, H)))
    qh, kh = (np.repeat(t, share, axis=2) for t in (q, k))
    h = np.zeros((B, H, N, P)) if h0 is None else np.array(h0, np.float64)
    y = np.zeros((B, L, H, P))
    states = [h]
    for t in range(L):
        h = e[:, t, :, None, None] * h + kh[:, t, :, :, None] * v[:, t, :, None, :]
        y[:, t] = np.einsum("bhn,bhnp->bhp", qh[:, t], h)
        states.append(h)
    out = {"y": y, "h_final": h}
    if dy is None:
        return out
    dy = np.asarray(dy, np.float64)
    a = np.zeros_like(h) if dh is None else np.array(dh, np.float64)
    dq, dk, dv = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v)
    dg = np.zeros((B, L, H))
    for t in range(L - 1, -1, -1):
        dq[:, t] = np.einsum("bhnp,bhp->bhn", states[t + 1], dy[:, t])
        a = a + qh[:, t, :, :, None] * dy[:, t, :, None, :]
        dk[:, t] = np.einsum("bhnp,bhp->bhn", a, v[:, t])
        dv[:, t] = np.einsum("bhnp,bhn->bhp", a, kh[:, t])
        a = e[:, t, :, None, None] * a
        dg[:, t] = (a * states[t]).sum((-1, -2))
    out["dq"] = dq.reshape(B, L, G, share, N).sum(3)
    out["dk"] = dk.reshape(B, L, G, share, N).sum(3)
    out["dv"] = dv
    out["dlog_decay"] = dg.sum((0, 1)) if form == 1 else dg
    out["dh0"] = a
    return out


def attention_sizes(q, k, v, log_decay, h0=None, dy=None, dh=None):
    """The sums of attention() over absolute values, and for the gradient of the
    log decays the sum over every later token of |q| |dq| + |k| |dk| (in one
    sequence and head the kernels add such terms up before they cancel)."""
    ab = [None if t is None else np.abs(np.asarray(t, np.float64)) for t in (q, k, v, h0, dy, dh)]
    out = attention(ab[0], ab[1], ab[2], log_decay, ab[3], ab[4], ab[5])
    if dy is None:
        return out
    B, L, H, P = np.asarray(v).shape
    share = H // np.asarray(q).shape[2]
    # per head: the group's sum is at least each head's own part
    terms = np.repeat((ab[0] * out["dq"] + ab[1] * out["dk"]).sum(-1), share, axis=2)
    later = terms[:, ::-1].cumsum(1)[:, ::-1]
    if dh is not None:
        later = later + (ab[5] * out["h_final"]).sum((-1, -2))[:, None, :]
    out["dlog_decay"] = later.sum((0, 1)) if np.asarray(log_decay).ndim == 1 else later
    return out


def attention_on_device(q, k, v, log_decay, h0=None, dy=None, dh=None):
    """attention() for long sequences and many heads: the same recurrence on torch
    tensors, in 64 bits, where they are.  Returns (values, sizes); the size of the
    decays' gradient sums over the later tokens of the same document only (up to
    the next decay below 2^-126, which no fp32 number passes)."""
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    share = H // G
    g = log_decay.double().expand(B, L, H)
    e = g.exp()

    def walk(q, k, v, h0, dy, dh):
        q, k = (t.double().repeat_interleave(share, dim=2) for t in (q, k))
        v = v.double()
        h = torch.zeros(B, H, N, P, dtype=torch.float64, device=v.device)
        if h0 is not None:
            h = h0.double()
        states, y = [h], torch.empty(B, L, H, P, dtype=torch.float64, device=v.device)
        for t in range(L):
            h = e[:, t, :, None, None] * h + k[:, t, :, :, None] * v[:, t, :, None, :]
            y[:, t] = (q[:, t, :, :, None] * h).sum(2)
            states.append(h)
        out = {"y": y, "h_final": h}
        if dy is None:
            return out
        dy = dy.double()
        a = torch.zeros_like(h) if dh is None else dh.double()
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dg = torch.empty(B, L, H, dtype=torch.float64, device=v.device)
        for t in range(L - 1, -1, -1):
            dq[:, t] = (states[t + 1] * dy[:, t, :, None, :]).sum(3)
            a = a + q[:, t, :, :, None] * dy[:, t, :, None, :]
            dk[:, t] = (a * v[:, t, :, None, :]).sum(3)
            dv[:, t] = (a * k[:, t, :, :, None]).sum(2)
            a = e[:, t, :, None, None] * a
            dg[:, t] = (a * states[t]).sum((-1, -2))
        out["dq"], out["dk"] = (t.reshape(B, L, G, share, N).sum(3) for t in (dq, dk))
        out["dv"], out["dh0"] = dv, a
        out["dlog_decay"] = dg
        out["terms"] = (q * dq + k * dk).sum(-1)
        return out

    def size(t):
        return None if t is None else t.abs()

    want = walk(q, k, v, h0, dy, dh)
    most = walk(size(q), size(k), size(v), size(h0), size(dy), size(dh))
    if dy is not None:
        later = torch.zeros(B, H, dtype=torch.float64, device=v.device)
        if dh is not None:
            later = (dh.double().abs() * most["h_final"]).sum((-1, -2))
        sums = torch.empty_like(g)
        passes = g * 1.4426950408889634 >= -126
        for t in range(L - 1, -1, -1):
            later = later + most["terms"][:, t]
            sums[:, t] = later
            later = torch.where(passes[:, t], later, torch.zeros_like(later))
        most["dlog_decay"] = sums
        want["dlog_decay"] = torch.where(passes, want["dlog_decay"], torch.zeros_like(g))
        if log_decay.dim() == 1:
            want["dlog_decay"], most["dlog_decay"] = (d["dlog_decay"].sum((0, 1)) for d in (want, most))
    return want, most


def roundings(N, P, L, terms3=True):
    """How many half steps of fp32 (relative to the sums of absolute values) an
    output may be off: one per addition along the way of a product into it --
    at most the products of one key and of one value row (N + P), a chunk's 64
    tokens through 64-token sums twice, per chunk passed the carry's exponential
    (2 ulp), product and sum -- and 32 for the splits (2^-24 each, three), the
    exponentials of the decays and the last conversions."""
    chunks = -(-L // 64)
    m = N + P + 128 + 6 * chunks + 32
    return m * U32 + (0.0 if terms3 else 2 * 2.0 ** -16)


def sort_tokens(idx, E):
    T, k = idx.shape
    flat = idx.reshape(-1)
    order, offsets = [], [0]
    for e in range(E):
        order += [s for s in range(T * k) if flat[s] == e]
        offsets.append(len(order))
    pos = -np.ones(T * k, np.int64)
    pos[order] = np.arange(len(order))
    return np.array(order + [-1] * (T * k - len(order))), pos.reshape(T, k), np.array(offsets)


def combine(rows, pos, gate):
    T, k = pos.shape
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < T * k:
                y[t] += (1.0 if gate is None else gate[t, j]) * rows[pos[t, j]]
    return y


def combine_backward(rows, pos, gate, dy, drows):
    T, k = pos.shape
    drows, dgate = np.array(drows, np.float64), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < T * k:
                drows[pos[t, j]] = gate[t, j] * dy[t]
                dgate[t, j] = dy[t] @ rows[pos[t, j]]
    return drows, dgate


def route_backward(x, Wr, idx, gate, dgate):
    T, k = idx.shape
    dx, dW = np.zeros_like(x), np.zeros_like(Wr)
    sx, sW = np.zeros_like(x), np.zeros_like(Wr)
    mean = (gate * dgate).sum(1)
    size = (np.abs(gate * dgate)).sum(1)
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < Wr.shape[1]:
                continue
            s = gate[t, j] * (dgate[t, j] - mean[t])
            z = gate[t, j] * (abs(dgate[t, j]) + size[t])
            dx[t] += s * Wr[:, e]
            dW[:, e] += s * x[t]
            sx[t] += z * np.abs(Wr[:, e])
            sW[:, e] += z * np.abs(x[t])
    return dx, dW, sx, sW

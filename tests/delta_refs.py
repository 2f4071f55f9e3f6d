"""64-bit references of the gated delta rule and of the norms of queries and keys,
straight from their definitions, and how far outputs may be off.  Nothing here is
shared with the library.

The bounds of the delta rule.  Its writes cancel (v - h^T k), so sums over absolute values
of the whole sequence would grow without limit.  But a token's transition
e^g (I - beta k k^T) has the norm e^g max(1, |1 - beta |k|^2|), so an error of a state's
column grows by no more than that.  bounds() therefore walks the sequence in the chunks of 64
that products are made over, takes each chunk's own roundings from sums over absolute
values inside it, and carries them on as the 2-norm of each column."""
from __future__ import annotations

import numpy as np
import torch

U0 = 2.0 ** -24   # half a step of fp32
U = 3 * U0        # per term of a sum whose products take three steps
S = 2.0 ** -27    # what three bf16 terms leave out
S2 = 2.0 ** -18   # and two
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
CHUNK = 64


def delta(q, k, v, g, beta, h0=None, dy=None, dh=None):
    """fp64 tensors q, k [B,L,G,N], v [B,L,H,P], g [H] or [B,L,H], beta [B,L,H].  A dict of y,
    h_final and, with dy, the gradients."""
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    share = H // G
    e = g.expand(B, L, H).exp()
    qh, kh = (t.repeat_interleave(share, dim=2) for t in (q, k))
    h = torch.zeros(B, H, N, P, dtype=torch.float64) if h0 is None else h0.clone()
    y = torch.zeros(B, L, H, P, dtype=torch.float64)
    kept = []
    for t in range(L):
        ht = e[:, t, :, None, None] * h
        o = v[:, t] - (ht * kh[:, t, :, :, None]).sum(2)
        h = ht + kh[:, t, :, :, None] * (beta[:, t, :, None] * o)[:, :, None]
        y[:, t] = (h * qh[:, t, :, :, None]).sum(2)
        kept.append((ht, o, h))
    out = {"y": y, "h_final": h}
    if dy is None:
        return out
    a = torch.zeros_like(h) if dh is None else dh.clone()
    dq, dk, dv = torch.zeros_like(qh), torch.zeros_like(kh), torch.zeros_like(v)
    dg, db = torch.zeros(B, L, H, dtype=torch.float64), torch.zeros(B, L, H, dtype=torch.float64)
    for t in range(L - 1, -1, -1):
        ht, o, after = kept[t]
        k1, b = kh[:, t, :, :, None], beta[:, t, :, None]
        dq[:, t] = (after * dy[:, t, :, None]).sum(-1)
        a = a + qh[:, t, :, :, None] * dy[:, t, :, None]
        du = (a * k1).sum(2)
        db[:, t] = (du * o).sum(-1)
        do = b * du
        dv[:, t] = do
        dk[:, t] = (a * (b * o)[:, :, None]).sum(-1) - (ht * do[:, :, None]).sum(-1)
        a = a - k1 * do[:, :, None]
        dg[:, t] = (a * ht).sum((-1, -2))
        a = e[:, t, :, None, None] * a
    out["dq"], out["dk"] = (t.reshape(B, L, G, share, N).sum(3) for t in (dq, dk))
    out["dv"], out["dbeta"], out["dh0"] = dv, db, a
    out["dlog_decay"] = dg.sum((0, 1)) if g.dim() == 1 else dg
    return out


def _chunks(t, heads, C):
    """[B, L, h, n] as [B, heads, chunks, C, n], zeros behind the last token."""
    B, L, h, n = t.shape
    t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, -L % C))
    t = t.reshape(B, -1, C, h, n).permute(0, 3, 1, 2, 4)
    return t.repeat_interleave(heads // h, dim=1)


def _tokens(t, L):
    B, h, c, C, n = t.shape
    return t.permute(0, 2, 3, 1, 4).reshape(B, c * C, h, n)[:, :L]


def bounds(f32, q, k, v, g, beta, h0=None, dy=None, dh=None, y_bf16=False):
    """How far each of delta()'s outputs may be off, apart from its own type's last rounding.
    f32: the inputs are fp32 (three terms in products; bf16 is exact).

    A product of an input and a computed operand is off by cx of the product of sizes, of two
    computed operands by cc, of two inputs by ci (each operand's S, and 2 S for the two pairs of
    terms left out); each sum of n terms by 3 n U where products take three terms.  A
    y in bf16 is made from two terms (S2, and S2 for the pair left out)."""
    cx, cc, ci = (4 * S, 4 * S, 4 * S) if f32 else (S, 4 * S, 0.0)
    yx, yc = (3 * S2 if f32 else S2, 3 * S2) if y_bf16 else (cx, cc)
    B, L, H, P = v.shape
    heads, N = q.shape[2:]
    Q, K, V = (_chunks(t, H, CHUNK) for t in (q, k, v))
    b = _chunks(beta.unsqueeze(-1), H, CHUNK)
    gg = _chunks(g.expand(B, L, H).clamp(min=-2000.0).unsqueeze(-1), H, CHUNK)[..., 0]
    nc = Q.shape[2]
    Gs = gg.cumsum(-1)
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool).tril()
    low = (Gs.unsqueeze(-1) - Gs.unsqueeze(-2)).masked_fill(~tri, -2000.0)
    D = low.exp()
    # an exponential of a difference x rounded to fp32: |x| + 8 half steps
    dD = D * (low.abs() * 1.4427 + 8) * U
    eG, w = Gs.exp().unsqueeze(-1), (Gs[..., -1:] - Gs).exp().unsqueeze(-1)
    end = eG[..., -1:, :]
    grow = (1 - b * (K * K).sum(-1, keepdim=True)).abs().clamp(min=1.0)  # [.., C, 1]
    upto = eG * grow.cumprod(-2)
    behind = w * grow.flip(-2).cumprod(-2).flip(-2)
    whole = (end * grow.prod(-2, keepdim=True))[..., 0, 0]
    aK, aQ, ab = K.abs(), Q.abs(), b.abs()
    bT = ab.transpose(-1, -2)
    KK = K @ K.transpose(-1, -2)
    aKK, aQK = aK @ aK.transpose(-1, -2), aQ @ aK.transpose(-1, -2)
    strict = D.tril(-1)
    A = strict * KK * b.transpose(-1, -2)
    dA = bT * ((ci + (N + 4) * U) * strict + dD.tril(-1)) * aKK
    eye = torch.eye(CHUNK, dtype=torch.float64)
    T = torch.linalg.inv(eye + A)
    aT = T.abs()
    # the computed inverse of I + A + dA, and what its own roundings (2 x 64 terms) leave
    eT = aT @ (dA + 128 * U * (eye + A.abs())) @ aT
    Sc = D * (Q @ K.transpose(-1, -2))
    eS = ((ci + (N + 4) * U) * D + dD) * aQK
    aS = Sc.abs()

    h = torch.zeros(B, H, N, P, dtype=torch.float64) if h0 is None else h0.clone()
    eh = torch.zeros(B, H, 1, P, dtype=torch.float64)
    states, ehs, Os, eOs, ey = [], [], [], [], []
    for c in range(nc):
        states.append(h)
        ehs.append(eh)
        ah = h.abs()
        Kc, aKc, aTc, wc, bc = K[:, :, c], aK[:, :, c], aT[:, :, c], w[:, :, c], b[:, :, c]
        z = aKc @ ah
        R = V[:, :, c] - eG[:, :, c] * (Kc @ h)
        eR = eG[:, :, c] * (cx + (N + 8) * U) * z + 2 * U * V[:, :, c].abs()
        O = T[:, :, c] @ R
        eO = aTc @ eR + (eT[:, :, c] + (cc + 64 * U) * aTc) @ (R.abs() + eR)
        Uc, eU = bc * O, bc.abs() * (eO + U * O.abs())
        here = (eG[:, :, c] * (yx + (N + 8) * U) * (aQ[:, :, c] @ ah) + aS[:, :, c] @ eU
                + (eS[:, :, c] + (yc + 66 * U) * aS[:, :, c]) @ (Uc.abs() + eU))
        ey.append(here + Q[:, :, c].norm(dim=-1, keepdim=True) * upto[:, :, c] * eh)
        Os.append(O)
        eOs.append(eO + Kc.norm(dim=-1, keepdim=True) * upto[:, :, c] * eh)
        eh_here = aKc.transpose(-1, -2) @ (wc * (eU + (cx + 72 * U) * Uc.abs())) + 4 * U * end[:, :, c] * ah
        h = end[:, :, c] * h + Kc.transpose(-1, -2) @ (wc * Uc)
        eh = whole[:, :, c, None, None] * eh + eh_here.norm(dim=2, keepdim=True) + U * h.norm(dim=2, keepdim=True)
    out = {"y": _tokens(torch.stack(ey, 2), L), "h_final": eh.expand(B, H, N, P)}
    if dy is None:
        return out

    dY = _chunks(dy, H, CHUNK)
    a = torch.zeros_like(h) if dh is None else dh.clone()
    ea = torch.zeros_like(eh)
    per = {n: [None] * nc for n in ("dq", "dk", "dv", "dbeta", "dg")}
    for c in range(nc - 1, -1, -1):
        h, eh, O, eO = states[c], ehs[c], Os[c], eOs[c]
        aa, ah, aO = a.abs(), h.abs(), O.abs()
        Kc, Qc, aKc, aQc, dYc, ady = K[:, :, c], Q[:, :, c], aK[:, :, c], aQ[:, :, c], dY[:, :, c], dY[:, :, c].abs()
        Tt, aTt, eTt = (t[:, :, c].transpose(-1, -2) for t in (T, aT, eT))
        St, aSt, eSt = (t[:, :, c].transpose(-1, -2) for t in (Sc, aS, eS))
        wc, bc, er, ec = w[:, :, c], b[:, :, c], eG[:, :, c], end[:, :, c]
        abc, bTc = bc.abs(), bT[:, :, c]
        dU = St @ dYc + wc * (Kc @ a)
        edU = (eSt + (cx + 66 * U) * aSt) @ ady + wc * (cx + (N + 8) * U) * (aKc @ aa)
        X, eX = bc * dU, abc * (edU + U * dU.abs())
        dV = Tt @ X
        edV = aTt @ eX + (eTt + (cc + 64 * U) * aTt) @ (X.abs() + eX)
        edVall = edV + abc * Kc.norm(dim=-1, keepdim=True) * behind[:, :, c] * ea
        adV = dV.abs()
        per["dv"][c] = edVall
        ea_here = ((aQc.transpose(-1, -2) @ (er * ady) + aKc.transpose(-1, -2) @ (er * adV)) * (cx + 72 * U)
                   + aKc.transpose(-1, -2) @ (er * edV) + 4 * U * ec * aa)
        # the other gradients
        Ot, aOt, eOt = (t.transpose(-1, -2) for t in (O, aO, eO))
        ht, aht, at, aat = h.transpose(-1, -2), ah.transpose(-1, -2), a.transpose(-1, -2), aa.transpose(-1, -2)
        one = torch.ones(N, dtype=torch.float64)
        F = dYc @ Ot
        eF = ady @ eOt + (cx + P * U) * ady @ aOt
        E = dV @ Ot
        eE = edVall @ aOt + adV @ eOt + (cc + P * U) * adV @ aOt
        Dc, dDc = D[:, :, c], dD[:, :, c]
        reads, eread = dYc @ ht, (ady @ eh.transpose(-1, -2)) * one + (cx + P * U) * ady @ aht
        erased, eer = dV @ ht, (adV @ eh.transpose(-1, -2)) * one + edVall @ aht + (cc + P * U) * adV @ aht
        written, ewr = O @ at, (aO @ ea.transpose(-1, -2)) * one + eO @ aat + (cc + P * U) * aO @ aat
        FD, eFD = Dc * F.abs() * bTc, bTc * (Dc * eF + (dDc + 2 * U * Dc) * F.abs())
        Ds = Dc.tril(-1)
        ED, eED = Ds * E.abs() * bTc, bTc * (Ds * eE + (dDc.tril(-1) + 2 * U * Ds) * E.abs())
        mix = cx + 66 * U
        per["dq"][c] = er * (eread + 6 * U * reads.abs()) + (eFD + mix * FD) @ aKc
        both, eboth = ED + ED.transpose(-1, -2), eED + eED.transpose(-1, -2)
        per["dk"][c] = (abc * wc * (ewr + 8 * U * written.abs()) + er * (eer + 6 * U * erased.abs())
                        + (eFD + (mix + 64 * U) * FD).transpose(-1, -2) @ aQc + (eboth + (mix + 64 * U) * both) @ aKc)
        # pairs before beta: D (q.k F - k.k E)
        aqk, akk = aQK[:, :, c], aKK[:, :, c]
        QKc, KKc = (Qc @ Kc.transpose(-1, -2)).abs(), KK[:, :, c].abs()
        size = Dc * QKc * F.abs() + Ds * KKc * E.abs()
        epair = (QKc * (Dc * eF + dDc * F.abs()) + Dc * (ci + (N + 4) * U) * aqk * F.abs()
                 + KKc * (Ds * eE + dDc.tril(-1) * E.abs()) + Ds * (ci + (N + 4) * U) * akk * E.abs() + 140 * U * size)
        ewrote = wc * ((aKc * (ewr + (N + 8) * U * written.abs())).sum(-1, keepdim=True))
        per["dbeta"][c] = epair.sum(-2).unsqueeze(-1) + ewrote + 4 * U * (size.sum(-2).unsqueeze(-1) + wc * (aKc * written.abs()).sum(-1, keepdim=True))
        eseen = er * (aQc * (eread + (2 * N + 8) * U * reads.abs()) + aKc * (eer + (2 * N + 8) * U * erased.abs())).sum(-1, keepdim=True)
        through = ec * (ah * ea + aa * eh + ah * aa * (N * P / 16 + 8) * U).sum((-1, -2), keepdim=True)
        # any token's dg sums pairs of its chunk and document: those up to it and from it on
        allpairs = (epair * bTc).sum((-1, -2), keepdim=True)
        edg = allpairs + eseen.flip(-2).cumsum(-2).flip(-2) + (abc * ewrote).cumsum(-2) + through
        per["dg"][c] = edg
        a_next = ec * a + Qc.transpose(-1, -2) @ (er * dYc) - Kc.transpose(-1, -2) @ (er * dV)
        ea = whole[:, :, c, None, None] * ea + ea_here.norm(dim=2, keepdim=True) + U * a_next.norm(dim=2, keepdim=True)
        a = a_next
    share = H // heads
    tok = {n: _tokens(torch.stack(x, 2), L) for n, x in per.items()}
    for n in ("dq", "dk"):
        out[n] = tok[n].reshape(B, L, heads, share, N).sum(3)
    out["dv"], out["dbeta"], out["dh0"] = tok["dv"], tok["dbeta"][..., 0], ea.expand(B, H, N, P)
    dg = tok["dg"][..., 0]
    out["dlog_decay"] = dg.sum((0, 1)) if g.dim() == 1 else dg
    return out


def norm_rotate(q, k, wq, wk, pos, rates, norm, pairs, eps, q_scale, dq=None, dk=None):
    """fp64 arrays q [T, Hq, N], k [T, Hk, N].  A dict of q, k and, with dq, of dq, dk, dwq,
    dwk; and of their sizes (the sums over absolute values)."""
    out, size = {}, {}
    N = q.shape[-1]
    R = 0 if rates is None else 2 * len(rates)
    c = 1.0 / N if norm == "rms" else 1.0
    i = np.arange(R // 2)
    first, second = (i, i + R // 2) if pairs == "halves" else (2 * i, 2 * i + 1)

    def turn(x, sign):
        y = x.copy()
        m = np.abs(x)
        if R:
            z = pos[:, None, None].astype(np.float64) * rates.astype(np.float64)
            co, si = np.cos(z), sign * np.sin(z)
            a, b = x[..., first], x[..., second]
            y[..., first], y[..., second] = a * co - b * si, b * co + a * si
            m[..., first] = m[..., second] = np.abs(a) + np.abs(b)
        return y, m

    for n, x, w, d in (("q", q, wq, dq), ("k", k, wk, dk)):
        scale = q_scale if n == "q" else 1.0
        w = np.ones(N) if w is None else w
        r = 1.0 / np.sqrt(c * (x * x).sum(-1, keepdims=True) + eps)
        y, m = turn(x * r * w, 1.0)
        out[n], size[n] = scale * y, abs(scale) * m
        if d is None:
            continue
        g, gm = turn(scale * d, -1.0)
        out["dw" + n] = (g * x * r).sum((0, 1))
        size["dw" + n] = (gm * np.abs(x * r)).sum((0, 1))
        dot = (g * w * x * r).sum(-1, keepdims=True)
        dm = (gm * np.abs(w * x * r)).sum(-1, keepdims=True)
        out["d" + n] = r * (g * w - x * r * c * dot)
        size["d" + n] = r * (gm * np.abs(w) + np.abs(x * r) * c * dm)
    return out, size

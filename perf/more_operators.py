"""The gated delta rule (prompt, training step, single token) and the norms and
rotation of queries and keys (forward, training step), as cases to be timed and
checked.

With `own` false `run` computes them in elementary torch operations; with `own`
true it calls the library's entry points."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # a 64K-token prompt: D = 2560 as 40 heads of 64, one key head shared by all, a decay per token and head
        {"name": "delta_prompt_long", "op": "delta", "B": 1, "L": 65536, "H": 40, "G": 1, "N": 128, "P": 64,
         "decay": "token", "dtype": "bf16", "h0": False, "reset": 0},
        # a batch of prompts on the 1.4B-like layer, D = 4096 as 32 heads of 128 with their own keys, a fixed decay per head
        {"name": "delta_prompt_1p4b", "op": "delta", "B": 8, "L": 4096, "H": 32, "G": 32, "N": 128, "P": 128,
         "decay": "head", "dtype": "bf16", "h0": True, "reset": 0},
        # packed documents of odd sizes in fp32, continued from a state
        {"name": "delta_prompt_odd_f32", "op": "delta", "B": 2, "L": 1537, "H": 6, "G": 2, "N": 80, "P": 50,
         "decay": "token", "dtype": "f32", "h0": True, "reset": 300},
        # a training step of the 130M-like layer, D = 1536 as 24 heads of 64
        {"name": "delta_train_130m", "op": "delta_train", "B": 4, "L": 2048, "H": 24, "G": 24, "N": 64, "P": 64,
         "decay": "head", "dtype": "bf16", "h0": False, "reset": 0},
        # a training step at D = 4096 with keys shared by eight heads, a decay per token, packed documents
        {"name": "delta_train_shared", "op": "delta_train", "B": 2, "L": 4096, "H": 32, "G": 4, "N": 128, "P": 128,
         "decay": "token", "dtype": "bf16", "h0": True, "reset": 1000},
        # one decode step of 256 sequences, D = 5120 as 40 heads of 128
        {"name": "delta_step_decode", "op": "delta_step", "B": 256, "H": 40, "G": 40, "N": 128, "P": 128,
         "decay": "token", "dtype": "bf16"},
        # one decode step of a single sequence on the 130M-like layer: latency
        {"name": "delta_step_one", "op": "delta_step", "B": 1, "H": 24, "G": 1, "N": 128, "P": 64,
         "decay": "head", "dtype": "bf16"},
        # queries and keys of a 64K-token prompt, 40 and 8 heads of 64, weights, half-split pairs
        {"name": "norm_prompt_long", "op": "norm", "T": 65536, "Hq": 40, "Hk": 8, "N": 64, "R": 64, "pairs": "halves",
         "norm": "rms", "weights": True, "dtype": "bf16", "far": 0},
        # a decode batch, unit vectors without rotation: latency
        {"name": "norm_decode", "op": "norm", "T": 256, "Hq": 40, "Hk": 40, "N": 128, "R": 0, "pairs": "halves",
         "norm": "l2", "weights": False, "dtype": "bf16", "far": 0},
        # a training step of 32K tokens, 32 and 4 heads of 128: forward and the gradients
        {"name": "norm_train", "op": "norm_train", "T": 32768, "Hq": 32, "Hk": 4, "N": 128, "R": 128, "pairs": "halves",
         "norm": "rms", "weights": True, "dtype": "bf16", "far": 0},
        # odd sizes in fp32, part of each head turned, neighbours as pairs, positions around a million
        {"name": "norm_train_odd_f32", "op": "norm_train", "T": 5001, "Hq": 6, "Hk": 2, "N": 80, "R": 48,
         "pairs": "neighbours", "norm": "l2", "weights": True, "dtype": "f32", "far": 1000000},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_train", "delta_train", "delta_step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = [16, 32, 64, 128, rng.randint(9, 127), 2 * rng.randint(5, 63)]
    if op.startswith("norm"):
        N = rng.choice(wide)
        case = {"op": op, "T": _log_int(rng, 1, 65536 if op == "norm" else 32768), "Hq": _log_int(rng, 1, 48), "N": N,
                "R": rng.choice([0, N // 2 * 2, 2 * rng.randint(1, N // 2)]), "pairs": rng.choice(["halves", "neighbours"]),
                "norm": rng.choice(["rms", "l2"]), "weights": rng.random() < 0.5, "dtype": dtype,
                "far": rng.choice([0, 0, 1000000])}
        case["Hk"] = min(case["Hq"], _log_int(rng, 1, 48))
        case["T"] = max(1, min(case["T"], (1 << 27) // ((case["Hq"] + case["Hk"]) * N)))
        return case
    heads = _log_int(rng, 1, 48)
    group = rng.choice([g for g in range(1, heads + 1) if heads % g == 0])
    case = {"op": op, "B": _log_int(rng, 1, 8), "H": heads, "G": group, "N": rng.choice(wide), "P": rng.choice(wide),
            "decay": rng.choice(["head", "token"]), "dtype": dtype}
    if op == "delta_step":
        case["B"] = _log_int(rng, 1, 256)
        return case
    most = (1 << 20) if op == "delta" else (1 << 17)
    case["L"] = max(1, min(_log_int(rng, 1, 65536), most // (case["B"] * heads)))
    case["h0"] = rng.random() < 0.5
    case["reset"] = rng.choice([0, 0, 100, 700]) if case["decay"] == "token" else 0
    return case


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV).to(dtype)

    st = {"case": case, "op": case["op"]}
    if case["op"].startswith("norm"):
        T, N, R = case["T"], case["N"], case["R"]
        train = case["op"] == "norm_train"
        for n in "qk":
            heads = case["H" + n]
            st[n] = normal(T, heads, N, dtype=dt)
            st["w" + n] = 1 + 0.1 * normal(N) if case["weights"] else None
            if train:
                st["d" + n] = normal(T, heads, N, dtype=dt)
        st["pos"] = st["rates"] = None
        if R:
            st["pos"] = torch.arange(case["far"], case["far"] + T, dtype=torch.int32, device=DEV)
            st["rates"] = torch.pow(10000.0, -torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R).float()
        return st
    B, H, G, N, P = (case[n] for n in "BHGNP")
    lead = (B, case["L"]) if "L" in case else (B,)

    def unit():  # as the norm of queries and keys leaves them
        x = normal(*lead, G, N)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    st["q"], st["k"], st["v"] = unit(), unit(), normal(*lead, H, P, dtype=dt)
    st["beta"] = torch.sigmoid(normal(*lead, H))
    if case["decay"] == "head":  # from 1 - 1/8 to 1 - 1/1024 over the heads
        st["g"] = torch.log1p(-torch.exp2(-torch.linspace(3, 10, H, device=DEV)))
    else:  # a softplus step times a rate per head, as the scans' exp(Delta A)
        rate = torch.exp(torch.rand(H, generator=gen, device=DEV) * math.log(16.0)) / 16
        st["g"] = -torch.nn.functional.softplus(normal(*lead, H) - 2) * rate
        if case.get("reset"):  # a document begins: the state is cleared
            starts = torch.rand(lead, generator=gen, device=DEV) < 1.0 / case["reset"]
            st["g"] = st["g"].masked_fill(starts.unsqueeze(-1), -math.inf)
    st["g"] = st["g"].float().contiguous()
    state = case["op"] == "delta_step" or case["h0"]
    st["h0"] = normal(B, H, N, P) if state else None
    if case["op"] == "delta_train":
        st["dy"] = normal(*lead, H, P, dtype=dt)
        st["dh"] = normal(B, H, N, P) if state else None
    return st


# ---- plain forms -----------------------------------------------------------

CHUNK, BLOCK = 64, 16


def _split(t, C, heads):
    """[B, L, h, n] as [B, heads, chunks, C, n], zero-padded, shared heads repeated."""
    B, L, h, n = t.shape
    t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, -L % C))
    t = t.reshape(B, -1, C, h, n).permute(0, 3, 1, 2, 4)
    return t.repeat_interleave(heads // h, dim=1) if heads != h else t


def _join(t, L):
    """[B, h, chunks, C, n] back to [B, L, h, n]."""
    B, h, c, C, n = t.shape
    return t.permute(0, 2, 3, 1, 4).reshape(B, c * C, h, n)[:, :L]


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., 64, 64], in 64 bits: products for
    the blocks of 16 on the diagonal, then blocks joined in twos."""
    def block(a):  # the sum of (-a)^i, i < 16
        eye = torch.eye(a.shape[-1], dtype=a.dtype, device=a.device)
        a2 = torch.matmul(a, a)
        a4 = torch.matmul(a2, a2)
        even = torch.matmul(eye + a4, eye + torch.matmul(a4, a4))
        return torch.matmul(torch.matmul(eye - a, eye + a2), even)

    n = A.shape[-1]
    if n == BLOCK:
        return block(A)
    h = n // 2
    first, last = _inverse(A[..., :h, :h]), _inverse(A[..., h:, h:])
    low = -torch.matmul(torch.matmul(last, A[..., h:, :h]), first)
    return torch.cat([torch.cat([first, torch.zeros_like(first)], -1), torch.cat([low, last], -1)], -2)


def _delta_forward(st):
    q, k, v = st["q"], st["k"], st["v"]
    B, L, H, P = v.shape
    N = q.shape[-1]
    Q, K, V = (_split(t.float(), CHUNK, H) for t in (q, k, v))
    beta = _split(st["beta"].unsqueeze(-1), CHUNK, H)  # [B, H, c, C, 1]
    # sums of log decays in 64 bits; e^-1000 is zero, and differences stay finite
    g = st["g"].double().clamp(min=-1000.0).expand(B, L, H)
    G = _split(g.unsqueeze(-1), CHUNK, H)[..., 0].cumsum(-1)  # [B, H, c, C]
    c = G.shape[2]
    D = G.unsqueeze(-1) - G.unsqueeze(-2)
    later = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).triu(1)
    D = D.masked_fill_(later, -math.inf).exp_().float()
    eG = G.exp().float().unsqueeze(-1)
    w = (G[..., -1:] - G).exp().float().unsqueeze(-1)
    end = eG[..., -1:, :]  # [B, H, c, 1, 1]
    KK = torch.matmul(K, K.transpose(-1, -2)) * D
    T = _inverse((KK.tril(-1) * beta.transpose(-1, -2)).double()).float()
    Ov, W = torch.matmul(T, V), torch.matmul(T, K * eG)  # O = Ov - W S
    Kw = K * w
    carry = torch.eye(N, device=q.device) * end - torch.matmul(Kw.transpose(-1, -2), beta * W)
    write = torch.matmul(Kw.transpose(-1, -2), beta * Ov)
    # the states before each chunk, and the last
    S = torch.zeros(c + 1, B * H, N, P, device=q.device)
    if st["h0"] is not None:
        S[0] = st["h0"].reshape(B * H, N, P)
    carry = carry.transpose(0, 2).reshape(c, H, B, N, N).transpose(1, 2).reshape(c, B * H, N, N)
    write = write.transpose(0, 2).reshape(c, H, B, N, P).transpose(1, 2).reshape(c, B * H, N, P)
    for i in range(c):
        torch.baddbmm(write[i], carry[i], S[i], out=S[i + 1])
    h = S.reshape(c + 1, B, H, N, P).permute(1, 2, 0, 3, 4)
    O = Ov - torch.matmul(W, h[:, :, :c])
    QK = torch.matmul(Q, K.transpose(-1, -2)) * D
    y = torch.matmul(QK, beta * O) + torch.matmul(Q * eG, h[:, :, :c])
    return {"y": _join(y, L).to(v.dtype).contiguous(), "h_final": h[:, :, c].contiguous(),
            "parts": (Q, K, V, beta, D, eG, w, end, KK, T, QK, carry, h, O)}


def _delta_backward(st, parts):
    Q, K, V, beta, D, eG, w, end, KK, T, QK, carry, h, O = parts
    B, L, H, P = st["v"].shape
    heads, N = st["q"].shape[2:]
    c = Q.shape[2]
    h = h[:, :, :c]
    dY = _split(st["dy"].float(), CHUNK, H)
    dU = torch.matmul(QK.transpose(-1, -2), dY)
    Tt, bT = T.transpose(-1, -2), beta.transpose(-1, -2)
    dVy = torch.matmul(Tt, beta * dU)  # dV = dVy + dVa a
    dVa = torch.matmul(Tt, beta * w * K)
    KeG = (K * eG).transpose(-1, -2)
    read = torch.matmul((Q * eG).transpose(-1, -2), dY) - torch.matmul(KeG, dVy)
    # the adjoints behind each chunk, and the first
    A = torch.zeros(c + 1, B * H, N, P, device=Q.device)
    if st["dh"] is not None:
        A[c] = st["dh"].reshape(B * H, N, P)
    read = read.transpose(0, 2).reshape(c, H, B, N, P).transpose(1, 2).reshape(c, B * H, N, P)
    back = carry.transpose(-1, -2).contiguous()
    for i in range(c - 1, -1, -1):
        torch.baddbmm(read[i], back[i], A[i + 1], out=A[i])
    a = A.reshape(c + 1, B, H, N, P).permute(1, 2, 0, 3, 4)
    dh0, a = a[:, :, 0].contiguous(), a[:, :, 1:]
    dV = dVy + torch.matmul(dVa, a)
    F = torch.matmul(dY, O.transpose(-1, -2))  # the scores' slopes, without D and beta
    E = torch.matmul(dV, O.transpose(-1, -2))
    FD, ED = F * D * bT, E * D.tril(-1) * bT
    reads, erased, written = (torch.matmul(t, s.transpose(-1, -2)) for t, s in ((dY, h), (dV, h), (O, a)))
    dQ = eG * reads + torch.matmul(FD, K)
    dK = (beta * w * written - eG * erased + torch.matmul(FD.transpose(-1, -2), Q)
          - torch.matmul(ED + ED.transpose(-1, -2), K))
    KK = KK.tril(-1)
    wrote = w * (K * written).sum(-1, keepdim=True)
    dbeta = (QK * F - KK * E).sum(-2).unsqueeze(-1) + wrote
    # a log decay scales what later tokens read of earlier ones
    pairs = ((QK * F - KK * E) * bT).double()
    rect = pairs.sum(-2) - pairs.sum(-1)  # the sum over r >= t > s, from its differences
    rect = rect.cumsum(-1) - rect
    seen = (eG * (Q * reads - K * erased).sum(-1, keepdim=True)).squeeze(-1).double()
    wrote = (beta * wrote).squeeze(-1).double()
    through = end.squeeze(-1).double() * (h.double() * a.double()).sum((-1, -2)).unsqueeze(-1)
    dg = rect + seen.flip(-1).cumsum(-1).flip(-1) + (wrote.cumsum(-1) - wrote) + through
    dg = _join(dg.unsqueeze(-1), L)[..., 0]
    dg = dg.masked_fill(st["g"].expand(B, L, H) == -math.inf, 0.0)  # e^g is zero there, and so is its slope
    if st["g"].dim() == 1:
        dg = dg.sum((0, 1))
    dt = st["v"].dtype

    def shared(t):
        return _join(t, L).reshape(B, L, heads, H // heads, N).sum(3).to(dt)

    return {"dq": shared(dQ), "dk": shared(dK), "dv": _join(dV, L).to(dt).contiguous(), "dlog_decay": dg.float(),
            "dbeta": _join(dbeta, L)[..., 0].contiguous(), "dh0": dh0}


def _delta_step(st):
    B, H, P = st["v"].shape
    share = H // st["q"].shape[1]
    q = st["q"].float().repeat_interleave(share, dim=1).unsqueeze(-1)
    k = st["k"].float().repeat_interleave(share, dim=1).unsqueeze(-1)
    h = st["h0"] * st["g"].exp().expand(B, H)[..., None, None]
    u = st["beta"].unsqueeze(-1) * (st["v"].float() - (h * k).sum(-2))
    h = h + k * u.unsqueeze(-2)
    return {"y": (h * q).sum(-2).to(st["v"].dtype), "state": h}


def _turn(x, cos, sin, pairs, R):
    """The first R columns of x [T, heads, N], in pairs, turned; cos and sin [T, 1, R/2]."""
    r = x[..., :R]
    if pairs == "halves":
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, x[..., R:]], -1)


def _norm(st):
    case = st["case"]
    N, R = case["N"], case["R"]
    c = 1.0 / N if case["norm"] == "rms" else 1.0
    cos = sin = None
    if R:
        angle = (st["pos"].double().unsqueeze(-1) * st["rates"].double()).unsqueeze(1)
        cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for n, scale in (("q", N ** -0.5), ("k", 1.0)):
        x, w = st[n].float(), st["w" + n]
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) * c + EPS)
        y = x * r if w is None else x * r * w
        if R:
            y = _turn(y, cos, sin, case["pairs"], R)
        out[n] = (y * scale).to(st[n].dtype)
        if case["op"] == "norm_train":
            d = st["d" + n].float() * scale
            if R:
                d = _turn(d, cos, -sin, case["pairs"], R)
            if w is not None:
                out["dw" + n] = (d * x * r).sum((0, 1))
                d = d * w
            dx = r * (d - x * (r * r * c * (d * x).sum(-1, keepdim=True)))
            out["d" + n] = dx.to(st[n].dtype)
    return out


def run(st):
    op = st["op"]
    if own:
        return _run_own(st, op)
    if op in ("delta", "delta_train"):
        f = _delta_forward(st)
        out = {"y": f["y"], "h_final": f["h_final"]}
        return {**out, **_delta_backward(st, f["parts"])} if op == "delta_train" else out
    return _delta_step(st) if op == "delta_step" else _norm(st)


def _run_own(st, op):
    from parameter_space_moe_amd import swimba
    if op in ("delta", "delta_train"):
        ops = (st["q"], st["k"], st["v"], st["g"], st["beta"])
        y, h = swimba.delta_rule(*ops, h0=st["h0"])
        out = {"y": y, "h_final": h}
        if op == "delta_train":
            out.update(swimba.delta_rule_backward(*ops, st["dy"], h0=st["h0"], dh_final=st["dh"],
                                                  grad_dtype=st["v"].dtype))
        return out
    if op == "delta_step":
        # a decode loop marshals its call once for its buffers (which the call holds); others get a call of their own
        ops = (st["q"], st["k"], st["v"], st["g"], st["beta"], st["h0"])
        made = st.get("made")
        if made is None or made[0] != list(map(id, ops)):
            out = torch.empty_like(st["h0"])
            made = st["made"] = (list(map(id, ops)), out, swimba.PreparedDeltaRuleStep(*ops, state_out=out))
        return {"y": made[2](), "state": made[1]}
    case = st["case"]
    how = {"norm": case["norm"], "pairs": case["pairs"], "eps": EPS, "q_scale": case["N"] ** -0.5,
           "wq": st["wq"], "wk": st["wk"], "positions": st["pos"], "rates": st["rates"]}
    out = dict(zip("qk", swimba.norm_rotate(st["q"], st["k"], **how)))
    if op == "norm_train":
        got = swimba.norm_rotate_backward(st["q"], st["k"], st["dq"], st["dk"], grad_dtype=st["q"].dtype, **how)
        out.update({n: t for n, t in got.items() if t is not None})
        # the order of the plain form
        out = {n: out[n] for x in "qk" for n in (x, "dw" + x, "d" + x) if n in out}
    return out


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        rows = case["T"] * (case["Hq"] + case["Hk"]) * case["N"]
        train = case["op"] == "norm_train"
        return {"bytes": rows * size * (4 if train else 2) + (4 * case["T"] if case["R"] else 0),
                "flops": rows * (16 if train else 6)}
    B, H, G, N, P = (case[n] for n in "BHGNP")
    t = B * case.get("L", 1)
    keys, values = t * G * N * size, t * H * P * size
    g = 4 * (H if case["decay"] == "head" else t * H)
    beta = 4 * t * H
    state = 4 * B * H * N * P
    if case["op"] == "delta_step":
        return {"bytes": 2 * keys + 2 * values + g + beta + 2 * state, "flops": 7 * B * H * N * P}
    first = 2 if case["h0"] else 1
    if case["op"] == "delta":
        return {"bytes": 2 * keys + 2 * values + g + beta + first * state, "flops": 6 * t * H * N * P}
    # y, h_final and the gradients of q, k, v, the decays, beta and the first state, from the inputs, dy and the last state's gradient
    return {"bytes": 4 * keys + 4 * values + 2 * g + 2 * beta + 2 * first * state, "flops": 20 * t * H * N * P}


# ---- 64 bits, from the definitions ----------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(st, case)
    return _exact_delta(st, case["op"])


def _exact_norm(st, case):
    N, R = case["N"], case["R"]
    # as complex numbers: a pair is turned by a factor of size one
    if R:
        angle = st["pos"].double()[:, None] * st["rates"].double()
        turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
        first = torch.arange(R // 2, device=DEV) * (1 if case["pairs"] == "halves" else 2)
        second = first + (R // 2 if case["pairs"] == "halves" else 1)

    def turned(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    out = {}
    for n in "qk":
        x = st[n].double()
        w = torch.ones(N, dtype=torch.float64, device=DEV) if st["w" + n] is None else st["w" + n].double()
        scale = N ** -0.5 if n == "q" else 1.0
        size = ((x ** 2).sum(-1) / (N if case["norm"] == "rms" else 1) + EPS).sqrt().unsqueeze(-1)
        z = x / size
        y = z * w
        out[n] = scale * (turned(y, turn) if R else y)
        if case["op"] != "norm_train":
            continue
        d = st["d" + n].double() * scale
        if R:
            d = turned(d, turn.conj())
        if st["w" + n] is not None:
            out["dw" + n] = (d * z).sum((0, 1))
        d = d * w
        along = (d * z).sum(-1, keepdim=True) / (N if case["norm"] == "rms" else 1)
        out["d" + n] = (d - z * along) / size
    return out


def _exact_delta(st, op):
    """The recurrence token by token, and its adjoint from the last token back (states kept every 64
    tokens, the others walked again)."""
    one = op == "delta_step"
    names = ("q", "k", "v", "beta")
    q, k, v, beta = (st[n].double().unsqueeze(1) if one else st[n].double() for n in names)
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    share = H // G
    g = st["g"].double()
    decay = (g.unsqueeze(1) if one and g.dim() == 2 else g).exp().expand(B, L, H)
    # token-major copies; q and k as columns for the state, v as a row
    q, k = (t.repeat_interleave(share, dim=2).transpose(0, 1).unsqueeze(-1).contiguous() for t in (q, k))
    v = v.transpose(0, 1).unsqueeze(-2).contiguous()
    e = decay.transpose(0, 1)[..., None, None].contiguous()
    beta = beta.transpose(0, 1)[..., None, None].contiguous()
    h = torch.zeros(B, H, N, P, dtype=torch.float64, device=DEV)
    if st["h0"] is not None:
        h += st["h0"].double()
    y = torch.empty(L, B, H, P, dtype=torch.float64, device=DEV)
    train, kept = op == "delta_train", []

    def step(h, t):
        """Updates h in place; returns what is written before beta."""
        h.mul_(e[t])
        o = v[t] - (h * k[t]).sum(-2, keepdim=True)
        h.addcmul_(k[t], beta[t] * o)
        return o

    for t in range(L):
        if train and t % 64 == 0:
            kept.append(h.clone())
        step(h, t)
        torch.sum(h * q[t], -2, out=y[t])
    out = {"y": y.transpose(0, 1) if not one else y[0], "state" if one else "h_final": h}
    if not train:
        return out
    a = torch.zeros_like(h) if st["dh"] is None else st["dh"].double()
    dy = st["dy"].double().transpose(0, 1).unsqueeze(-2).contiguous()
    dq, dk = (torch.empty(L, B, H, N, dtype=torch.float64, device=DEV) for _ in range(2))
    dv = torch.empty_like(y)
    dg, dbeta = (torch.empty(L, B, H, dtype=torch.float64, device=DEV) for _ in range(2))
    for t0 in range((L - 1) // 64 * 64, -1, -64):
        states, written = [kept[t0 // 64]], []
        for t in range(t0, min(L, t0 + 64)):
            states.append(states[-1].clone())
            written.append(step(states[-1], t))
        for t in range(min(L, t0 + 64) - 1, t0 - 1, -1):
            after, before, o = states[t + 1 - t0], states[t - t0] * e[t], written[t - t0]
            torch.sum(after * dy[t], -1, out=dq[t])
            a = a.addcmul(q[t], dy[t])
            du = (a * k[t]).sum(-2, keepdim=True)
            dbeta[t] = (du * o).sum((-1, -2))
            do = beta[t] * du
            dv[t] = do.squeeze(-2)
            torch.sum(a * (beta[t] * o) - before * do, -1, out=dk[t])
            a = a - k[t] * do
            dg[t] = (a * before).sum((-1, -2))
            a = a * e[t]
    dg = dg.transpose(0, 1)

    def shared(t):
        return t.transpose(0, 1).reshape(B, L, G, share, N).sum(3)

    out.update(dq=shared(dq), dk=shared(dk), dv=dv.transpose(0, 1), dlog_decay=dg.sum((0, 1)) if g.dim() == 1 else dg,
               dbeta=dbeta.transpose(0, 1), dh0=a)
    return out

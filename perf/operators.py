"""The operators around the routed scan, as cases to be timed and checked: linear
attention with a decay per head (prompt, training step, single token), tokens
sorted by expert and back (out, back, training step), and the router's backward.

With `own` false `run` computes them in elementary torch operations; with `own`
true it calls the library's entry points."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a 64K-token prompt: D = 2560 as 40 heads of 64, one key head shared by all, a decay per token and head
        {"name": "la_prompt_long", "op": "la", "B": 1, "L": 65536, "H": 40, "G": 1, "N": 128, "P": 64,
         "decay": "token", "dtype": "bf16", "h0": False, "reset": 0},
        # a batch of prompts on the 1.4B-like layer, D = 4096 as 32 heads of 128 with their own keys, a fixed decay per head
        {"name": "la_prompt_1p4b", "op": "la", "B": 8, "L": 4096, "H": 32, "G": 32, "N": 128, "P": 128,
         "decay": "head", "dtype": "bf16", "h0": True, "reset": 0},
        # packed documents of odd sizes in fp32, continued from a state
        {"name": "la_prompt_odd_f32", "op": "la", "B": 2, "L": 1537, "H": 6, "G": 2, "N": 80, "P": 50,
         "decay": "token", "dtype": "f32", "h0": True, "reset": 300},
        # a training step of the 130M-like layer, D = 1536 as 24 heads of 64
        {"name": "la_train_130m", "op": "la_train", "B": 4, "L": 2048, "H": 24, "G": 24, "N": 64, "P": 64,
         "decay": "head", "dtype": "bf16", "h0": False, "reset": 0},
        # a training step at D = 4096 with keys shared by eight heads, a decay per token, packed documents
        {"name": "la_train_shared", "op": "la_train", "B": 2, "L": 4096, "H": 32, "G": 4, "N": 128, "P": 128,
         "decay": "token", "dtype": "bf16", "h0": True, "reset": 1000},
        # one decode step of 256 sequences, D = 5120 as 40 heads of 128
        {"name": "la_step_decode", "op": "la_step", "B": 256, "H": 40, "G": 40, "N": 128, "P": 128,
         "decay": "token", "dtype": "bf16"},
        # one decode step of a single sequence on the 130M-like layer: latency
        {"name": "la_step_one", "op": "la_step", "B": 1, "H": 24, "G": 1, "N": 128, "P": 64,
         "decay": "head", "dtype": "bf16"},
        # 64K tokens sorted by their two of 16 experts and copied out
        {"name": "tokens_out_long", "op": "tokens_out", "T": 65536, "D": 2560, "E": 16, "k": 2, "dtype": "bf16", "drop": 0.0},
        # the rows of a decode batch brought back, some slots dropped
        {"name": "tokens_back_decode", "op": "tokens_back", "T": 256, "D": 5120, "E": 8, "k": 2, "dtype": "bf16", "drop": 0.1},
        # a training step's way back on the 1.4B-like layer: outputs combined, then the gradients of rows, gates and tokens
        {"name": "tokens_train_1p4b", "op": "tokens_train", "T": 32768, "D": 4096, "E": 8, "k": 2, "dtype": "bf16", "drop": 0.0},
        # the router's gradients over the 64K-token prompt
        {"name": "route_grad_long", "op": "route_grad", "T": 65536, "D": 2560, "E": 16, "k": 2, "dtype": "bf16"},
        # the router's gradients with 64 experts, four active, odd sizes, fp32
        {"name": "route_grad_wide", "op": "route_grad", "T": 5001, "D": 1538, "E": 64, "k": 4, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["la", "la", "la_train", "la_step", "tokens_out", "tokens_back", "tokens_train", "route_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("la", "la_train", "la_step"):
        heads = _log_int(rng, 1, 48)
        group = rng.choice([g for g in range(1, heads + 1) if heads % g == 0])
        wide = [16, 32, 64, 128, rng.randint(9, 127), 2 * rng.randint(5, 63)]
        case = {"op": op, "B": _log_int(rng, 1, 8), "H": heads, "G": group, "N": rng.choice(wide), "P": rng.choice(wide),
                "decay": rng.choice(["head", "token"]), "dtype": dtype}
        if op == "la_step":
            case["B"] = _log_int(rng, 1, 256)
            return case
        most = (1 << 20) if op == "la" else (1 << 17)
        case["L"] = max(1, min(_log_int(rng, 1, 65536), most // (case["B"] * heads)))
        case["h0"] = rng.random() < 0.5
        case["reset"] = rng.choice([0, 0, 100, 700]) if case["decay"] == "token" else 0
        return case
    experts = _log_int(rng, 2, 64)
    case = {"op": op, "T": _log_int(rng, 1, 32768), "D": _log_int(rng, 64, 4096), "E": experts,
            "k": min(experts, rng.choice([1, 2, 2, 3, 4])), "dtype": dtype}
    if op != "route_grad":
        case["drop"] = rng.choice([0.0, 0.0, 0.2])
    return case


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV).to(dtype)

    st = {"case": case, "op": case["op"]}
    if case["op"] in ("la", "la_train", "la_step"):
        B, H, G, N, P = (case[n] for n in "BHGNP")
        lead = (B, case["L"]) if "L" in case else (B,)
        root = N ** -0.25  # q.k of order one
        st["q"] = (normal(*lead, G, N) * root).to(dt)
        st["k"] = (normal(*lead, G, N) * root).to(dt)
        st["v"] = normal(*lead, H, P, dtype=dt)
        if case["decay"] == "head":  # from 1 - 1/8 to 1 - 1/1024 over the heads
            st["g"] = torch.log1p(-torch.exp2(-torch.linspace(3, 10, H, device=DEV)))
        else:  # a softplus step times a rate per head, as the scans' exp(Delta A)
            rate = torch.exp(torch.rand(H, generator=gen, device=DEV) * math.log(16.0)) / 16
            st["g"] = -torch.nn.functional.softplus(normal(*lead, H) - 2) * rate
            if case.get("reset"):  # a document begins: the state is cleared
                starts = torch.rand(lead, generator=gen, device=DEV) < 1.0 / case["reset"]
                st["g"] = st["g"].masked_fill(starts.unsqueeze(-1), -math.inf)
        st["g"] = st["g"].float().contiguous()
        state = case["op"] == "la_step" or case["h0"]
        st["h0"] = normal(B, H, N, P) if state else None
        if case["op"] == "la_train":
            st["dy"] = normal(*lead, H, P, dtype=dt)
            st["dh"] = normal(B, H, N, P) if state else None
        return st
    T, D, E, k = (case[n] for n in ("T", "D", "E", "k"))
    logits = normal(T, E)
    top, idx = torch.topk(logits, k, dim=1)
    st["gate"] = torch.softmax(top, dim=1)
    st["idx"] = idx.to(torch.int32)
    if case["op"] == "route_grad":
        st["x"] = normal(T, D, dtype=dt)
        st["Wr"] = normal(D, E) * D ** -0.5
        st["dgate"] = normal(T, k)
        return st
    if case["drop"]:  # over an expert's capacity: the slot takes no row
        st["idx"] = st["idx"].masked_fill(torch.rand((T, k), generator=gen, device=DEV) < case["drop"], -1)
    if case["op"] == "tokens_out":
        st["x"] = normal(T, D, dtype=dt)
        st["rows"] = torch.zeros((T * k, D), dtype=dt, device=DEV)  # rows behind the last one stay zero
        return st
    st["pos"] = _sort(st["idx"], E)[1]
    st["ys"] = normal(T * k, D, dtype=dt)
    if case["op"] == "tokens_train":
        st["dy"] = normal(T, D, dtype=dt)
        st["dxs"] = normal(T * k, D, dtype=dt)
        st["rows"] = torch.zeros((T * k, D), dtype=dt, device=DEV)
    return st


# ---- plain forms -----------------------------------------------------------

CHUNK = 128


def _sort(idx, E):
    """Slots in order of their expert, equal ones in order of the slot: (order, pos, offsets)."""
    T, k = idx.shape
    e = idx.reshape(-1).long()
    valid = (e >= 0) & (e < E)
    key = torch.where(valid, e, torch.full_like(e, E))
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=idx.device)
    count = (key[:, None] == torch.arange(E, device=idx.device)).sum(0)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    pos = torch.where(valid, place, torch.full_like(place, -1)).reshape(T, k)
    order = torch.where(valid[order], order, torch.full_like(order, -1))
    return order.int(), pos.int(), offsets.int()


def _split(t, C, heads):
    """[B, L, h, n] as fp32 [B, heads, chunks, C, n], zero-padded, shared heads repeated."""
    B, L, h, n = t.shape
    t = torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, -L % C))
    t = t.reshape(B, -1, C, h, n).permute(0, 3, 1, 2, 4)
    return t.repeat_interleave(heads // h, dim=1) if heads != h else t


def _join(t, L):
    """[B, h, chunks, C, n] back to [B, L, h, n]."""
    B, h, c, C, n = t.shape
    return t.permute(0, 2, 3, 1, 4).reshape(B, c * C, h, n)[:, :L]


def _la_forward(st):
    q, k, v = st["q"], st["k"], st["v"]
    B, L, H, P = v.shape
    N = q.shape[-1]
    C = min(CHUNK, L)
    Q, K, V = (_split(t, C, H) for t in (q, k, v))
    # sums of log decays in 64 bits; e^-1000 is zero, and differences stay finite
    g = st["g"].double().clamp(min=-1000.0).expand(B, L, H)
    G = _split64(g, C).cumsum(-1)  # [B, H, c, C]
    c = G.shape[2]
    D = G.unsqueeze(-1) - G.unsqueeze(-2)
    later = torch.ones(C, C, dtype=torch.bool, device=q.device).triu(1)
    D = D.masked_fill_(later, -math.inf).exp_().float()
    w = (G[..., -1:] - G).exp().float().unsqueeze(-1)
    eG = G.exp().float().unsqueeze(-1)
    U = torch.matmul((K * w).transpose(-1, -2), V)  # [B, H, c, N, P]
    T = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))  # decay before each chunk, and in all
    W = T[..., :, None] - T[..., None, 1:]
    W = W.masked_fill_(torch.ones(c + 1, c, dtype=torch.bool, device=q.device).triu(0), -math.inf).exp_().float()
    S = torch.matmul(W, U.reshape(B, H, c, N * P)).reshape(B, H, c + 1, N, P)
    if st["h0"] is not None:
        S = S + T.exp().float()[..., None, None] * st["h0"].unsqueeze(2)
    M = torch.matmul(Q, K.transpose(-1, -2)) * D
    y = torch.matmul(M, V) + torch.matmul(Q * eG, S[:, :, :c])
    return {"y": _join(y, L).to(v.dtype).contiguous(), "h_final": S[:, :, c].contiguous(),
            "parts": (Q, K, V, G, D, w, eG, T, S, M)}


def _split64(g, C):
    B, L, H = g.shape
    g = torch.nn.functional.pad(g, (0, 0, 0, -L % C))
    return g.reshape(B, -1, C, H).permute(0, 3, 1, 2)


def _la_backward(st, parts):
    Q, K, V, G, D, w, eG, T, S, M = parts
    B, L, H, P = st["v"].shape
    g_heads, N = st["q"].shape[2:]
    c, C = G.shape[2:]
    dY = _split(st["dy"], C, H)
    R = torch.matmul((Q * eG).transpose(-1, -2), dY)
    W = T[..., None, :c] - T[..., :, None]  # chunk j's readers seen from before chunk i
    W = W.masked_fill_(torch.ones(c + 1, c, dtype=torch.bool, device=W.device).tril(-1), -math.inf).exp_().float()
    A = torch.matmul(W, R.reshape(B, H, c, N * P)).reshape(B, H, c + 1, N, P)
    if st["dh"] is not None:
        A = A + (T[..., c:] - T).exp().float()[..., None, None] * st["dh"].unsqueeze(2)
    adj = A[:, :, 1:]  # the adjoint of each chunk's end state
    h_in = S[:, :, :c]
    DA = torch.matmul(dY, V.transpose(-1, -2)) * D
    dQ = torch.matmul(DA, K) + torch.matmul(dY * eG, h_in.transpose(-1, -2))
    dK = torch.matmul(DA.transpose(-1, -2), Q) + torch.matmul(V * w, adj.transpose(-1, -2))
    dV = torch.matmul(M.transpose(-1, -2), dY) + torch.matmul(K * w, adj)
    MA = (M * torch.matmul(dY, V.transpose(-1, -2))).double()
    reads = (torch.matmul(Q * eG, h_in) * dY).double().sum(-1)
    writes = (torch.matmul(K * w, adj) * V).double().sum(-1)
    through = G[..., -1].exp() * (h_in.double() * adj.double()).sum((-1, -2))
    after = (MA.sum(-1) - MA.sum(-2) + reads).flip(-1).cumsum(-1).flip(-1)
    before = writes.cumsum(-1) - writes
    dg = (after + before + through.unsqueeze(-1)).permute(0, 2, 3, 1).reshape(B, c * C, H)[:, :L]
    dg = dg.masked_fill(st["g"].expand(B, L, H) == -math.inf, 0.0)  # e^g is zero there, and so is its slope
    if st["g"].dim() == 1:
        dg = dg.sum((0, 1))
    dt = st["v"].dtype

    def shared(t):
        return _join(t, L).reshape(B, L, g_heads, H // g_heads, N).sum(3).to(dt)

    return {"dq": shared(dQ), "dk": shared(dK), "dv": _join(dV, L).to(dt).contiguous(), "dlog_decay": dg.float(),
            "dh0": A[:, :, 0].contiguous()}


def _la_step(st):
    B, H, P = st["v"].shape
    share = H // st["q"].shape[1]
    q = st["q"].float().repeat_interleave(share, dim=1)
    k = st["k"].float().repeat_interleave(share, dim=1)
    decay = st["g"].exp().expand(B, H)[..., None, None]
    h = st["h0"] * decay + k.unsqueeze(-1) * st["v"].float().unsqueeze(-2)
    y = (h * q.unsqueeze(-1)).sum(-2)
    return {"y": y.to(st["v"].dtype), "state": h}


def _take(rows, pos):
    """rows[pos] in fp32 [T, k, D], zero where a slot has no row."""
    got = rows[pos.clamp(min=0).long()].float()
    return got * (pos >= 0).unsqueeze(-1)


def _put(rows, pos, values):
    """`rows` with values [T, k, D] at pos, other rows as they were."""
    keep = (pos >= 0).reshape(-1)
    out = rows.clone()
    out[pos.reshape(-1)[keep].long()] = values.reshape(-1, values.shape[-1])[keep].to(rows.dtype)
    return out


def _route_grad(st):
    g, dg, idx = st["gate"], st["dgate"], st["idx"].long()
    slope = g * (dg - (g * dg).sum(1, keepdim=True))
    dl = torch.zeros(g.shape[0], st["Wr"].shape[1], device=g.device).scatter_add_(1, idx, slope)
    dx = torch.matmul(dl, st["Wr"].t())
    return {"dx": dx.to(st["x"].dtype), "dWr": torch.matmul(st["x"].float().t(), dl)}


def run(st):
    op = st["op"]
    if own:
        return _run_own(st, op)
    if op in ("la", "la_train"):
        f = _la_forward(st)
        out = {"y": f["y"], "h_final": f["h_final"]}
        return {**out, **_la_backward(st, f["parts"])} if op == "la_train" else out
    if op == "la_step":
        return _la_step(st)
    if op == "route_grad":
        return _route_grad(st)
    if op == "tokens_out":
        T, k = st["idx"].shape
        order, pos, offsets = _sort(st["idx"], st["case"]["E"])
        rows = _put(st["rows"], pos, st["x"].unsqueeze(1).expand(-1, k, -1))
        return {"order": order, "pos": pos, "offsets": offsets, "rows": rows}
    pos, gate = st["pos"], st["gate"].unsqueeze(-1)
    dt = st["ys"].dtype
    ys = _take(st["ys"], pos)
    out = {"y": (ys * gate).sum(1).to(dt)}
    if op == "tokens_train":
        dy = st["dy"].float().unsqueeze(1)
        out["dys"] = _put(st["rows"], pos, dy * gate)
        out["dgate"] = (dy * ys).sum(-1)
        out["dx"] = _take(st["dxs"], pos).sum(1).to(dt)
    return out


def _run_own(st, op):
    from parameter_space_moe_amd import swimba
    if op in ("la", "la_train"):
        y, h = swimba.linear_attention(st["q"], st["k"], st["v"], st["g"], h0=st["h0"])
        out = {"y": y, "h_final": h}
        if op == "la_train":
            out.update(swimba.linear_attention_backward(st["q"], st["k"], st["v"], st["g"], st["dy"], h0=st["h0"],
                                                        dh_final=st["dh"], grad_dtype=st["v"].dtype))
        return out
    if op == "la_step":
        # a decode loop marshals its call once for its buffers (which the call holds); others get a call of their own
        ops = (st["q"], st["k"], st["v"], st["g"], st["h0"])
        made = st.get("made")
        if made is None or made[0] != list(map(id, ops)):
            out = torch.empty_like(st["h0"])
            made = st["made"] = (list(map(id, ops)), out, swimba.PreparedLinearAttentionStep(*ops, state_out=out))
        return {"y": made[2](), "state": made[1]}
    if op == "route_grad":
        dx, dWr = swimba.route_backward(st["x"], st["Wr"], st["idx"], st["gate"], st["dgate"], grad_dtype=st["x"].dtype)
        return {"dx": dx, "dWr": dWr}
    if op == "tokens_out":
        order, pos, offsets = swimba.sort_tokens(st["idx"], st["case"]["E"])
        rows = swimba.dispatch_tokens(st["x"], pos, rows=st["rows"])
        return {"order": order, "pos": pos, "offsets": offsets, "rows": rows}
    out = {"y": swimba.combine_tokens(st["ys"], st["pos"], st["gate"])}
    if op == "tokens_train":
        out["dys"], out["dgate"] = swimba.combine_tokens_backward(st["ys"], st["pos"], st["gate"], st["dy"], drows=st["rows"])
        out["dx"] = swimba.dispatch_tokens_backward(st["dxs"], st["pos"])
    return out


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("la", "la_train", "la_step"):
        B, H, G, N, P = (case[n] for n in "BHGNP")
        L = case.get("L", 1)
        t = B * L
        keys, values = t * G * N * size, t * H * P * size
        g = 4 * (H if case["decay"] == "head" else t * H)
        state = 4 * B * H * N * P
        if op == "la_step":
            return {"bytes": 2 * keys + 2 * values + g + 2 * state, "flops": 5 * B * H * N * P}
        first = 2 if case["h0"] else 1
        forward = {"bytes": 2 * keys + 2 * values + g + first * state, "flops": 4 * t * H * N * P}
        if op == "la":
            return forward
        # y, h_final and the gradients of q, k, v, the decays and the first state, from the inputs, dy and the last state's gradient
        return {"bytes": 4 * keys + 4 * values + 2 * g + (2 * first) * state, "flops": 14 * t * H * N * P}
    T, D, E, k = (case[n] for n in ("T", "D", "E", "k"))
    used = T * k * (1 - case.get("drop", 0.0))
    if op == "route_grad":
        return {"bytes": 2 * T * D * size + 8 * D * E + 12 * T * k, "flops": 4 * T * k * D}
    if op == "tokens_out":
        return {"bytes": int((T + used) * D * size + 12 * T * k + 4 * (E + 1)), "flops": 0}
    if op == "tokens_back":
        return {"bytes": int((T + used) * D * size + 8 * T * k), "flops": int(2 * used * D)}
    return {"bytes": int((3 * T + 3 * used) * D * size + 12 * T * k), "flops": int(6 * used * D)}


# ---- 64 bits, from the definitions ----------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("la", "la_train", "la_step"):
        return _exact_la(st, op)
    if op == "route_grad":
        gate, dgate = st["gate"].double(), st["dgate"].double()
        mean = (gate * dgate).sum(1)
        dx = torch.zeros(case["T"], case["D"], dtype=torch.float64, device=DEV)
        dW = torch.zeros(case["E"], case["D"], dtype=torch.float64, device=DEV)
        W, x = st["Wr"].double().t(), st["x"].double()
        for j in range(case["k"]):
            e = st["idx"][:, j].long()
            slope = (gate[:, j] * (dgate[:, j] - mean)).unsqueeze(1)
            dx += slope * W[e]
            for i in range(case["E"]):
                mine = e == i
                dW[i] += (slope[mine] * x[mine]).sum(0)
        return {"dx": dx, "dWr": dW.t()}
    T, D, k = case["T"], case["D"], case["k"]
    if op == "tokens_out":
        rows = torch.zeros(T * k, D, dtype=torch.float64, device=DEV)
        slots = st["idx"].reshape(-1)
        x, first = st["x"].double(), 0
        for e in range(case["E"]):
            mine = torch.nonzero(slots == e).squeeze(1)  # ascending
            rows[first:first + len(mine)] = x[mine // k]
            first += len(mine)
        return {"order": None, "pos": None, "offsets": None, "rows": rows}
    y = torch.zeros(T, D, dtype=torch.float64, device=DEV)
    out = {"y": y}
    if op == "tokens_train":
        out.update(dys=torch.zeros(T * k, D, dtype=torch.float64, device=DEV),
                   dgate=torch.zeros(T, k, dtype=torch.float64, device=DEV), dx=torch.zeros_like(y))
    for j in range(k):
        at = torch.nonzero(st["pos"][:, j] >= 0).squeeze(1)
        row = st["pos"][at, j].long()
        gate = st["gate"][at, j].double().unsqueeze(1)
        ys = st["ys"][row].double()
        y[at] += gate * ys
        if op == "tokens_train":
            dy = st["dy"][at].double()
            out["dys"][row] = gate * dy
            out["dgate"][at, j] = (dy * ys).sum(1)
            out["dx"][at] += st["dxs"][row].double()
    return out


def _exact_la(st, op):
    """The recurrence token by token, and its adjoint from the last token back."""
    one = op == "la_step"
    q, k, v = (st[n].double().unsqueeze(1) if one else st[n].double() for n in "qkv")
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    share = H // G
    g = st["g"].double()
    decay = (g.unsqueeze(1) if one and g.dim() == 2 else g).exp().expand(B, L, H)
    # token-major copies; two of q and k, as a column for the state
    q, k = (t.repeat_interleave(share, dim=2).transpose(0, 1).unsqueeze(-1).contiguous() for t in (q, k))
    v = v.transpose(0, 1).unsqueeze(-2).contiguous()
    e = decay.transpose(0, 1)[..., None, None].contiguous()
    h = torch.zeros(B, H, N, P, dtype=torch.float64, device=DEV)
    if st["h0"] is not None:
        h += st["h0"].double()
    y = torch.empty(L, B, H, P, dtype=torch.float64, device=DEV)
    train = op == "la_train"
    if train:
        dy = st["dy"].double().transpose(0, 1).unsqueeze(-2).contiguous()
        dq = torch.empty(L, B, H, N, dtype=torch.float64, device=DEV)
    for t in range(L):
        h.mul_(e[t]).addcmul_(k[t], v[t])
        torch.sum(h * q[t], -2, out=y[t])
        if train:
            torch.sum(h * dy[t], -1, out=dq[t])
    out = {"y": y.transpose(0, 1) if not one else y[0], "state" if one else "h_final": h}
    if not train:
        return out
    a = torch.zeros_like(h) if st["dh"] is None else st["dh"].double()
    ends = (a * h).sum((-1, -2))  # [B, H]
    dk, dv = torch.empty_like(dq), torch.empty_like(y)
    for t in range(L - 1, -1, -1):
        a = a.addcmul(q[t], dy[t])
        torch.sum(a * v[t], -1, out=dk[t])
        torch.sum(a * k[t], -2, out=dv[t])
        a.mul_(e[t])
    # a log decay scales what later tokens read of earlier ones
    dg = ((q.squeeze(-1) * dq).sum(-1) - (k.squeeze(-1) * dk).sum(-1)).flip(0).cumsum(0).flip(0) + ends
    dg = dg.transpose(0, 1).masked_fill(decay == 0, 0.0)

    def shared(t):
        return t.transpose(0, 1).reshape(B, L, G, share, N).sum(3)

    out.update(dq=shared(dq), dk=shared(dk), dv=dv.transpose(0, 1), dlog_decay=dg.sum((0, 1)) if g.dim() == 1 else dg, dh0=a)
    return out

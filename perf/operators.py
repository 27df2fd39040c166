"""The training operators of the MoE layer as measured cases: the balance loss with its gradient,
the router's dense gradients, 8-bit activation checkpoints (codes of 32 columns with a shared
power-of-two scale), the gate/up product that keeps them, and the SwiGLU backward that reads them.

Every operator has a plain form in elementary torch operations (32 bits, rounded once at the
end) and, where ``own`` is true, the framework's calls.
"""
import math

import torch

own = False

BLOCK = 32          # columns that share a scale
MIN_EXP = -117      # the smallest scale is 2^-117: every code's value is a normal bf16 number


def listed():
    return [
        # a handful of tokens with an odd expert count (the last batch of an epoch): launch latency
        dict(name="balance_small", op="balance", N=7, E=60, k=4, S=1, mask=False, bias=False, gates=False, dz="f32"),
        # one training batch of the DeepSeek-V3-shaped layer: loss, counts and the logits' whole gradient
        dict(name="balance_batch", op="balance", N=8192, E=256, k=8, S=1, mask=False, bias=False, gates=True,
             dz="bf16"),
        # ragged sequences packed into one batch with padding behind the last: per-sequence loss, biased logits
        dict(name="balance_packed", op="balance", N=32768, E=160, k=6, S=61, mask=True, bias=True, gates=False,
             dz="f32"),
        # fp32 layer, odd sizes
        dict(name="router_grad_f32", op="router", N=1000, E=60, H=520, dt="f32", dw="f32", rest=True),
        # few experts, wide rows (the Mixtral-shaped layer)
        dict(name="router_grad_few", op="router", N=4096, E=8, H=4096, dt="bf16", dw="f32", rest=False),
        # many experts (the DeepSeek-V3-shaped layer), the shared expert's input gradient added
        dict(name="router_grad_many", op="router", N=8192, E=256, H=7168, dt="bf16", dw="bf16", rest=True),
        # fp32 activations kept and read back in place
        dict(name="keep_f32", op="keep", N=301, H=1056, k=0, dt="f32"),
        # a batch's tokens kept in 8 bits, read back as expert-ordered rows
        dict(name="keep_tokens", op="keep", N=8191, H=7168, k=8, dt="bf16"),
        # a small layer with a shared expert
        dict(name="gate_up_small", op="gate_up", N=509, H=1024, E=16, k=4, I=512, shared=True),
        # the Mixtral-shaped layer
        dict(name="gate_up_wide", op="gate_up", N=4096, H=4096, E=8, k=2, I=14336, shared=False),
        # ungated rows (a shared expert), wide, odd count
        dict(name="swiglu_shared", op="swiglu", N=1021, k=0, I=14336, drop=False, dt="bf16"),
        # the routed rows of the DeepSeek-V3-shaped layer, some slots dropped
        dict(name="swiglu_routed", op="swiglu", N=8192, k=8, I=2048, drop=True, dt="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "router", "keep", "gate_up", "swiglu"])
    if op == "balance":
        E = _log(rng, 4, 1024)
        N = _log(rng, 1, min(32768, (32768 * 160) // E))
        return dict(op=op, N=N, E=E, k=rng.randint(1, min(E, 8)), S=_log(rng, 1, 64), mask=rng.random() < 0.5,
                    bias=rng.random() < 0.5, gates=rng.random() < 0.4, dz=rng.choice(["f32", "bf16"]))
    if op == "router":
        dt = rng.choice(["f32", "bf16", "bf16"])
        E = _log(rng, 4, 512 if dt == "bf16" else 128)
        H = 8 * _log(rng, 16, 1024)
        N = _log(rng, 1, 8192 if dt == "bf16" else 2048)
        N = max(1, min(N, 8192 * 256 * 7168 // (E * H)))
        return dict(op=op, N=N, E=E, H=H, dt=dt, dw=rng.choice(["f32", "bf16"]), rest=rng.random() < 0.5)
    if op == "keep":
        k = rng.choice([0, 0, 1, 2, 8])
        H = BLOCK * _log(rng, 2, 256)
        N = max(1, min(_log(rng, 1, 32768), 8191 * 8 * 7168 // (H * max(k, 1))))
        return dict(op=op, N=N, H=H, k=k, dt=rng.choice(["f32", "bf16"]))
    if op == "gate_up":
        E = _log(rng, 1, 32)
        k = rng.randint(1, min(E, 4))
        H, I = 128 * _log(rng, 2, 32), 128 * _log(rng, 2, 32)
        N = max(1, min(_log(rng, 1, 4096), 4096 * 2 * 4096 * 14336 // (k * H * I)))
        return dict(op=op, N=N, H=H, E=E, k=k, I=I, shared=rng.random() < 0.5)
    k = rng.choice([0, 1, 4, 8])
    I = BLOCK * _log(rng, 2, 448)
    N = max(1, min(_log(rng, 1, 8192), 65536 * 2048 // (I * max(k, 1))))
    return dict(op=op, N=N, k=k, I=I, drop=rng.random() < 0.5, dt=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------------------- inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _seq_starts(N, S, g):
    """S ragged sequences (some may be empty) over the first 15/16 of the tokens; one
    sequence takes all of them."""
    if S == 1:
        return torch.tensor([0, N], dtype=torch.int32)
    cut = torch.randint(0, N - N // 16 + 1, (S - 1,), generator=g).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([N - N // 16])]).to(torch.int32)


def _send_pos(idx, drop, g):
    """Row of every slot when the slots are ordered by expert; dropped slots get -1."""
    flat = idx.reshape(-1).clone()
    if drop:
        flat[torch.rand(flat.shape, generator=g) < 0.01] = 1 << 20
    kept = flat < (1 << 20)
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel())
    return torch.where(kept, pos, torch.full_like(pos, -1)).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)             # small host-made arrays
    gd = torch.Generator(device=dev).manual_seed(seed)  # large ones
    rn = lambda *s: torch.randn(*s, generator=gd, device=dev)  # noqa: E731
    s = {"case": case}
    N = case["N"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        # logits of a router in training: unit spread, some experts favoured
        s["z"] = rn(N, E) + 0.5 * rn(E)
        s["bias"] = 0.1 * rn(E) if case["bias"] else None
        b = s["z"] if s["bias"] is None else s["z"] + s["bias"]
        top = torch.topk(b, k, dim=1)
        s["idx"] = top.indices.to(torch.int32).contiguous()
        s["alpha"] = 0.01
        s["seq"] = None if S == 1 else _seq_starts(N, S, g).to(dev)
        s["mask"] = (torch.rand(N, generator=g) < 0.9).to(torch.uint8).to(dev) if case["mask"] else None
        s["gate"] = torch.softmax(top.values, dim=1).contiguous() if case["gates"] else None
        s["dg"] = rn(N, k) / N if case["gates"] else None
        s["d_loss"] = torch.full((1,), 0.7, device=dev)
    elif case["op"] == "router":
        dt = _DT[case["dt"]]
        s["dz"] = (rn(N, case["E"]) / 1024).to(dt)
        s["x"] = rn(N, case["H"]).to(dt)
        s["w"] = (0.02 * rn(case["E"], case["H"])).to(dt)
        s["rest"] = (0.01 * rn(N, case["H"])).to(dt) if case["rest"] else None
    elif case["op"] == "keep":
        # rows of differing scale with a few large columns, as hidden states have
        x = rn(N, case["H"]) * torch.exp(rn(N, 1))
        x[:, ::97] *= 20
        s["x"] = x.to(_DT[case["dt"]])
        k = case["k"]
        s["pos"] = _send_pos(torch.randint(0, 32, (N, k), generator=g), False, g).to(dev) if k else None
    elif case["op"] == "gate_up":
        E, k, H, I = case["E"], case["k"], case["H"], case["I"]
        s["x"] = rn(N, H).to(torch.bfloat16)
        std = 1.0 / math.sqrt(H)
        s["w"] = torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device=dev)
        for e in range(E):
            s["w"][e] = (std * rn(2 * I, H)).to(torch.bfloat16)
        s["sw"] = (std * rn(1, 2 * I, H)).to(torch.bfloat16) if case["shared"] else None
        idx = torch.rand(N, E, generator=g).topk(k, dim=1).indices
        pos = _send_pos(idx, False, g)
        slot = torch.empty(N * k, dtype=torch.int32)
        slot[pos.long()] = torch.arange(N * k, dtype=torch.int32)
        n_e = torch.bincount(idx.reshape(-1), minlength=E)
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[1:] = n_e.cumsum(0)
        s["off"], s["slot"], s["cap"] = off.to(dev), slot.to(dev), int(n_e.max())
    else:
        I, k = case["I"], case["k"]
        rows = N * max(k, 1)
        dt = _DT[case["dt"]]
        s["q"], s["e"] = _codes(rn(rows, 2 * I).to(dt).float())
        s["dh"] = (rn(rows, I) / 64).to(dt)
        s["pos"] = s["gate"] = None
        if k:
            s["pos"] = _send_pos(torch.rand(N, 32, generator=g).topk(k, dim=1).indices, case["drop"], g).to(dev)
            s["gate"] = torch.softmax(rn(N, k), dim=1).contiguous()
        # the step's buffers: rows that no slot names stay as they are
        s["d_au"] = torch.zeros(rows, 2 * I, dtype=dt, device=dev)
        s["h"] = torch.zeros(rows, I, dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------------------- plain forms

def _codes(x):
    """e4m3 codes and biased scale exponents of the 32-column blocks of fp32 x."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(dim=2))        # amax = m 2^e, m in [1/2, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=MIN_EXP)
    q = torch.ldexp(b, -e.unsqueeze(2)).to(torch.float8_e4m3fn)
    return q.reshape(x.shape).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(q, e):
    """fp32 values of codes and scales."""
    v = q.view(torch.float8_e4m3fn).float().reshape(q.shape[0], -1, BLOCK)
    return (v * torch.exp2(e.float() - 127).unsqueeze(2)).reshape(q.shape)


def _membership(s):
    """[S, N]: 1 where token t counts in sequence s."""
    N, dev = s["case"]["N"], s["z"].device
    t = torch.arange(N, device=dev)
    seq = torch.tensor([0, N], device=dev) if s["seq"] is None else s["seq"]
    m = (t >= seq[:-1, None]) & (t < seq[1:, None])
    return (m if s["mask"] is None else m & (s["mask"] != 0)).float()


def _plain_balance(s):
    c = s["case"]
    N, E, k, S = c["N"], c["E"], c["k"], c["S"]
    b = s["z"] if s["bias"] is None else s["z"] + s["bias"]
    ex = torch.exp(b - b.amax(dim=1, keepdim=True))
    p = ex / ex.sum(dim=1, keepdim=True)
    member = _membership(s)
    hot = torch.zeros(N, E, device=b.device).scatter_add_(1, s["idx"].long(), torch.ones_like(s["idx"]).float())
    counts = member @ hot
    T = member.sum(dim=1, keepdim=True)
    T1 = T.clamp(min=1)
    P = (member @ p) / T1
    f = counts * E / (k * T1)
    loss = (s["alpha"] / S) * (f * P).sum().reshape(1)
    # an even load k / E a token moves nothing (the probabilities sum to 1): only what a count
    # is away from it enters
    coef = (member.t() @ ((counts - k * T / E) / (T1 * T1))) * (s["d_loss"] * s["alpha"] * E / (S * k))
    dz = p * (coef - (p * coef).sum(dim=1, keepdim=True))
    if s["gate"] is not None:
        sel = s["gate"] * (s["dg"] - (s["gate"] * s["dg"]).sum(dim=1, keepdim=True))
        dz = dz.scatter_add(1, s["idx"].long(), sel)
    return {"loss": loss, "counts": counts.to(torch.int32), "prob": P, "dz": dz.to(_DT[c["dz"]])}


def _plain_router(s):
    dt, dz = s["x"].dtype, s["dz"].float()
    dw = dz.t() @ s["x"].float()
    dx = dz @ s["w"].float()
    if s["rest"] is not None:
        dx = dx + s["rest"].float()
    return {"dw": dw.to(_DT[s["case"]["dw"]]), "dx": dx.to(dt)}


def _plain_keep(s):
    v = _values(*_codes(s["x"].float())).to(s["x"].dtype)
    if s["pos"] is None:
        return {"x": v}
    k = s["case"]["k"]
    out = torch.empty(v.shape[0] * k, v.shape[1], dtype=v.dtype, device=v.device)
    out[s["pos"].long()] = v.repeat_interleave(k, dim=0)
    return {"x": out}


def _plain_gate_up(s):
    c = s["case"]
    rows, E, I = c["N"] * c["k"], c["E"], c["I"]
    # every expert's rows padded to the fullest one's count, one batched product
    at = s["off"][:-1, None].long() + torch.arange(s["cap"], device=s["x"].device)
    inside = at < s["off"][1:, None]
    token = (s["slot"].long() // c["k"])[at.clamp(max=rows - 1)]
    au = torch.bmm(s["x"].float()[token], s["w"].float().transpose(1, 2).contiguous())[inside]
    if s["sw"] is not None:
        au = torch.cat([au, s["x"].float() @ s["sw"][0].float().t()])
    h = au[:, :I] / (1 + torch.exp(-au[:, :I])) * au[:, I:]
    kept = _values(*_codes(au.to(torch.bfloat16).float()))
    return {"h": h.to(torch.bfloat16), "au": kept.to(torch.bfloat16)}


def _plain_swiglu(s):
    c = s["case"]
    I = c["I"]
    au = _values(s["q"], s["e"])
    a, u, dh = au[:, :I], au[:, I:], s["dh"].float()
    sg = 1 / (1 + torch.exp(-a))
    h = a * sg * u
    da, du = dh * u * sg * (1 + a * (1 - sg)), dh * a * sg
    dt = s["dh"].dtype
    if s["pos"] is None:
        return {"d_au": torch.cat([da, du], dim=1).to(dt), "h": h.to(dt)}
    pos = s["pos"].long()
    ok = pos >= 0
    spare = torch.where(ok, pos, torch.full_like(pos, au.shape[0]))   # (one row more for the dropped slots)
    g = torch.zeros(au.shape[0] + 1, device=a.device).scatter_(0, spare, s["gate"].reshape(-1))[:-1, None]
    dot = (dh * h).sum(dim=1)
    dg = torch.where(ok, dot[pos.clamp(min=0)], torch.zeros((), device=a.device)).reshape(s["gate"].shape)
    return {"d_au": torch.cat([g * da, g * du], dim=1).to(dt), "h": (g * h).to(dt), "d_gate": dg}


# ------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"balance": _plain_balance, "router": _plain_router, "keep": _plain_keep, "gate_up": _plain_gate_up,
                "swiglu": _plain_swiglu}[op](state)
    import combine_grouped_gemm_amd as moe
    c, s = state["case"], state
    if op == "balance":
        loss, counts, prob, tokens = moe.moe_balance_loss(s["z"], s["idx"], s["alpha"], bias=s["bias"],
                                                          seq_start=s["seq"], token_mask=s["mask"])
        dz = moe.moe_balance_loss_backward(s["z"], s["idx"], s["alpha"], counts, tokens, bias=s["bias"],
                                           seq_start=s["seq"], token_mask=s["mask"], d_loss=s["d_loss"],
                                           topk_gate=s["gate"], d_gate=s["dg"], dz_dtype=_DT[c["dz"]])
        return {"loss": loss, "counts": counts, "prob": prob, "dz": dz}
    if op == "router":
        return {"dw": moe.moe_router_dense_wgrad(s["dz"], s["x"], dw_dtype=_DT[c["dw"]]),
                "dx": moe.moe_router_dense_dgrad(s["dz"], s["w"], rest=s["rest"])}
    if op == "keep":
        q, e = moe.moe_quantize_mxfp8(s["x"])
        return {"x": moe.moe_dequantize_mxfp8(q, e, dtype=s["x"].dtype, send_pos=s["pos"], k=max(c["k"], 1))}
    if op == "gate_up":
        h, q, e = moe.moe_expert_gate_up_mxfp8(s["x"], s["slot"], c["k"], s["off"], s["w"], s["sw"])
        return {"h": h, "au": moe.moe_dequantize_mxfp8(q, e)}
    d_au, h, d_gate = moe.moe_swiglu_backward_mxfp8(s["q"], s["e"], s["dh"], send_pos=s["pos"], topk_gate=s["gate"],
                                                    d_au=s["d_au"], h=s["h"])
    return {"d_au": d_au, "h": h} if d_gate is None else {"d_au": d_au, "h": h, "d_gate": d_gate}


def work(case):
    op, N = case["op"], case["N"]
    if op == "balance":
        E, k = case["E"], case["k"]
        b = 4 * N * E + 4 * N * k * (3 if case["gates"] else 1) + 8 * case["S"] * E
        b += N * E * (4 if case["dz"] == "f32" else 2) + (N if case["mask"] else 0) + (4 * E if case["bias"] else 0)
        return {"bytes": b, "flops": 12 * N * E}
    if op == "router":
        E, H, sz = case["E"], case["H"], 4 if case["dt"] == "f32" else 2
        b = sz * (N * E + N * H + E * H + N * H * (2 if case["rest"] else 1)) + E * H * (4 if case["dw"] == "f32" else 2)
        return {"bytes": b, "flops": 4 * N * E * H}
    if op == "keep":
        H, sz = case["H"], 4 if case["dt"] == "f32" else 2
        kept = N * H * (1 + 1 / BLOCK)
        return {"bytes": N * H * sz * (1 + max(case["k"], 1)) + 2 * kept + 4 * N * case["k"], "flops": 4 * N * H}
    if op == "gate_up":
        E, k, H, I = case["E"], case["k"], case["H"], case["I"]
        rows = N * k + (N if case["shared"] else 0)
        w = (min(E, N * k) + (1 if case["shared"] else 0)) * 2 * I * H * 2
        # the kept codes are written, read and shown as bf16 values
        return {"bytes": 2 * N * H + w + rows * I * 2 + rows * 2 * I * (2 * (1 + 1 / BLOCK) + 2),
                "flops": 4 * rows * H * I}
    I, sz = case["I"], 4 if case["dt"] == "f32" else 2
    rows = N * max(case["k"], 1)
    return {"bytes": rows * I * (2 * (1 + 1 / BLOCK) + 4 * sz) + 12 * N * case["k"], "flops": 14 * rows * I}


# ------------------------------------------------------------------------------- in 64 bits

def _grid(v):
    """v (64 bits) rounded to the e4m3 code grid, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _kept64(x):
    """The kept values of 64-bit x."""
    b = x.reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    top = b.abs().max(dim=2, keepdim=True).values
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448))
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)       # (log2 next to a power of two)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(min=MIN_EXP)
    return (_grid(b * torch.exp2(-e)) * torch.exp2(e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: t.double()  # noqa: E731
    op, N = case["op"], case["N"]
    if op == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        logit = d(s["z"]) if s["bias"] is None else d(s["z"] + s["bias"])   # (the biased logit is one fp32 sum)
        p = torch.softmax(logit, dim=1)
        dev = p.device
        starts = [0, N] if s["seq"] is None else s["seq"].tolist()
        on = torch.ones(N, dtype=torch.bool, device=dev) if s["mask"] is None else s["mask"] != 0
        counts = torch.zeros(S, E, dtype=torch.int32, device=dev)
        prob = torch.zeros(S, E, dtype=torch.float64, device=dev)
        dz = torch.zeros(N, E, dtype=torch.float64, device=dev)
        loss = torch.zeros(1, dtype=torch.float64, device=dev)
        for q in range(S):
            rows = torch.nonzero(on[starts[q]:starts[q + 1]])[:, 0] + starts[q]
            T = rows.numel()
            if T == 0:
                continue
            ps = p[rows]
            c = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E)
            counts[q], prob[q] = c.to(torch.int32), ps.mean(dim=0)
            share = d(c) * E / (k * T)
            loss += s["alpha"] / S * (share * prob[q]).sum()
            grad = share * (s["alpha"] / (S * T)) * d(s["d_loss"])
            dz[rows] = ps * (grad - (ps @ grad)[:, None])
        if s["gate"] is not None:
            g, dg = d(s["gate"]), d(s["dg"])
            dz.scatter_add_(1, s["idx"].long(), g * (dg - (g * dg).sum(dim=1, keepdim=True)))
        return {"loss": loss, "counts": counts, "prob": prob, "dz": dz}
    if op == "router":
        dz = d(s["dz"])
        dx = torch.matmul(dz, d(s["w"]))
        return {"dw": torch.matmul(dz.t().contiguous(), d(s["x"])), "dx": dx if s["rest"] is None else dx + d(s["rest"])}
    if op == "keep":
        v = _kept64(d(s["x"]))
        if s["pos"] is None:
            return {"x": v}
        back = torch.empty_like(s["pos"]).long()
        back[s["pos"].long()] = torch.arange(back.numel(), device=back.device)
        return {"x": v[back // case["k"]]}
    if op == "gate_up":
        k, I = case["k"], case["I"]
        off = s["off"].tolist()
        token = s["slot"].long() // k
        parts = [d(s["x"])[token[off[e]:off[e + 1]]] @ d(s["w"][e]).t() for e in range(case["E"])]
        if case["shared"]:
            parts.append(d(s["x"]) @ d(s["sw"][0]).t())
        au = torch.cat(parts)
        return {"h": au[:, :I] * torch.sigmoid(au[:, :I]) * au[:, I:], "au": _kept64(d(au.to(torch.bfloat16)))}
    I = case["I"]
    au = d(s["q"].view(torch.float8_e4m3fn).float()).reshape(s["q"].shape[0], -1, BLOCK)
    au = (au * torch.exp2(d(s["e"]) - 127)[:, :, None]).reshape(s["q"].shape)
    a, u, dh = au[:, :I], au[:, I:], d(s["dh"])
    sg = torch.sigmoid(a)
    h, da, du = a * sg * u, dh * u * (sg + a * sg * (1 - sg)), dh * a * sg
    if s["pos"] is None:
        return {"d_au": torch.cat([da, du], dim=1), "h": h}
    named = torch.nonzero(s["pos"] >= 0)[:, 0]
    row = s["pos"][named].long()
    gate = torch.zeros(au.shape[0], 1, dtype=torch.float64, device=a.device)
    gate[row, 0] = d(s["gate"]).reshape(-1)[named]
    dg = torch.zeros(s["gate"].numel(), dtype=torch.float64, device=a.device)
    dg[named] = (dh * h).sum(dim=1)[row]
    return {"d_au": torch.cat([gate * da, gate * du], dim=1), "h": gate * h, "d_gate": dg.reshape(s["gate"].shape)}

"""The layer's operators for experts with biases and plain activations, and for a dropped-out sum
with the residual stream, as measured cases: the expert product with bias, activation and residual in its
epilogue, the activation's gradient with the biases' gradients, combine with dropout and residual, its gradient,
and dropout of rows.

Every operator has a plain form in elementary torch operations (32 bits, rounded once at the end)
and, where ``own`` is true, the framework's calls.
"""
import math

import numpy as np
import torch

own = False

ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # one token through plain experts of the Mixtral-shaped layer (serving): the weights' bytes
        dict(name="linear_token", op="linear", N=1, k=2, E=8, K=4096, I=14336, gather=True, act="gelu_tanh",
             gated=False, bias="f32", res=False, z=False, dt="bf16"),
        # a dense MLP's product back to the hidden size (4096 tokens): bias and residual stream added
        dict(name="linear_dense", op="linear", N=4096, k=0, E=1, K=14336, I=4096, gather=False, act="none",
             gated=False, bias="bf16", res=True, z=False, dt="bf16"),
        # a training batch's routed rows into gated experts with biases, pre-activations kept
        dict(name="linear_routed", op="linear", N=4096, k=4, E=32, K=2048, I=1408, gather=True, act="silu",
             gated=True, bias="f32", res=False, z=True, dt="bf16"),
        # an fp32 layer with odd sizes
        dict(name="linear_f32", op="linear", N=333, k=3, E=6, K=520, I=1016, gather=False, act="relu2",
             gated=False, bias="f32", res=True, z=False, dt="f32"),
        # a small fp32 layer's step
        dict(name="act_grad_small", op="act_grad", rows=301, E=7, I=520, act="gelu", gated=False, dt="f32", h=False),
        # routed rows of the DeepSeek-V3-shaped batch, gated experts, h for the next weight gradient
        dict(name="act_grad_routed", op="act_grad", rows=65536, E=256, I=2048, act="silu", gated=True, dt="bf16",
             h=True),
        # sixteen tokens of the Mixtral-shaped layer (fine-tuning with tiny batches): launch latency
        dict(name="combine_drop_small", op="combine", N=16, k=2, H=4096, E=8, p=0.1, shared=False, res=True,
             drop=False, dt="bf16", y="bf16"),
        # the DeepSeek-V3-shaped batch, shared expert, fp32 residual stream
        dict(name="combine_drop_batch", op="combine", N=8192, k=8, H=7168, E=256, p=0.1, shared=True, res=True,
             drop=True, dt="bf16", y="f32"),
        # an odd fp32 batch
        dict(name="combine_grad_f32", op="combine_grad", N=509, k=3, H=1032, E=12, p=0.25, shared=False, drop=False,
             dt="f32", y="f32"),
        # the DeepSeek-V3-shaped batch
        dict(name="combine_grad_batch", op="combine_grad", N=8192, k=8, H=7168, E=256, p=0.1, shared=True, drop=True,
             dt="bf16", y="bf16"),
        # a few rows
        dict(name="dropout_small", op="dropout", rows=33, H=1000, p=0.5, res=False, dt="f32", y="f32"),
        # a batch's hidden states onto the residual stream
        dict(name="dropout_batch", op="dropout", rows=8191, H=7168, p=0.1, res=True, dt="bf16", y="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "act_grad", "combine", "combine_grad", "dropout"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    E = _log(rng, 1, 64)
    k = rng.randint(1, min(E, 8))
    p = rng.choice([0.0, 0.1, 0.25, 0.5, rng.random()])
    if op == "linear":
        gated = rng.random() < 0.4
        K, I = 8 * _log(rng, 4, 1024), 8 * _log(rng, 4, 1024)
        kind = rng.choice(["dense", "routed", "rows"])
        if kind == "dense":
            E, k = 1, 0
        elif E * K * I > 8 * 4096 * 14336 // 4:
            E = max(1, 8 * 4096 * 14336 // (4 * K * I))
            k = min(k, E)
        flop = 4096 * 14336 * 4096 if dt == "bf16" else 1000 * 4096 * 4096
        N = max(1, min(_log(rng, 1, 8192), flop // (2 * max(k, 1) * K * I * (2 if gated else 1))))
        return dict(op=op, N=N, k=k, E=E, K=K, I=I, gather=kind == "routed", act=rng.choice(ACTS), gated=gated,
                    bias=rng.choice(["none", "f32", "f32" if dt == "f32" else "bf16"]), res=rng.random() < 0.4,
                    z=rng.random() < 0.4, dt=dt)
    if op == "act_grad":
        I = 8 * _log(rng, 4, 1792)
        rows = max(1, min(_log(rng, 1, 65536), 65536 * 2048 // (2 * I)))
        return dict(op=op, rows=rows, E=_log(rng, 1, 256), I=I, act=rng.choice(ACTS), gated=rng.random() < 0.5, dt=dt,
                    h=rng.random() < 0.5)
    H = 8 * _log(rng, 4, 1024)
    y = rng.choice([dt, "f32"])
    if op == "dropout":
        rows = max(1, min(_log(rng, 1, 32768), 8192 * 7168 // H))
        return dict(op=op, rows=rows, H=H, p=p, res=rng.random() < 0.5, dt=dt, y=y)
    N = max(1, min(_log(rng, 1, 32768), 8192 * 8 * 7168 // (2 * H * k)))
    c = dict(op=op, N=N, k=k, H=H, E=E, p=p, shared=rng.random() < 0.5, drop=rng.random() < 0.3, dt=dt, y=y)
    return dict(c, res=rng.random() < 0.7) if op == "combine" else c


# ------------------------------------------------------------------------------- inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _routes(N, k, E, drop, g):
    """k different experts a token: (row of every slot in expert order, rows an expert has). Some slots are
    dropped (-1) where drop is true."""
    idx = torch.rand(N, E, generator=g).topk(k, dim=1).indices.reshape(-1)
    if drop:
        idx[torch.rand(N * k, generator=g) < 0.02] = E
    order = torch.argsort(idx, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(N * k)
    return torch.where(idx < E, pos, torch.full_like(pos, -1)), torch.bincount(idx, minlength=E)[:E]


def _offsets(n_e):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n_e.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)             # small host-made arrays
    gd = torch.Generator(device=dev).manual_seed(seed)  # large ones
    rn = lambda *s: torch.randn(*s, generator=gd, device=dev)  # noqa: E731
    op, dt = case["op"], _DT[case["dt"]]
    s = {"case": case}
    if op == "linear":
        N, k, E, K, I = case["N"], case["k"], case["E"], case["K"], case["I"]
        Nw = 2 * I if case["gated"] else I
        rows = N * max(k, 1)
        s["a"] = rn(N if case["gather"] else rows, K).to(dt)
        s["w"] = torch.empty(E, Nw, K, dtype=dt, device=dev)
        for e in range(E):
            s["w"][e] = (rn(Nw, K) / math.sqrt(K)).to(dt)
        s["bias"] = None if case["bias"] == "none" else (0.5 * rn(E, Nw)).to(_DT[case["bias"]])
        s["res"] = rn(rows, I).to(dt) if case["res"] else None
        s["off"] = s["slot"] = None
        s["cap"] = rows
        if k:
            pos, n_e = _routes(N, k, E, False, g)
            s["off"], s["cap"] = _offsets(n_e).to(dev), int(n_e.max())
            if case["gather"]:
                slot = torch.empty(rows, dtype=torch.int32)
                slot[pos] = torch.arange(rows, dtype=torch.int32)
                s["slot"] = slot.to(dev)
    elif op == "act_grad":
        rows, I, E = case["rows"], case["I"], case["E"]
        Nw = 2 * I if case["gated"] else I
        s["z"] = None if case["act"] == "none" and not case["gated"] else (1.5 * rn(rows, Nw)).to(dt)
        s["dout"] = (rn(rows, I) / 64).to(dt)
        # uneven loads, some experts without rows
        load = torch.rand(E, generator=g).pow(3) * (torch.rand(E, generator=g) < 0.9)
        load[0] += 0.1
        cut = (load.cumsum(0) / load.sum() * rows).round().to(torch.int64)
        cut[-1] = rows
        s["off"] = torch.cat([torch.zeros(1, dtype=torch.int64), cut]).to(torch.int32).to(dev)
    else:
        # the generator's state: a seed and the step's offset
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g).to(dev)
        if op == "dropout":
            s["x"] = rn(case["rows"], case["H"]).to(dt)
            s["res"] = rn(case["rows"], case["H"]).to(_DT[case["y"]]) if case["res"] else None
        else:
            N, k, H = case["N"], case["k"], case["H"]
            pos, _ = _routes(N, k, case["E"], case["drop"], g)
            s["pos"] = pos.to(torch.int32).to(dev)
            s["gate"] = torch.softmax(rn(N, k), dim=1).contiguous()
            s["eo"] = rn(N * k, H).to(dt)
            if op == "combine":
                s["shared"] = rn(N, H).to(dt) if case["shared"] else None
                s["res"] = rn(N, H).to(_DT[case["y"]]) if case["res"] else None
            else:
                s["dy"] = (rn(N, H) / 64).to(_DT[case["y"]])
                # the step's buffer: rows that no slot names stay as they are
                s["d_eo"] = torch.zeros(N * k, H, dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------------------- plain forms

def _act(name, u):
    if name == "relu":
        return u.clamp(min=0)
    if name == "relu2":
        return u.clamp(min=0) * u.clamp(min=0)
    if name == "gelu":
        return 0.5 * u * torch.erfc(-u * math.sqrt(0.5))
    if name == "gelu_tanh":
        return u / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u * u * u)))
    return u / (1 + torch.exp(-u)) if name == "silu" else u


def _act_slope(name, u):
    if name == "relu":
        return (u > 0).float()
    if name == "relu2":
        return 2 * u.clamp(min=0)
    if name == "gelu":
        return 0.5 * torch.erfc(-u * math.sqrt(0.5)) + u * torch.exp(-0.5 * u * u) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        sg = 1 / (1 + torch.exp(-c * (u + 0.044715 * u * u * u)))
        return sg + u * sg * (1 - sg) * c * (1 + 3 * 0.044715 * u * u)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-u))
        return sg * (1 + u * (1 - sg))
    return torch.ones_like(u)


def _row_expert(s, rows):
    """(expert of every row, its place among the expert's rows)."""
    r = torch.arange(rows, device=s["off"].device)
    e = torch.searchsorted(s["off"][1:].contiguous(), r.to(torch.int32), right=True)
    return e, r - s["off"][e].long()


def _plain_linear(s):
    c = s["case"]
    E, k, I, dt = c["E"], c["k"], c["I"], _DT[c["dt"]]
    if not k:
        u = s["a"].float() @ s["w"][0].float().t()
        if s["bias"] is not None:
            u = u + s["bias"].float()
    else:
        # every expert's rows padded to the fullest one's count, one batched product
        rows = c["N"] * k
        e, at = _row_expert(s, rows)
        token = torch.arange(rows, device=e.device) if s["slot"] is None else s["slot"].long() // k
        place = e * s["cap"] + at
        pad = torch.zeros(E * s["cap"], c["K"], device=e.device)
        pad[place] = s["a"].float()[token]
        u = torch.bmm(pad.reshape(E, s["cap"], c["K"]), s["w"].float().transpose(1, 2).contiguous())
        u = u.reshape(E * s["cap"], -1)[place]
        if s["bias"] is not None:
            u = u + s["bias"].float()[e]
    h = _act(c["act"], u[:, :I]) * u[:, I:] if c["gated"] else _act(c["act"], u)
    if s["res"] is not None:
        h = h + s["res"].float()
    return {"out": h.to(dt), "z": u.to(dt)} if c["z"] else {"out": h.to(dt)}


def _plain_act_grad(s):
    c = s["case"]
    I, dt, d = c["I"], _DT[c["dt"]], s["dout"].float()
    if s["z"] is None:
        du, h = d, None
    else:
        z = s["z"].float()
        u = z[:, :I]
        a, slope = _act(c["act"], u), _act_slope(c["act"], u)
        if c["gated"]:
            du, h = torch.cat([d * z[:, I:] * slope, d * a], dim=1), a * z[:, I:]
        else:
            du, h = d * slope, a
    # sums over long columns in 64 bits
    top = torch.cat([torch.zeros(1, du.shape[1], dtype=torch.float64, device=d.device), du.double().cumsum(0)])
    db = (top[s["off"][1:].long()] - top[s["off"][:-1].long()]).float()
    out = {"db": db}
    if s["z"] is not None:
        out["du"] = du.to(dt)
        if c["h"]:
            out["h"] = h.to(dt)
    return out


def _philox(rng, n):
    """n 16-bit random numbers, 8 from each counter (i / 8, offset) under the key (seed): the ten-round 4 x 32
    generator of Salmon et al., "Parallel random numbers: as easy as 1, 2, 3" (2011)."""
    low = 0xFFFFFFFF
    i = torch.arange((n + 7) // 8, device=rng.device)
    key = [rng[0] & low, (rng[0] >> 32) & low]
    x = [i & low, i >> 32, (rng[1] & low).expand_as(i), ((rng[1] >> 32) & low).expand_as(i)]
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57    # (64-bit products: their bits are right, the sign is not)
        x = [((b >> 32) & low) ^ x[1] ^ key[0], b & low, ((a >> 32) & low) ^ x[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    words = torch.stack(x, dim=1)
    return torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(-1)[:n]


def _drop(v, s):
    """v (fp32) with the elements dropped that the generator names, the others scaled."""
    cut = int(math.floor(s["case"]["p"] * 65536 + 0.5))
    keep = (_philox(s["rng"], v.numel()) >= cut).reshape(v.shape)
    scale = 65536 / (65536 - cut) if cut < 65536 else 0.0
    return torch.where(keep, v * scale, torch.zeros((), device=v.device))


def _plain_combine(s):
    c = s["case"]
    pos = s["pos"].reshape(c["N"], c["k"]).long()
    v = torch.zeros(c["N"], c["H"], device=pos.device)
    for j in range(c["k"]):
        g = torch.where(pos[:, j] >= 0, s["gate"][:, j], torch.zeros((), device=v.device))
        v = v + g[:, None] * s["eo"][pos[:, j].clamp(min=0)].float()
    if s["shared"] is not None:
        v = v + s["shared"].float()
    v = _drop(v, s)
    return {"y": (v if s["res"] is None else v + s["res"].float()).to(_DT[c["y"]])}


def _plain_combine_grad(s):
    c = s["case"]
    dt = _DT[c["dt"]]
    pos = s["pos"].reshape(c["N"], c["k"]).long()
    d = _drop(s["dy"].float(), s)
    spare = torch.zeros(c["N"] * c["k"] + 1, c["H"], dtype=dt, device=d.device)   # (one row more: dropped slots)
    dg = []
    for j in range(c["k"]):
        ok = pos[:, j] >= 0
        spare[torch.where(ok, pos[:, j], torch.full_like(pos[:, j], spare.shape[0] - 1))] = (
            s["gate"][:, j, None] * d).to(dt)
        dot = (d * s["eo"][pos[:, j].clamp(min=0)].float()).sum(dim=1)
        dg.append(torch.where(ok, dot, torch.zeros((), device=d.device)))
    named = torch.zeros(c["N"] * c["k"] + 1, 1, dtype=torch.bool, device=d.device)
    named[torch.where(pos >= 0, pos, torch.full_like(pos, spare.shape[0] - 1)).reshape(-1)] = True
    out = {"d_eo": torch.where(named[:-1], spare[:-1], s["d_eo"]), "d_gate": torch.stack(dg, dim=1)}
    return dict(out, d_shared=d.to(dt)) if c["shared"] else out


def _plain_dropout(s):
    v = _drop(s["x"].float(), s)
    return {"y": (v if s["res"] is None else v + s["res"].float()).to(_DT[s["case"]["y"]])}


# ------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "act_grad": _plain_act_grad, "combine": _plain_combine,
                "combine_grad": _plain_combine_grad, "dropout": _plain_dropout}[op](state)
    import combine_grouped_gemm_amd as moe
    c, s = state["case"], state
    if op in ("linear", "act_grad"):
        act = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "relu2": moe.MOE_ACT_RELU2,
               "gelu": moe.MOE_ACT_GELU, "gelu_tanh": moe.MOE_ACT_GELU_TANH, "silu": moe.MOE_ACT_SILU}[c["act"]]
    if op == "linear":
        out, z = moe.moe_expert_linear(s["a"], s["w"], bias=s["bias"], offsets=s["off"], act=act, gated=c["gated"],
                                       src_slot=s["slot"], k=max(c["k"], 1), residual=s["res"], want_z=c["z"])
        return {"out": out, "z": z} if c["z"] else {"out": out}
    if op == "act_grad":
        du, db, h = moe.moe_expert_act_backward(s["dout"], z=s["z"], offsets=s["off"], act=act, gated=c["gated"],
                                                want_dz=s["z"] is not None, want_h=c["h"] and s["z"] is not None)
        out = {"db": db}
        if du is not None:
            out["du"] = du
        if h is not None:
            out["h"] = h
        return out
    if op == "combine":
        return {"y": moe.moe_combine_dropout(s["eo"], s["pos"], s["gate"], c["p"], s["rng"], shared_out=s["shared"],
                                             residual=s["res"], y_dtype=_DT[c["y"]])}
    if op == "combine_grad":
        d_eo, d_gate, d_shared = moe.moe_combine_dropout_backward(
            s["dy"], s["pos"], s["gate"], s["eo"], c["p"], s["rng"], d_expert_out=s["d_eo"], want_shared=c["shared"])
        out = {"d_eo": d_eo, "d_gate": d_gate}
        return dict(out, d_shared=d_shared) if c["shared"] else out
    return {"y": moe.moe_dropout(s["x"], c["p"], s["rng"], residual=s["res"], y_dtype=_DT[c["y"]])}


_SIZE = {"none": 0, "f32": 4, "bf16": 2}


def work(case):
    op, sz = case["op"], _SIZE[case["dt"]]
    if op == "linear":
        N, k, E, K, I = case["N"], case["k"], case["E"], case["K"], case["I"]
        Nw = 2 * I if case["gated"] else I
        rows, hit = N * max(k, 1), min(E, N * max(k, 1))
        b = sz * ((N if case["gather"] else rows) * K + hit * Nw * K + rows * I * (2 if case["res"] else 1))
        b += hit * Nw * _SIZE[case["bias"]] + (sz * rows * Nw if case["z"] else 0)
        return {"bytes": b, "flops": 2 * rows * K * Nw}
    if op == "act_grad":
        rows, I = case["rows"], case["I"]
        Nw = 2 * I if case["gated"] else I
        plain = case["act"] == "none" and not case["gated"]
        b = sz * rows * I + 4 * min(case["E"], rows) * Nw
        b += 0 if plain else sz * rows * (2 * Nw + (I if case["h"] else 0))
        return {"bytes": b, "flops": 12 * rows * Nw}
    H, ysz = case["H"], _SIZE[case["y"]]
    if op == "dropout":
        n = case["rows"] * H
        return {"bytes": n * (sz + ysz * (2 if case["res"] else 1)), "flops": 20 * n}
    N, k = case["N"], case["k"]
    if op == "combine":
        b = N * H * (sz * (k + (1 if case["shared"] else 0)) + ysz * (2 if case["res"] else 1))
        return {"bytes": b + 8 * N * k, "flops": N * H * (2 * k + 20)}
    b = N * H * (ysz + sz * (2 * k + (1 if case["shared"] else 0)))
    return {"bytes": b + 12 * N * k, "flops": N * H * (3 * k + 20)}


# ------------------------------------------------------------------------------- in 64 bits

def _keep64(rng, n, cut):
    """Which of n elements stay, on the host with unsigned 64-bit products."""
    seed, off = (int(v) for v in rng.tolist())
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    i = np.arange((n + 7) // 8, dtype=np.uint64)
    c0, c1 = i & low, i >> half
    c2, c3 = np.full_like(i, off & 0xFFFFFFFF), np.full_like(i, off >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        m0, m2 = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = (m2 >> half) ^ c1 ^ u(k0), m2 & low, (m0 >> half) ^ c3 ^ u(k1), m0 & low
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    w = np.stack([c0, c1, c2, c3], axis=1).astype("<u4")
    return w.view("<u2").reshape(-1)[:n] >= cut


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: t.double()  # noqa: E731
    op = case["op"]

    def act(u):
        n = case["act"]
        if n in ("relu", "relu2"):
            return torch.relu(u) if n == "relu" else torch.relu(u).square()
        if n == "gelu":
            return u * torch.special.ndtr(u)
        if n == "gelu_tanh":
            return u * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))
        return u * torch.sigmoid(u) if n == "silu" else u

    if op == "linear":
        I, k = case["I"], case["k"]
        off = [0, case["N"]] if s["off"] is None else s["off"].tolist()
        outs, us = [], []
        for e in range(case["E"]):
            r = slice(off[e], off[e + 1])
            a = s["a"][r] if s["slot"] is None else s["a"][s["slot"][r].long() // k]
            u = torch.matmul(d(a), d(s["w"][e]).t())
            us.append(u if s["bias"] is None else u + d(s["bias"][e]))
        u = torch.cat(us)
        out = act(u[:, :I]) * u[:, I:] if case["gated"] else act(u)
        if s["res"] is not None:
            out = out + d(s["res"])
        return {"out": out, "z": u} if case["z"] else {"out": out}
    if op == "act_grad":
        I, off = case["I"], s["off"].tolist()
        g = d(s["dout"])
        if s["z"] is None:
            du, h = g, None
        else:
            # the chain rule left to differentiation in 64 bits, some rows at a time
            du, h = [], []
            for r in range(0, case["rows"], 8192):
                z = d(s["z"][r:r + 8192]).requires_grad_(True)
                o = act(z[:, :I]) * z[:, I:] if case["gated"] else act(z)
                du.append(torch.autograd.grad(o, z, g[r:r + 8192])[0])
                h.append(o.detach() if case["h"] else None)
            du, h = torch.cat(du), torch.cat(h) if case["h"] else None
        out = {"db": torch.stack([du[off[e]:off[e + 1]].sum(dim=0) for e in range(case["E"])])}
        if s["z"] is not None:
            out["du"] = du
            if h is not None:
                out["h"] = h
        return out
    cut = int(math.floor(case["p"] * 65536 + 0.5))
    scale = 65536 / (65536 - cut) if cut < 65536 else 0.0
    rows = case["rows"] if op == "dropout" else case["N"]
    keep = torch.from_numpy(_keep64(s["rng"], rows * case["H"], cut)).to(s["rng"].device).reshape(rows, case["H"])
    if op == "dropout":
        v = d(s["x"]) * keep * scale
        return {"y": v if s["res"] is None else v + d(s["res"])}
    N, k = case["N"], case["k"]
    pos = s["pos"].reshape(N, k).long()
    ok = pos >= 0
    if op == "combine":
        v = torch.zeros(N, case["H"], dtype=torch.float64, device=pos.device)
        for j in range(k):
            t = torch.nonzero(ok[:, j])[:, 0]
            v[t] += d(s["gate"][t, j])[:, None] * d(s["eo"][pos[t, j]])
        if s["shared"] is not None:
            v += d(s["shared"])
        v *= keep * scale
        return {"y": v if s["res"] is None else v + d(s["res"])}
    dv = d(s["dy"]) * keep * scale
    d_eo = d(s["d_eo"])
    d_gate = torch.zeros(N, k, dtype=torch.float64, device=pos.device)
    for j in range(k):
        t = torch.nonzero(ok[:, j])[:, 0]
        d_eo[pos[t, j]] = d(s["gate"][t, j])[:, None] * dv[t]
        d_gate[t, j] = (dv[t] * d(s["eo"][pos[t, j]])).sum(dim=1)
    out = {"d_eo": d_eo, "d_gate": d_gate}
    return dict(out, d_shared=dv) if case["shared"] else out

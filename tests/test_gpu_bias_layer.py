"""Whole layers with biases, other activations, dropout and the residual stream: forward and backward against the oracle's
chain rule in float64, as a training program runs them."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
import workload as w
from combine_grouped_gemm_amd.layer import BiasedMoELayer, MoELayer
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync, token_rel_err, with_logits
from tests.test_gpu_backward import GRAD_BAR, SMALL, mat_rel_err
from tests.test_gpu_bias_experts import ACT
from tests.test_gpu_layer import SMALL as FORWARD

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _return_cached_blocks():
    """The allocator's cached blocks go back afterwards: a test elsewhere counts the bytes it hands out."""
    yield
    torch.cuda.empty_cache()


def _t(shape, seed, dt, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale).to(F32).to(dt).to(DEV)


def _biased(N, H, E, k, I, dt, act, gated, biases=True, w_r=True, seed=0):
    Nw = 2 * I if gated else I
    w1, w2 = _t((E, Nw, H), seed + 1, dt, H ** -0.5), _t((E, H, I), seed + 2, dt, I ** -0.5)
    b1, b2 = (_t((E, Nw), seed + 3, F32, 0.3), _t((E, H), seed + 4, dt, 0.3)) if biases else (None, None)
    wr = _t((E, H), seed + 5, dt, H ** -0.5)
    layer = BiasedMoELayer(N, H, E, k, I, w1, w2, b1, b2, ACT[act], gated, w_r=wr if w_r else None)
    x, res = _t((N, H), seed + 6, dt), _t((N, H), seed + 7, dt)
    z = torch.from_numpy(oracle.router_logits(f64(x), f64(wr))).to(DEV)
    return layer, x, res, z


def _reference(layer, x, res, act, gated, p, seed, off):
    """(y, h, pre, expert outputs, offsets, send_pos, gates) in float64 on the layer's own routes and gates."""
    idx, g = layer.topk_idx.cpu().numpy(), f64(layer.topk_gate)
    n_e, offsets, send_pos, src_slot = oracle.dispatch_layout(idx, layer.E)
    b = lambda t: None if t is None else f64(t)  # noqa: E731
    h, pre = oracle.expert_linear(f64(x), offsets, f64(layer.w1), b(layer.b1), act, gated, tokens=src_slot // layer.k)
    eo, _ = oracle.expert_linear(h, offsets, f64(layer.w2), b(layer.b2))
    y = oracle.combine_dropout(eo, send_pos, g, p, seed, off, None, None if res is None else f64(res))
    return y, h, pre, eo, offsets, send_pos, g


@pytest.mark.parametrize("dt,bar", [(F32, 2e-5), (BF, 2e-2)])
@pytest.mark.parametrize("act,gated,N,H,E,k,I", [("gelu_tanh", False, 37, 136, 5, 2, 264), ("silu", True, 130, 64, 8, 3, 72),
                                                 ("relu2", False, 1, 256, 4, 4, 128), ("gelu", True, 300, 128, 3, 1, 256)])
def test_biased_forward(act, gated, N, H, E, k, I, dt, bar):
    """y and every intermediate; bars as the repository's layers have them (three roundings in bf16: 1e-2, the fp32
    sums of the products 1e-5, each doubled for the biased sums' cancellation)."""
    say(f"biased layer {act} gated={gated} N={N} H={H} E={E} k={k} I={I} {dt}")
    layer, x, res, z = _biased(N, H, E, k, I, dt, act, gated)
    rng = torch.tensor([5, 9], dtype=torch.int64, device=DEV)
    for kw in (dict(), dict(residual=res), dict(residual=res, dropout=0.3, rng=rng), dict(dropout=0.5, rng=rng)):
        y = layer.forward(x, z, save_for_backward=True, **kw)
        sync()
        ref = _reference(layer, x, kw.get("residual"), act, gated, kw.get("dropout", 0.0), 5, 9)
        assert token_rel_err(f64(layer.pre), ref[2]) <= bar and token_rel_err(f64(layer.h), ref[1]) <= bar
        assert token_rel_err(f64(layer.expert_out), ref[3]) <= bar
        # a token whose experts' sum is dropped nearly whole: relative to the largest term, not to what is left
        err = np.abs(f64(y) - ref[0]).max(axis=1)
        scale = np.abs(ref[3]).max() + (np.abs(f64(res)).max(axis=1) if "residual" in kw else 0)
        assert (err / scale).max() <= bar
    own = layer.forward(x, None, residual=res)   # its own logits: the same routes but for near ties
    sync()
    assert own.shape == (N, H) and torch.isfinite(own).all()


@pytest.mark.parametrize("act,gated,biases,w_r,p", [("gelu_tanh", False, True, True, 0.2), ("silu", True, True, True, 0.0),
                                                    ("relu2", False, False, False, 0.5), ("gelu", True, True, False, 0.1)])
def test_biased_backward(act, gated, biases, w_r, p):
    N, H, E, k, I = 300, 256, 12, 3, 384
    say(f"biased backward {act} gated={gated} biases={biases} w_r={w_r} p={p}")
    layer, x, res, z = _biased(N, H, E, k, I, BF, act, gated, biases, w_r, seed=20)
    rng = torch.tensor([3, 4], dtype=torch.int64, device=DEV)
    dy = _t((N, H), 30, BF)
    layer.forward(x, z, save_for_backward=True, residual=res, dropout=p, rng=rng)
    rng += 1   # (the backward goes by the state that the forward used)
    gr = layer.backward(x, dy, dw_dtype=F32)
    sync()
    off, sp = layer.layout[1].cpu().numpy(), layer.layout[2].cpu().numpy()
    g = f64(layer.topk_gate)
    pre, eo = f64(layer.pre), f64(layer.expert_out)
    d_eo, dg, _ = oracle.combine_dropout_backward(f64(dy), sp, g, eo, p, 3, 4)
    dh = np.zeros((N * k, I))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        dh[s] = d_eo[s] @ f64(layer.w2[e])
    dpre, db1, h = oracle.expert_act_backward(pre, dh, off, act, gated)
    d_perm = np.zeros((N * k, H))
    xp = oracle.permute(f64(x), sp, k)
    errs = {"d_eo": token_rel_err(f64(gr["d_eo"]), d_eo), "dg": np.abs(f64(gr["dg"]) - dg).max() / np.abs(dg).max(),
            "dh": token_rel_err(f64(gr["dh"]), dh), "dpre": token_rel_err(f64(gr["dpre"]), dpre)}
    for e in range(E):
        s = slice(off[e], off[e + 1])
        d_perm[s] = dpre[s] @ f64(layer.w1[e])
        errs[f"dw1 {e}"] = mat_rel_err(f64(gr["dw1"][e]), dpre[s].T @ xp[s])
        errs[f"dw2 {e}"] = mat_rel_err(f64(gr["dw2"][e]), d_eo[s].T @ h[s])
    errs["db1"] = mat_rel_err(f64(gr["db1"]), db1)
    errs["db2"] = mat_rel_err(f64(gr["db2"]), np.stack([d_eo[off[e]:off[e + 1]].sum(axis=0) for e in range(E)]))
    dx = oracle.dispatch_backward(d_perm, sp, N, k)
    if w_r:
        dz = oracle.gates_backward(g, dg)
        dxr, dwr = np.zeros((N, H)), np.zeros((E, H))
        idx = layer.topk_idx.cpu().numpy()
        for t in range(N):
            for j in range(k):
                dxr[t] += dz[t, j] * f64(layer.w_r[idx[t, j]])
                dwr[idx[t, j]] += dz[t, j] * f64(x[t])
        dx = dx + dxr
        errs["dw_r"] = mat_rel_err(f64(gr["dw_r"]), dwr)
    errs["dx"] = token_rel_err(f64(gr["dx"]), dx)
    say("  " + ", ".join(f"{n} {v:.1e}" for n, v in errs.items()))
    assert all(v <= GRAD_BAR for v in errs.values())


def test_biased_gradient_by_differences():
    """<dy, y> moves along a direction of b1, b2 and x as the gradients say (fp32 would need no more than the
    bf16 roundings of y: a step that moves y by many of them)."""
    N, H, E, k, I = 200, 128, 4, 2, 128
    layer, x, res, z = _biased(N, H, E, k, I, BF, "gelu_tanh", False, seed=40)
    ref = lambda b1, b2, xx: _reference_sum(layer, xx, b1, b2)  # noqa: E731
    rng = torch.tensor([8, 1], dtype=torch.int64, device=DEV)
    dy = _t((N, H), 50, BF)
    layer.forward(x, z, save_for_backward=True, dropout=0.25, rng=rng)
    gr = layer.backward(x, dy, dw_dtype=F32)
    sync()
    b1, b2 = f64(layer.b1), f64(layer.b2)
    mask = oracle.dropout_mask(0.25, 8, 1, N * H).reshape(N, H)
    f = lambda b1, b2: (ref(b1, b2, f64(x)) * mask * f64(dy)).sum()  # noqa: E731
    d1, d2 = f64(_t(b1.shape, 51, F32)), f64(_t(b2.shape, 52, F32))
    eps = 1e-4
    for v1, v2, got, mag in ((d1, 0 * d2, (d1 * f64(gr["db1"])).sum(), np.linalg.norm(d1) * np.linalg.norm(f64(gr["db1"]))),
                             (0 * d1, d2, (d2 * f64(gr["db2"])).sum(), np.linalg.norm(d2) * np.linalg.norm(f64(gr["db2"])))):
        want = (f(b1 + eps * v1, b2 + eps * v2) - f(b1 - eps * v1, b2 - eps * v2)) / (2 * eps)
        assert abs(got - want) <= GRAD_BAR * mag   # (the gradient's error is below GRAD_BAR of its norm)


def _reference_sum(layer, x, b1, b2):
    idx, g = layer.topk_idx.cpu().numpy(), f64(layer.topk_gate)
    _, offsets, send_pos, src_slot = oracle.dispatch_layout(idx, layer.E)
    h, _ = oracle.expert_linear(x, offsets, f64(layer.w1), b1, "gelu_tanh", False, tokens=src_slot // layer.k)
    eo, _ = oracle.expert_linear(h, offsets, f64(layer.w2), b2)
    return oracle.combine_dropout(eo, send_pos, g, 0.0, 0, 0)


def test_biased_step_captured():
    """A training step in a graph, replayed with the generator advanced and new tokens between."""
    N, H, E, k, I = 150, 128, 6, 2, 256
    say("biased layer: graph")
    layer, x, res, z = _biased(N, H, E, k, I, BF, "silu", True, seed=60)
    dy, rng = _t((N, H), 70, BF), torch.tensor([1, 0], dtype=torch.int64, device=DEV)
    step = lambda: (layer.forward(x, None, True, res, 0.2, rng), layer.backward(x, dy))  # noqa: E731
    step()
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    names = ("dx", "dw1", "dw2", "db1", "db2", "dw_r", "dg")
    for _ in range(3):
        x.normal_()
        dy.normal_()
        rng[1] += 1
        graph.replay()
        sync()
        got = [layer.y.clone()] + [layer.grads[n].clone() for n in names]
        step()
        sync()
        assert all(torch.equal(a, b) for a, b in zip(got, [layer.y] + [layer.grads[n] for n in names]))


# ------------------------------------------------------------------------------- the SwiGLU layer

@pytest.mark.parametrize("save", [False, True, "mxfp8"])
@pytest.mark.parametrize("name", ["dsv3_small", "mixtral_small"])
def test_swiglu_layer_with_dropout_and_residual(name, save):
    """The layer's dropped-out sum plus the residual, and its gradients: those of the layer without dropout for the
    upstream gradient behind the mask."""
    cfg = SMALL[name]
    say(f"SwiGLU layer with dropout {name} save={save}")
    inp = with_logits(w.make_layer_inputs(cfg, DEV))
    make = lambda: MoELayer(cfg.N, cfg.H, cfg.E, cfg.k, cfg.I, cfg.dtype, inp["w13"], inp["w2"], inp.get("sw13"),  # noqa: E731
                            inp.get("sw2"), cfg.n_group, cfg.topk_group, inp["bias"], w_r=inp["w_r"])
    layer, plain = make(), make()
    x, z = inp["x"], inp["z"]
    res, dy = _t((cfg.N, cfg.H), 80, BF), _t((cfg.N, cfg.H), 81, BF)
    rng = torch.tensor([6, 2 ** 35], dtype=torch.int64, device=DEV)
    y0 = plain.forward(x, z, save_for_backward=save).clone()
    only = layer.forward(x, z, save_for_backward=save, residual=res).clone()
    y = layer.forward(x, z, save_for_backward=save, residual=res, dropout=0.25, rng=rng)
    sync()
    eo = f64(layer.expert_out)
    sh = f64(layer.shared_out) if layer.shared else None
    args = (eo, layer.layout[2].cpu().numpy(), f64(layer.topk_gate))
    for got, p in ((only, 0.0), (y, 0.25)):
        ref = oracle.combine_dropout(*args, p, 6, 2 ** 35, sh, f64(res))
        assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 20 * 2.0 ** -24 * np.abs(ref).max())
    rng += 1
    mask = torch.from_numpy(oracle.dropout_mask(0.25, 6, 2 ** 35, cfg.N * cfg.H)).reshape(cfg.N, cfg.H)
    masked = (dy.double().cpu() * mask).float().to(BF).to(DEV)   # (the upstream gradient behind the mask, rounded)
    gr = {n: t.clone() for n, t in layer.backward(None if save == "mxfp8" else x, dy, F32).items() if torch.is_tensor(t)}
    side = {n: t.clone() for n, t in layer.backward(None if save == "mxfp8" else x, dy, F32, overlap_shared=True).items()
            if torch.is_tensor(t)}
    ref = plain.backward(None if save == "mxfp8" else x, masked, F32)
    sync()
    assert torch.equal(y0, plain.y)
    for n in ("dx", "dw13", "dw2", "dsw13", "dsw2", "dw_r", "dg"):
        if n not in ref:
            continue
        assert torch.equal(gr[n], side[n]), n
        # the masked gradient's own rounding (2^-8 a value) beside what the plain layer's roundings are
        err = mat_rel_err(f64(gr[n]).reshape(-1, gr[n].shape[-1]), f64(ref[n]).reshape(-1, gr[n].shape[-1]))
        assert err <= GRAD_BAR, (n, err)
    # without dropout again: the plain layer's bits
    layer.forward(x, z, save_for_backward=save)
    again = layer.backward(None if save == "mxfp8" else x, dy, F32)
    plain_gr = plain.backward(None if save == "mxfp8" else x, dy, F32)
    sync()
    assert torch.equal(layer.y, y0) and all(torch.equal(again[n], plain_gr[n]) for n in ("dx", "dw13", "dw2", "dw_r"))


@pytest.mark.parametrize("name,gate_in_down", [("tiny_f32", False), ("decode_fp8_small", False), ("dsv3_fp8_small", False),
                                               ("dsv3_small", True)])
def test_other_layers_with_dropout_and_residual(name, gate_in_down):
    """fp32 and fp8 layers, and gates applied in the down projection: the same sum, dropped out onto the residual."""
    cfg = FORWARD[name]
    say(f"layer with dropout {name} gate_in_down={gate_in_down}")
    inp = with_logits(w.make_layer_inputs(cfg, DEV))
    layer = MoELayer(cfg.N, cfg.H, cfg.E, cfg.k, cfg.I, cfg.dtype, inp["w13"], inp["w2"], inp.get("sw13"), inp.get("sw2"),
                     cfg.n_group, cfg.topk_group, inp["bias"], gate_in_down=gate_in_down)
    y0 = layer.forward(inp["x"], inp["z"]).clone()
    res = _t((cfg.N, cfg.H), 82, y0.dtype)
    rng = torch.tensor([7, 3], dtype=torch.int64, device=DEV)
    y = layer.forward(inp["x"], inp["z"], residual=res, dropout=0.5, rng=rng).clone()
    sync()
    gate = np.ones((cfg.N, cfg.k)) if layer.gate_in_down else f64(layer.topk_gate)
    args = (f64(layer.expert_out), layer.layout[2].cpu().numpy(), gate, 0.5, 7, 3,
            f64(layer.shared_out) if layer.shared else None, f64(res))
    ref = oracle.combine_dropout(*args)
    mag = oracle.combine_dropout(*[np.abs(v) if isinstance(v, np.ndarray) and v.dtype == np.float64 else v for v in args])
    # y's rounding; at most k + 3 fp32 ones (k slots, the shared row, the scale, the residual less the last)
    half = 2.0 ** -24 if y.dtype == F32 else 2.0 ** -8
    assert np.all(np.abs(f64(y) - ref) <= half * np.abs(ref) + (cfg.k + 3) * 2.0 ** -23 * mag)
    assert torch.equal(layer.forward(inp["x"], inp["z"]), y0)


@pytest.mark.parametrize("act,gated", [("gelu_tanh", False), ("silu", True), ("relu2", False)])
def test_second_weights_gradient_takes_the_forwards_h(act, gated):
    """dw2 is d_eo^T h of the h that w2 multiplied, to the rounding of its fp32 sums: act of the kept, rounded
    pre-activations differs from that h in every other digit of bf16."""
    N, H, E, k, I = 300, 256, 5, 2, 384
    say(f"dw2 of the forward's h {act} gated={gated}")
    layer, x, res, z = _biased(N, H, E, k, I, BF, act, gated, seed=90)
    layer.forward(x, z, save_for_backward=True, residual=res)
    gr = layer.backward(x, _t((N, H), 91, BF), dw_dtype=F32)
    sync()
    off, h, d_eo = layer.layout[1].tolist(), f64(layer.h), f64(gr["d_eo"])
    for e in range(E):
        s = slice(off[e], off[e + 1])
        # products of bf16 values are exact in fp32; their sum rounds once an addition, in any order
        lim = 2 * (off[e + 1] - off[e] + 16) * 2.0 ** -24 * (np.abs(d_eo[s]).T @ np.abs(h[s]))
        assert np.all(np.abs(f64(gr["dw2"][e]) - d_eo[s].T @ h[s]) <= lim), e


@pytest.mark.parametrize("act,gated,p", [("gelu_tanh", False, 0.25), ("silu", True, 0.25), ("gelu", False, 0.0)])
def test_biased_gradients_along_themselves(act, gated, p):
    """<dy, y> moves along each returned gradient, of b1, b2, w1, w2 and x (routes and gates held), by its square norm.

    For a gradient within GRAD_BAR of the true one g in norm, <g, v> along v = got / |got| lies within GRAD_BAR |g| of
    |got|; a missing dropout scale (4/3) or a missing part of the chain rule moves it by a quarter and more."""
    N, H, E, k, I = 200, 128, 4, 2, 128
    say(f"gradients along themselves {act} gated={gated} p={p}")
    layer, x, res, z = _biased(N, H, E, k, I, BF, act, gated, w_r=False, seed=40)
    rng = torch.tensor([8, 1], dtype=torch.int64, device=DEV)
    dy = _t((N, H), 50, BF)
    layer.forward(x, z, save_for_backward=True, residual=res, dropout=p, rng=rng)
    gr = layer.backward(x, dy, dw_dtype=F32)
    sync()
    g = f64(layer.topk_gate)
    _, offsets, send_pos, src_slot = oracle.dispatch_layout(layer.topk_idx.cpu().numpy(), E)
    mask = oracle.dropout_mask(p, 8, 1, N * H).reshape(N, H)
    at = {n: f64(t) for n, t in (("b1", layer.b1), ("b2", layer.b2), ("w1", layer.w1), ("w2", layer.w2), ("x", x))}

    def value(q):
        h, _ = oracle.expert_linear(q["x"], offsets, q["w1"], q["b1"], act, gated, tokens=src_slot // k)
        eo, _ = oracle.expert_linear(h, offsets, q["w2"], q["b2"])
        return (oracle.combine_dropout(eo, send_pos, g, 0.0, 0, 0) * mask * f64(dy)).sum()

    for n, got in (("b1", gr["db1"]), ("b2", gr["db2"]), ("w1", gr["dw1"]), ("w2", gr["dw2"]), ("x", gr["dx"])):
        got = f64(got).reshape(at[n].shape)
        norm = np.linalg.norm(got)
        step = 1e-4 / norm * got      # (a unit direction: the next term of the difference is below 1e-8 of it)
        want = (value({**at, n: at[n] + step}) - value({**at, n: at[n] - step})) / 2e-4
        say(f"  {n}: {want / norm:.4f}")
        assert abs(want / norm - 1) <= GRAD_BAR / (1 - GRAD_BAR), n

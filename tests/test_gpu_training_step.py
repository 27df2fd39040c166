"""The layer's training step with the balance loss and 8-bit kept activations: the operators together,
as a training program uses them, against the chain rule in float64 on the kept values."""
import numpy as np
import pytest
import torch

import workload as w
from combine_grouped_gemm_amd.layer import MoELayer
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync, token_rel_err, with_logits
from tests.test_gpu_backward import GRAD_BAR, SMALL, mat_rel_err

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(autouse=True, scope="module")
def _return_cached_blocks():
    """The allocator's cached blocks go back afterwards: a test elsewhere counts the bytes it hands out, and
    an unsplit block of these sizes would count as more."""
    yield
    torch.cuda.empty_cache()
U32 = 2.0 ** -24


def _layer(cfg, w_r=True, **kw):
    inp = with_logits(w.make_layer_inputs(cfg, DEV))
    layer = MoELayer(cfg.N, cfg.H, cfg.E, cfg.k, cfg.I, cfg.dtype, inp["w13"], inp["w2"], inp.get("sw13"),
                     inp.get("sw2"), cfg.n_group, cfg.topk_group, inp["bias"], w_r=inp["w_r"] if w_r else None, **kw)
    dy = w.normal((cfg.N, cfg.H), w.stream_key(cfg.seed, w.T_EO, 5), DEV, torch.bfloat16, std=1.0)
    return inp, layer, dy


def _kept(pair):
    return oracle.mx_dequantize(pair[0].cpu().numpy(), pair[1].cpu().numpy())


def _reference(cfg, layer, inp, dy, dense=None):
    """Every gradient by the chain rule in float64 from the kept tokens and pre-activations; dense: the
    balance loss's part of the logit gradient."""
    N, E, k, I = cfg.N, cfg.E, cfg.k, cfg.I
    rows = N * k
    x, au, d = _kept(layer.kept_x), _kept(layer.kept_au), f64(dy)
    off, sp = layer.layout[1].cpu().numpy(), layer.layout[2].cpu().numpy()
    g, idx = f64(layer.topk_gate), layer.topk_idx.cpu().numpy()
    r = {"dw13": {}, "dw2": {}}
    dyp, xp = oracle.permute(d, sp, k), oracle.permute(x, sp, k)
    dh = np.zeros((rows, I))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        dh[s] = dyp[s] @ f64(inp["w2"][e])
    d_au, hg, dg = oracle.kept_swiglu_backward(au[:rows], dh, sp, g)
    d_perm = np.zeros((rows, cfg.H))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            r["dw13"][e], r["dw2"][e] = d_au[s].T @ xp[s], dyp[s].T @ hg[s]
            d_perm[s] = d_au[s] @ f64(inp["w13"][e])
    dx = oracle.dispatch_backward(d_perm, sp, N, k)
    if layer.shared:
        dhs = d @ f64(inp["sw2"][0])
        das, hs, _ = oracle.kept_swiglu_backward(au[rows:], dhs)
        r["dsw13"], r["dsw2"] = das.T @ x, d.T @ hs
        dx = dx + das @ f64(inp["sw13"][0])
    dg = dg.reshape(N, k)
    dz = np.zeros((N, E))
    np.put_along_axis(dz, idx.astype(np.int64), oracle.gates_backward(g, dg), axis=1)
    if dense is not None:
        dz = dz + dense
    if layer.w_r is not None:
        r["dw_r"] = dz.T @ x
        dx = dx + dz @ f64(inp["w_r"])
    r.update(dg=dg, dz=dz, dh=dh, d_au=d_au, dx=dx)
    return r


def _compare(cfg, layer, gr, ref):
    errs = {"d_gate": float(np.abs(f64(gr["dg"]) - ref["dg"]).max() / np.abs(ref["dg"]).max())}
    for n in ("dh", "d_au", "dx"):
        errs[n] = token_rel_err(f64(gr[n]), ref[n])
    for n in ("dw13", "dw2"):
        errs[n] = max(mat_rel_err(f64(gr[n][e]), v) for e, v in ref[n].items())
        empty = [e for e in range(cfg.E) if e not in ref[n]]
        assert not f64(gr[n][empty]).any()
    if layer.shared:
        for n in ("dsw13", "dsw2"):
            errs[n] = mat_rel_err(f64(gr[n][0]), ref[n])
    if layer.w_r is not None:
        errs["dw_r"] = mat_rel_err(f64(gr["dw_r"]), ref["dw_r"])
    if "dz_all" in gr:
        assert "dz" not in gr
        errs["dz_all"] = float(np.abs(f64(gr["dz_all"]) - ref["dz"]).max() / np.abs(ref["dz"]).max())
    say("  " + ", ".join(f"{n} {v:.2e}" for n, v in errs.items()))
    # bf16 intermediates round by at most 2^-9 of their row's scale, as in the bf16 layer's backward
    for n, v in errs.items():
        assert v <= GRAD_BAR, n


def _sequences(N):
    seq = torch.tensor([0, N // 3, N // 3, N - 40], dtype=torch.int32, device=DEV)   # one empty, padding behind
    mask = torch.ones(N, dtype=torch.uint8, device=DEV)
    mask[5::9] = 0
    return seq, mask


@pytest.mark.parametrize("name", list(SMALL))
def test_kept_layer_backward(name):
    """Gradients from the kept codes alone (no x); y and the routes are those of the plain forward."""
    cfg = SMALL[name]
    say(f"kept layer backward {name}")
    inp, layer, dy = _layer(cfg)
    y0 = layer.forward(inp["x"], inp["z"]).clone()
    y = layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8")
    sync()
    assert torch.equal(y, y0)
    q, s = oracle.mx_quantize(f64(inp["x"]))
    assert np.array_equal(layer.kept_x[0].cpu().numpy(), q) and np.array_equal(layer.kept_x[1].cpu().numpy(), s)
    # the kept pre-activations: half a code step (2^-4 of the value, 2^-10 of the scale for the
    # smallest), the bf16 rounding before it and the fp32 sum over H
    rows, sp, off = cfg.N * cfg.k, layer.layout[2].cpu().numpy(), layer.layout[1].cpu().numpy()
    xp, got = oracle.permute(f64(inp["x"]), sp, cfg.k), _kept(layer.kept_au)
    for e in range(0, cfg.E, 5):
        a, we = xp[off[e]:off[e + 1]], f64(inp["w13"][e]).T
        au = a @ we
        err = 2 * (cfg.H + 2) * U32 * (np.abs(a) @ np.abs(we))
        err = err + 2.0 ** -8 * (np.abs(au) + err)
        sc = np.repeat(np.exp2(layer.kept_au[1][off[e]:off[e + 1]].cpu().numpy().astype(np.float64) - 127), 32, axis=1)
        assert np.all(np.abs(got[off[e]:off[e + 1]] - au) <= err + 2.0 ** -4 * (np.abs(au) + err) + 2.0 ** -10 * sc)
    layer.out_all = layer._expert_out = None   # the backward does not read the expert outputs
    gr = layer.backward(None, dy, dw_dtype=torch.float32)
    sync()
    assert "au" not in gr
    _compare(cfg, layer, gr, _reference(cfg, layer, inp, dy))


@pytest.mark.parametrize("name", list(SMALL))
@pytest.mark.parametrize("w_r", [True, False], ids=["router", "logits"])
def test_training_step(name, w_r):
    """Balance loss over packed sequences and 8-bit kept activations in one step, then a step without
    either: its gradients are a fresh layer's."""
    cfg = SMALL[name]
    say(f"training step {name} router={w_r}")
    inp, layer, dy = _layer(cfg, w_r)
    seq, mask = _sequences(cfg.N)
    alpha, d_loss = 40.0, torch.full((1,), 0.5, device=DEV)   # (large: both parts of dz count)
    layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8", balance_alpha=alpha, seq_start=seq, token_mask=mask)
    gr = layer.backward(None, dy, d_loss=d_loss)
    sync()
    b = inp["bias_cpu"]
    kw = dict(bias=None if b is None else b.numpy(), seq_start=seq.cpu().numpy(), mask=mask.cpu().numpy())
    z, idx = inp["z_cpu"].numpy(), layer.topk_idx.cpu().numpy()
    rl, rc, rp, rt = oracle.balance_loss(z, idx, alpha, **kw)
    loss, counts, prob, tokens = layer.balance
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    # (logits within 1 of each other: every probability within 2^-23 25, sums of 512 tokens and 64
    # experts within 2^-23 100)
    assert np.abs(f64(prob) - rp).max() <= 2 * U32 * 125 and abs(float(loss) - rl) <= 2 * U32 * 250 * rl
    dense = oracle.balance_loss_backward(z, idx, alpha, d_loss=0.5, **kw)
    assert gr["dz_all"].dtype == (torch.bfloat16 if w_r else torch.float32)
    _compare(cfg, layer, gr, _reference(cfg, layer, inp, dy, dense))
    if not w_r:
        return
    layer.forward(inp["x"], inp["z"])
    gr = layer.backward(inp["x"], dy)
    inp2, fresh, _ = _layer(cfg)
    fresh.forward(inp2["x"], inp2["z"])
    want = fresh.backward(inp2["x"], dy)
    sync()
    assert layer.balance is None and "dz_all" not in gr and set(want) <= set(gr)
    for n in ("dx", "dw13", "dw2", "dw_r", "dz", "dg"):
        assert torch.equal(gr[n], want[n]), n


def test_overlapped_shared_expert_and_repeats():
    """The shared expert's steps on a second stream: the same bits, call after call."""
    cfg = SMALL["dsv3_small"]
    say("training step, shared expert on a second stream")
    inp, layer, dy = _layer(cfg)
    layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8", balance_alpha=0.1)
    names = ("dx", "dw13", "dw2", "dsw13", "dsw2", "dw_r", "dz_all", "dg")
    gr = layer.backward(None, dy)
    ref = {n: gr[n].clone() for n in names}
    for _ in range(3):
        got = layer.backward(None, dy, overlap_shared=True)
        sync()
        for n in names:
            assert torch.equal(got[n], ref[n]), n


def test_captured_training_step():
    """Forward and backward in one captured graph, replayed on new tokens and upstream gradients, with
    eager steps of other kinds on the same layer between the replays."""
    cfg = SMALL["dsv3_small"]
    say("training step in a graph")
    inp, layer, dy = _layer(cfg)
    x, kw = inp["x"].clone(), dict(save_for_backward="mxfp8", balance_alpha=0.1)
    layer.forward(x, **kw)
    layer.backward(None, dy)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, **kw)
        gr = layer.backward(None, dy)
    names = ("dx", "dw13", "dw2", "dsw13", "dsw2", "dw_r", "dz_all", "dg")
    _, other, _ = _layer(cfg)
    for i in range(3):
        x.copy_(w.normal((cfg.N, cfg.H), w.stream_key(77, w.T_X, i), DEV, torch.bfloat16))
        dy.normal_()
        graph.replay()
        sync()
        other.forward(x, **kw)
        want = other.backward(None, dy)
        sync()
        assert torch.equal(layer.balance[0], other.balance[0]) and torch.equal(layer.y, other.y)
        for n in names:
            assert torch.equal(gr[n], want[n]), (i, n)
        saved = layer.balance, layer.balance_args
        layer.forward(inp["x"], save_for_backward=True)      # an eager step of another kind
        layer.backward(inp["x"], dy)
        layer.balance, layer.balance_args = saved
        sync()


def test_refusals():
    cfg = w.CONFIGS["tiny_f32"]
    say("training step: refusals")
    inp, layer, _ = _layer(cfg)
    with pytest.raises(ValueError):
        layer.forward(inp["x"], save_for_backward="mxfp8")
    with pytest.raises(ValueError):
        layer.forward(inp["x"], save_for_backward="fp8")
    cfg = SMALL["dsv3_small"]
    inp, layer, dy = _layer(cfg, fuse_shared=False)
    with pytest.raises(ValueError):
        layer.forward(inp["x"], save_for_backward="mxfp8")
    inp, layer, dy = _layer(cfg)
    layer.forward(inp["x"], save_for_backward=None)   # (any false value)
    with pytest.raises(ValueError):
        layer.backward(None, dy)
    with pytest.raises(ValueError):
        layer.backward(inp["x"], dy, d_loss=torch.ones(1, device=DEV))
    with pytest.raises(ValueError):
        layer.forward(inp["x"], token_mask=torch.ones(cfg.N, dtype=torch.uint8, device=DEV))
    # gates inside the down projection: the kept backward does not need the unscaled outputs
    inp, layer, dy = _layer(cfg, gate_in_down=True)
    layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8")
    gr = layer.backward(None, dy, dw_dtype=torch.float32)
    sync()
    _compare(cfg, layer, gr, _reference(cfg, layer, inp, dy))

"""The training step's digits: the balance loss's part of the router gradients beside a gates' part that is far larger."""
import numpy as np
import pytest
import torch

import workload as w
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync
from tests.test_gpu_balance import U32, _prob_rel, _return_cached_blocks  # noqa: F401
from tests.test_gpu_training_step import _kept, _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k,share", [(32, 4, 2.0 ** -8), (32, 4, 2.0 ** -11), (20, 2, 2.0 ** -10)])
def test_balance_part_of_the_router_gradient(E, k, share):
    """dW_r with the loss less dW_r without it is the loss's own part, to the digits that fp32 sums have, where that
    part is a small share of the gates' part.  (A logit gradient rounded to bf16 is off by 2^-9 of the larger part
    in every summand.)"""
    say(f"balance part of the router gradient E={E} k={k} share={share}")
    N, H = 64, 256
    cfg = w.CONFIGS["dsv3_bf16"].scaled(N=N, H=H, E=E, k=k, I=128, n_group=4, topk_group=2)
    inp, layer, dy = _layer(cfg)
    layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8")
    gr = layer.backward(None, dy, dw_dtype=torch.float32)
    without, g, dg = gr["dw_r"].clone(), f64(layer.topk_gate), f64(gr["dg"])
    sync()
    idx, x, z = layer.topk_idx.cpu().numpy(), _kept(layer.kept_x), inp["z_cpu"].numpy()
    b = inp["bias_cpu"]
    kw = dict(bias=None if b is None else b.numpy())
    gates = np.zeros((N, E))
    np.put_along_axis(gates, idx.astype(np.int64), oracle.gates_backward(g, dg), axis=1)
    alpha = share * np.abs(gates).max() / np.abs(oracle.balance_loss_backward(z, idx, 1.0, **kw)).max()
    layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8", balance_alpha=alpha)
    gr = layer.backward(None, dy, dw_dtype=torch.float32)
    sync()
    assert np.array_equal(f64(gr["dg"]), dg) and np.array_equal(layer.topk_idx.cpu().numpy(), idx)
    part = oracle.balance_loss_backward(z, idx, float(np.float32(alpha)), **kw)
    # both results are fp32 sums of N terms (3 N, where a term is a sum of three) in some order, doubled for second
    # order; a gate's gradient g (dg - sum g dg) takes k + 2 roundings in either, the sum of the two parts one; the
    # loss's own part p (a - sum p a), a about the even load: a within 8 roundings, p within its bound, a 22-step sum
    xa = np.abs(x)
    sel = np.zeros((N, E))
    gd = np.abs(g) * (np.abs(dg) + np.abs(g * dg).sum(axis=1, keepdims=True))
    np.put_along_axis(sel, idx.astype(np.int64), 4 * (k + 2) * U32 * gd, axis=1)
    _, counts, _, _ = oracle.balance_loss(z, idx, alpha, **kw)
    p = oracle._row_softmax(oracle.biased_logits(z, kw["bias"]))
    a = alpha * np.abs(E * counts[0] - k * N) / (k * float(N) ** 2)
    own = p * (a[None, :] + (p @ a)[:, None]) * (2 * _prob_rel(dict(z=z, bias=kw["bias"])) + 2 * U32 * 32)
    err = 2 * 2 * (3 * N + 16) * U32 * ((np.abs(gates) + np.abs(part)).T @ xa)
    err += (2 * sel + own + 2 * U32 * (np.abs(gates) + np.abs(part))).T @ xa
    got, want = f64(gr["dw_r"]) - f64(without), part.T @ x
    say(f"  off by {np.abs(got - want).max():.2e}, allowed {err.max():.2e}, part {np.abs(want).max():.2e}")
    assert np.all(np.abs(got - want) <= err)

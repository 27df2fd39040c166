"""The balance loss on the CPU: the oracle against closed forms and central differences, and the
refusals of its entry points (no GPU needed)."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from combine_grouped_gemm_amd import MOE_BF16, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_F32, \
    MOE_FP8_E4M3, MOE_OK
from oracle import moe_oracle as oracle

FAKE = 4096   # never dereferenced on these paths


def test_even_load_has_loss_alpha():
    """Uniform probabilities (or uniform counts): sum_e (E c/(kT)) P = 1, so the loss is alpha."""
    N, E, k = 12, 6, 2
    idx = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(N)])
    loss, counts, prob, T = oracle.balance_loss(np.zeros((N, E)), idx, 0.25)
    assert abs(loss - 0.25) < 1e-15 and (counts == 4).all() and T[0] == N and np.allclose(prob, 1 / E)
    hot = np.zeros((N, k), np.int64)
    hot[:, 1] = 1
    assert abs(oracle.balance_loss(np.zeros((N, E)), hot, 0.25)[0] - 0.25) < 1e-15
    assert not oracle.balance_loss_backward(np.random.default_rng(0).normal(size=(N, E)), idx, 0.25).round(17).any()


def test_gradient_against_central_differences():
    rng = np.random.default_rng(1)
    N, E, k = 11, 5, 2
    z = rng.normal(size=(N, E)).astype(np.float32)
    idx = rng.integers(-1, E, size=(N, k))
    seq, mask, alpha = [1, 4, 4, 9], rng.random(N) < 0.8, 0.3
    dz = oracle.balance_loss_backward(z, idx, alpha, seq_start=seq, mask=mask, d_loss=1.7)
    # steps of 2^-6 are exact in fp32 (the oracle rounds the biased logits once); the loss's third
    # derivative is below alpha E (each factor of the softmax's below 1), so a central difference
    # is off by at most h^2 / 6 alpha E d_loss
    h = 2.0 ** -6
    z = np.round(z * 1024) / 1024
    dz = oracle.balance_loss_backward(z, idx, alpha, seq_start=seq, mask=mask, d_loss=1.7)
    f = lambda y: 1.7 * oracle.balance_loss(y, idx, alpha, seq_start=seq, mask=mask)[0]  # noqa: E731
    for t in range(N):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - dz[t, e]) <= h * h / 6 * alpha * E * 1.7


def test_refusals():
    L = moe.lib()
    ws = moe.moe_workspace_bytes(moe.MOE_OP_BALANCE_LOSS, 100, 0, 0, 16, 3, 0)
    assert ws > 0 and moe.moe_workspace_bytes(moe.MOE_OP_BALANCE_LOSS, 100, 0, 0, 16, 0, 0) == 0

    def fwd(**kw):
        a = dict(z=FAKE, bias=None, idx=FAKE, N=100, E=16, k=4, seq=FAKE, S=3, mask=None, alpha=0.1, loss=FAKE,
                 counts=FAKE, prob=FAKE, tokens=FAKE, ws=FAKE, ws_bytes=ws, s=None)
        a.update(kw)
        return L.moe_balance_loss(*a.values())

    def bwd(**kw):
        a = dict(z=FAKE, bias=None, idx=FAKE, N=100, E=16, k=4, seq=FAKE, S=3, mask=None, alpha=0.1, counts=FAKE,
                 tokens=FAKE, d_loss=None, gate=None, dg=None, dz=FAKE, dt=MOE_F32, s=None)
        a.update(kw)
        return L.moe_balance_loss_backward(*a.values())

    for f in (fwd, bwd):
        assert f(N=-1) == MOE_ERR_INVALID_ARG and f(E=0) == MOE_ERR_INVALID_ARG and f(k=0) == MOE_ERR_INVALID_ARG
        assert f(k=17) == MOE_ERR_INVALID_ARG and f(S=0) == MOE_ERR_INVALID_ARG
        assert f(seq=None) == MOE_ERR_INVALID_ARG                      # three sequences, no starts
        assert f(E=2000) == MOE_ERR_UNSUPPORTED and f(E=64, k=33) == MOE_ERR_UNSUPPORTED
        assert f(S=70000) == MOE_ERR_UNSUPPORTED and f(N=1 << 28) == MOE_ERR_UNSUPPORTED
        assert f(N=1 << 30, E=1, k=1) == MOE_ERR_UNSUPPORTED
        assert f(z=None) == MOE_ERR_INVALID_ARG and f(idx=None) == MOE_ERR_INVALID_ARG
    for name in ("loss", "counts", "prob", "tokens"):
        assert fwd(**{name: None}) == MOE_ERR_INVALID_ARG
    assert fwd(ws_bytes=ws - 1) == MOE_ERR_WORKSPACE and fwd(ws=None) == MOE_ERR_WORKSPACE
    assert fwd(ws=FAKE + 4) == MOE_ERR_INVALID_ARG
    for name in ("counts", "tokens", "dz"):
        assert bwd(**{name: None}) == MOE_ERR_INVALID_ARG
    assert bwd(gate=FAKE) == MOE_ERR_INVALID_ARG and bwd(dg=FAKE) == MOE_ERR_INVALID_ARG
    assert bwd(dt=MOE_FP8_E4M3) == MOE_ERR_UNSUPPORTED
    assert bwd(N=0, z=None, idx=None, dz=None, dt=MOE_BF16) == MOE_OK


def test_binding_checks_shapes_and_types():
    z, idx = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32)
    for bad in (dict(topk_idx=idx.long()), dict(z=z.double()), dict(topk_idx=idx[:5]), dict(bias=torch.zeros(3)),
                dict(seq_start=torch.zeros(3, dtype=torch.int64)), dict(token_mask=torch.ones(5, dtype=torch.uint8)),
                dict(token_mask=torch.ones(6))):
        with pytest.raises(ValueError):
            moe.moe_balance_loss(**{**dict(z=z, topk_idx=idx, alpha=0.1), **bad})
    c, t = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(counts=c.long()), dict(tokens=torch.zeros(2, dtype=torch.int32)), dict(d_loss=torch.zeros(())),
                dict(topk_gate=torch.zeros(6, 3)), dict(dz=torch.zeros(6, 4, dtype=torch.float16))):
        with pytest.raises(ValueError):
            moe.moe_balance_loss_backward(**{**dict(z=z, topk_idx=idx, alpha=0.1, counts=c, tokens=t), **bad})


def test_dense_router_refusals():
    L = moe.lib()
    need = moe.moe_workspace_bytes(moe.MOE_OP_ROUTER_WGRAD, 4096, 512, 0, 16, 0, MOE_BF16)
    assert need > 0 and need % (16 * 512 * 4) == 0
    assert moe.moe_workspace_bytes(moe.MOE_OP_ROUTER_WGRAD, 1, 512, 0, 16, 0, MOE_BF16) == 0

    def wgrad(**kw):
        a = dict(dz=FAKE, x=FAKE, dt=MOE_BF16, N=4096, E=16, H=512, dw=FAKE, dw_dt=MOE_F32, ws=FAKE, ws_bytes=need, s=None)
        a.update(kw)
        return L.moe_router_dense_wgrad(*a.values())

    def dgrad(**kw):
        a = dict(dz=FAKE, w=FAKE, dt=MOE_BF16, N=4096, E=16, H=512, rest=FAKE, dx=FAKE, s=None)
        a.update(kw)
        return L.moe_router_dense_dgrad(*a.values())

    for f in (wgrad, dgrad):
        assert f(N=-1) == MOE_ERR_INVALID_ARG and f(E=0) == MOE_ERR_INVALID_ARG and f(H=0) == MOE_ERR_INVALID_ARG
        assert f(E=1025) == MOE_ERR_UNSUPPORTED and f(H=516) == MOE_ERR_UNSUPPORTED and f(H=1 << 21) == MOE_ERR_UNSUPPORTED
        assert f(N=1 << 24) == MOE_ERR_UNSUPPORTED and f(dt=MOE_FP8_E4M3) == MOE_ERR_UNSUPPORTED
        assert f(dz=None) == MOE_ERR_INVALID_ARG
    assert wgrad(dw_dt=MOE_FP8_E4M3) == MOE_ERR_UNSUPPORTED
    assert wgrad(ws_bytes=need - 1) == MOE_ERR_WORKSPACE and wgrad(ws=None) == MOE_ERR_WORKSPACE
    for name in ("x", "dw"):
        assert wgrad(**{name: None}) == MOE_ERR_INVALID_ARG and wgrad(**{name: FAKE + 8}) == MOE_ERR_INVALID_ARG
    for name in ("w", "dx"):
        assert dgrad(**{name: None}) == MOE_ERR_INVALID_ARG and dgrad(**{name: FAKE + 8}) == MOE_ERR_INVALID_ARG
    assert dgrad(rest=FAKE + 2) == MOE_ERR_INVALID_ARG and wgrad(ws=FAKE + 8) == MOE_ERR_INVALID_ARG
    assert dgrad(N=0, dz=None) == MOE_OK


def test_dense_router_binding_checks():
    dz, x, w = torch.zeros(6, 4), torch.zeros(6, 8), torch.zeros(4, 8)
    for bad in (dict(dz=dz[:5]), dict(dz=dz.bfloat16()), dict(x=x.half()), dict(dw=torch.zeros(4, 16))):
        with pytest.raises(ValueError):
            moe.moe_router_dense_wgrad(**{**dict(dz=dz, x=x), **bad})
    for bad in (dict(dz=dz[:, :3]), dict(w_r=w.bfloat16()), dict(rest=x[:5]), dict(dx=x.bfloat16())):
        with pytest.raises(ValueError):
            moe.moe_router_dense_dgrad(**{**dict(dz=dz, w_r=w), **bad})


def test_workspaces_at_the_ends_of_their_ranges():
    """Every size of the workspace queries is answered: no tokens, one token, more sequences than
    tokens, the largest counts."""
    for N in (0, 1, 2, 63, 8192, 2 ** 24 - 1, 2 ** 31 - 1):
        for E in (1, 7, 8, 160, 1024):
            for S in (1, 2, 64, 2 ** 20):
                assert 0 <= moe.moe_workspace_bytes(moe.MOE_OP_BALANCE_LOSS, N, 0, 0, E, S, 0) < 2 ** 45
            for H in (8, 7168, 2 ** 20):
                for dt in (MOE_F32, MOE_BF16):
                    ws = moe.moe_workspace_bytes(moe.MOE_OP_ROUTER_WGRAD, N, H, 0, E, 0, dt)
                    assert 0 <= ws <= 1024 * 4 * E * H + 255

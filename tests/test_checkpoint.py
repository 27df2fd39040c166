"""Activations kept in 8 bits, on the CPU: the oracle's format against a brute-force search, its SwiGLU
gradients against central differences, and the refusals of the entry points (no GPU needed)."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from combine_grouped_gemm_amd import MOE_BF16, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_F32, MOE_FP8_E4M3, MOE_OK
from oracle import moe_oracle as oracle

FAKE = 4096   # never dereferenced on these paths


def test_format_against_brute_force():
    """Nearest of all 256 codes at the smallest scale that does not saturate; edge maxima: 448 2^e
    itself, one step above it, zero, the smallest scale, the largest finite value, infinities."""
    rng = np.random.default_rng(0)
    x = rng.normal(size=(12, 64)) * np.exp2(rng.integers(-40, 40, size=(12, 1)).astype(np.float64))
    x[0], x[1, :32], x[1, 32:] = 0, 448 * 2.0 ** 3, np.nextafter(448 * 2.0 ** 3, np.inf)
    x[2] = 2.0 ** -140
    x[3, 5] = np.finfo(np.float32).max
    x[4, 3], x[5, 40] = np.inf, np.nan
    codes, scales = oracle.mx_quantize(x)
    vals = oracle.e4m3_decode(np.arange(256))
    vals = np.unique(vals[np.isfinite(vals)])
    for r in range(12):
        for b in range(2):
            blk = x[r, 32 * b:32 * b + 32]
            if not np.isfinite(blk).all():
                assert scales[r, b] == 255
                continue
            e = int(scales[r, b]) - 127
            amax = np.abs(blk).max()
            assert e >= -117 and amax <= 448 * 2.0 ** e and (e == -117 or amax > 448 * 2.0 ** (e - 1))
            got = oracle.mx_dequantize(codes, scales)[r, 32 * b:32 * b + 32]
            best = np.abs(vals[None, :] * 2.0 ** e - blk[:, None]).min(axis=1)
            assert np.array_equal(np.abs(got - blk), best)
    assert np.isnan(oracle.mx_dequantize(codes, scales)[4, :32]).all()


def test_gate_and_swiglu_gradients_against_differences():
    """y = sum_s g_s W h_row(s), L = <dy, y>: d_gate and d_au against central differences of L."""
    rng = np.random.default_rng(1)
    rows, I, H = 3, 32, 5
    au, g, W = rng.normal(size=(rows, 2 * I)), rng.random(4), rng.normal(size=(H, I))
    pos, dy = np.array([2, -1, 0, 1]), rng.normal(size=(4, H))

    def loss(au, g):
        h = oracle.silu(au[:, :I]) * au[:, I:]
        return sum(g[s] * dy[s] @ (W @ h[r]) for s, r in enumerate(pos) if r >= 0)

    dh = np.zeros((rows, I))
    for s, r in enumerate(pos):
        if r >= 0:
            dh[r] = dy[s] @ W
    d_au, hg, dg = oracle.kept_swiglu_backward(au, dh, pos, g)
    # third derivatives of silu(a) u are below 2 |u| |dh g|, so a step of 2^-10 is off by h^2 / 6 of
    # that, below 2^-20 * 100; the differences themselves round by 2^-52 * 1000 / 2^-10
    tol, st = 2.0 ** -20 * 100 + 2.0 ** -42 * 1000, 2.0 ** -10
    for s in range(4):
        up, dn = g.copy(), g.copy()
        up[s] += st
        dn[s] -= st
        assert abs((loss(au, up) - loss(au, dn)) / (2 * st) - dg[s]) <= tol
    for r in range(rows):
        for c in range(0, 2 * I, 7):
            up, dn = au.copy(), au.copy()
            up[r, c] += st
            dn[r, c] -= st
            assert abs((loss(up, g) - loss(dn, g)) / (2 * st) - d_au[r, c]) <= tol
    assert dg[1] == 0
    # dW = dy^T (g h) over the rows
    dW = sum(np.outer(dy[s], hg[r]) for s, r in enumerate(pos) if r >= 0)
    up, dn = W.copy(), W.copy()
    up[1, 3] += st
    dn[1, 3] -= st
    h = oracle.silu(au[:, :I]) * au[:, I:]
    f = lambda w: sum(g[s] * dy[s] @ (w @ h[r]) for s, r in enumerate(pos) if r >= 0)  # noqa: E731
    assert abs((f(up) - f(dn)) / (2 * st) - dW[1, 3]) <= tol


def test_refusals():
    L = moe.lib()

    def quant(**kw):
        a = dict(x=FAKE, dt=MOE_BF16, rows=10, cols=96, q=FAKE, scale=FAKE, s=None)
        a.update(kw)
        return L.moe_quantize_mxfp8(*a.values())

    def deq(**kw):
        a = dict(q=FAKE, scale=FAKE, rows=10, cols=96, k=2, pos=FAKE, out_rows=20, out=FAKE, dt=MOE_BF16, s=None)
        a.update(kw)
        return L.moe_dequantize_mxfp8(*a.values())

    def bwd(**kw):
        a = dict(q=FAKE, scale=FAKE, dh=FAKE, dt=MOE_BF16, rows=10, I=96, slots=12, pos=FAKE, gate=FAKE, d_au=FAKE,
                 h=FAKE, dg=FAKE, s=None)
        a.update(kw)
        return L.moe_swiglu_backward_mxfp8(*a.values())

    for f in (quant, deq):
        assert f(rows=-1) == MOE_ERR_INVALID_ARG and f(cols=0) == MOE_ERR_INVALID_ARG
        assert f(cols=100) == MOE_ERR_UNSUPPORTED and f(dt=MOE_FP8_E4M3) == MOE_ERR_UNSUPPORTED
        assert f(q=None) == MOE_ERR_INVALID_ARG and f(scale=None) == MOE_ERR_INVALID_ARG
        assert f(q=FAKE + 8) == MOE_ERR_INVALID_ARG
        assert f(rows=0, q=None, scale=None) == MOE_OK
    assert quant(x=None) == MOE_ERR_INVALID_ARG and quant(x=FAKE + 2) == MOE_ERR_INVALID_ARG
    assert deq(out=None) == MOE_ERR_INVALID_ARG and deq(out=FAKE + 2) == MOE_ERR_INVALID_ARG
    assert deq(pos=None) == MOE_ERR_INVALID_ARG          # k = 2 without positions
    assert deq(k=0) == MOE_ERR_INVALID_ARG and deq(k=33) == MOE_ERR_UNSUPPORTED
    assert deq(out_rows=-1) == MOE_ERR_INVALID_ARG and deq(rows=1 << 24) == MOE_ERR_UNSUPPORTED
    assert bwd(rows=-1) == MOE_ERR_INVALID_ARG and bwd(I=0) == MOE_ERR_INVALID_ARG and bwd(slots=-1) == MOE_ERR_INVALID_ARG
    assert bwd(I=100) == MOE_ERR_UNSUPPORTED and bwd(dt=MOE_FP8_E4M3) == MOE_ERR_UNSUPPORTED
    assert bwd(slots=1 << 24) == MOE_ERR_UNSUPPORTED and bwd(pos=None) == MOE_ERR_INVALID_ARG   # 12 slots, 10 rows
    for name in ("q", "scale", "dh", "d_au", "h"):
        assert bwd(**{name: None}) == MOE_ERR_INVALID_ARG
    for name in ("q", "dh", "d_au", "h"):
        assert bwd(**{name: FAKE + 4}) == MOE_ERR_INVALID_ARG
    assert bwd(slots=0) == MOE_OK and MOE_F32 == 0


def test_binding_checks_shapes_and_types():
    x = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp8(x.half())
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp8(x, scale=s[:, :1])
    for bad in (dict(q=q.float()), dict(scale=s[:3]), dict(send_pos=torch.zeros(4, dtype=torch.int64)),
                dict(send_pos=torch.zeros(5, dtype=torch.int32)), dict(out=torch.zeros(4, 64, dtype=torch.float16))):
        with pytest.raises(ValueError):
            moe.moe_dequantize_mxfp8(**{**dict(q=q, scale=s), **bad})
    dh = torch.zeros(4, 32)
    for bad in (dict(dh=dh.half()), dict(au_q=q[:, :32]), dict(au_scale=s[:3]), dict(topk_gate=torch.zeros(2, 3)),
                dict(d_au=torch.zeros(4, 64, dtype=torch.bfloat16)), dict(h=torch.zeros(4, 64)),
                dict(send_pos=torch.zeros(4, dtype=torch.int64)), dict(d_gate=torch.zeros(4, dtype=torch.float64))):
        with pytest.raises(ValueError):
            moe.moe_swiglu_backward_mxfp8(**{**dict(au_q=q, au_scale=s, dh=dh), **bad})


def test_gate_up_refusals():
    L = moe.lib()
    ws = moe.moe_workspace_bytes(moe.MOE_OP_EXPERT_GEMM, 80 + 40, 256, 128, 9, 1, MOE_BF16)

    def f(**kw):
        a = dict(x=FAKE, dt=MOE_BF16, N=40, ss=FAKE, k=2, off=FAKE, E=8, rows=80, H=256, I=128, w13=FAKE, sw=FAKE, h=FAKE,
                 q=FAKE, scale=FAKE, ws=FAKE, ws_bytes=ws, s=None)
        a.update(kw)
        return L.moe_expert_gate_up_mxfp8(*a.values())

    assert f(dt=MOE_F32) == MOE_ERR_UNSUPPORTED and f(E=1024) == MOE_ERR_UNSUPPORTED
    assert f(H=200) == MOE_ERR_UNSUPPORTED and f(I=96) == MOE_ERR_UNSUPPORTED
    assert f(E=0) == MOE_ERR_INVALID_ARG and f(rows=-1) == MOE_ERR_INVALID_ARG and f(k=0) == MOE_ERR_INVALID_ARG
    assert f(N=0) == MOE_ERR_INVALID_ARG and f(off=None) == MOE_ERR_INVALID_ARG
    for name in ("x", "ss", "w13", "h", "q", "scale"):
        assert f(**{name: None}) == MOE_ERR_INVALID_ARG
    for name in ("x", "w13", "sw", "h", "q"):
        assert f(**{name: FAKE + 8}) == MOE_ERR_INVALID_ARG
    assert f(ws_bytes=ws - 1) == moe.MOE_ERR_WORKSPACE and f(ws=None) == moe.MOE_ERR_WORKSPACE
    assert f(N=0, rows=0, x=None, h=None) == MOE_OK
    x, ss, off = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 256, 128, dtype=torch.bfloat16)
    for bad in (dict(x=x.float()), dict(w13=w.float()), dict(offsets=off[:2]), dict(src_slot=ss.long()), dict(rows=9),
                dict(shared_w13=w), dict(h=torch.zeros(8, 64, dtype=torch.bfloat16)),
                dict(au_scale=torch.zeros(8, 4, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            moe.moe_expert_gate_up_mxfp8(**{**dict(x=x, src_slot=ss, k=2, offsets=off, w13=w), **bad})

"""Experts with biases, other activations and dropout, on the CPU: the oracle's functions against known answers and
differences, and the refusals of the C entry points and of their bindings (no GPU needed)."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from combine_grouped_gemm_amd import (MOE_BF16, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_F32,
                                      MOE_FP8_E4M3, MOE_OK)
from oracle import moe_oracle as oracle

FAKE = 4096   # a non-null, 16-byte aligned host integer: never dereferenced on these paths


# ------------------------------------------------------------------------------- the oracle

def test_philox_known_answers():
    """The generator's published test vectors (ten rounds)."""
    assert oracle.philox((0,) * 4, (0,) * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert oracle.philox((f,) * 4, (f,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert oracle.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_mask():
    m = oracle.dropout_mask(0.25, 7, 3, 40000)
    assert set(np.unique(m)) == {0.0, 4 / 3}
    # 40000 draws: the share dropped within 5 standard deviations of 1/4
    assert abs((m == 0).mean() - 0.25) < 5 * np.sqrt(0.25 * 0.75 / 40000)
    assert np.array_equal(m[:1000], oracle.dropout_mask(0.25, 7, 3, 1000))   # a place's number is its own
    assert not np.array_equal(m, oracle.dropout_mask(0.25, 7, 4, 40000))
    assert not np.array_equal(m, oracle.dropout_mask(0.25, 8, 3, 40000))
    assert np.all(oracle.dropout_mask(0.0, 1, 2, 100) == 1) and np.all(oracle.dropout_mask(1.0, 1, 2, 100) == 0)
    # the high words of seed and offset count
    assert not np.array_equal(m, oracle.dropout_mask(0.25, 7 + 2 ** 32, 3, 40000))
    assert not np.array_equal(m, oracle.dropout_mask(0.25, 7, 3 + 2 ** 32, 40000))


@pytest.mark.parametrize("act", sorted(oracle.ACTIVATIONS))
def test_activation_slopes_by_differences(act):
    x = np.linspace(-6, 6, 241) + 0.01   # (not at the kinks)
    f = oracle.ACTIVATIONS[act]
    h = 1e-5
    assert np.allclose((f(x + h) - f(x - h)) / (2 * h), oracle.ACTIVATION_SLOPES[act](x), atol=1e-8)


def test_activations_against_torch():
    x = torch.linspace(-8, 8, 400, dtype=torch.float64)
    F = torch.nn.functional
    for act, ref in (("relu", F.relu(x)), ("gelu", F.gelu(x)), ("gelu_tanh", F.gelu(x, approximate="tanh")),
                     ("silu", F.silu(x)), ("relu2", F.relu(x) ** 2)):
        assert np.allclose(oracle.ACTIVATIONS[act](x.numpy()), ref.numpy(), atol=1e-14)


def test_normal_tail_polynomial():
    """The polynomial by which rounded values take Phi, its coefficients read from the source: within 1.2e-5 of
    the scaled tail exp(x^2 / 2) Phi(-x)."""
    import os
    import re
    from scipy.special import erfcx
    text = open(os.path.join(os.path.dirname(moe.library_path()), "csrc", "activation.h")).read()
    body = text[text.index("const float t = "):text.index("q *= t * e")]
    c = float(re.search(r"fmaf\(([\d.]+)f, fabsf", body).group(1))
    co = [float(v) for v in re.findall(r"(-?\d\.\d{6,})f", body)]
    assert len(co) == 6
    x = np.concatenate([np.linspace(0, 8, 20001), np.linspace(8, 40, 10001)])
    t = 1 / (1 + c * x)
    q = np.polyval(co + [0.0], t)
    assert np.abs(q / (0.5 * erfcx(x / np.sqrt(2))) - 1).max() < 1.2e-5


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", sorted(oracle.ACTIVATIONS))
def test_act_backward_by_differences(act, gated):
    """<d_out, out> moves with the biases and with z as db and dz say."""
    rng = np.random.default_rng(5)
    off, N, K = [0, 3, 3, 8], 4, 5
    Nw = 8 if gated else 4
    a, w, b = rng.normal(size=(8, K)), rng.normal(size=(3, Nw, K)), rng.normal(size=(3, Nw))
    d = rng.normal(size=(8, N))
    _, z = oracle.expert_linear(a, off, w, b, act, gated)
    dz, db, h = oracle.expert_act_backward(z, d, off, act, gated)
    f = lambda bias: (oracle.expert_linear(a, off, w, bias, act, gated)[0] * d).sum()  # noqa: E731
    eps = 1e-6
    for e, c in ((0, 0), (2, Nw - 1), (1, 1), (2, N - 1)):
        up, dn = b.copy(), b.copy()
        up[e, c] += eps
        dn[e, c] -= eps
        assert abs((f(up) - f(dn)) / (2 * eps) - db[e, c]) < 1e-7
    assert np.allclose(h, oracle.expert_linear(a, off, w, b, act, gated)[0]) and not db[1].any()


def test_combine_dropout_backward_by_differences():
    rng = np.random.default_rng(6)
    N, k, H = 5, 2, 16
    pos = np.array([3, 0, -1, 5, 1, 2, 4, 6, 7, 8])
    eo, g, sh, dy = rng.normal(size=(10, H)), rng.random((N, k)), rng.normal(size=(N, H)), rng.normal(size=(N, H))
    d_eo, dg, dsh = oracle.combine_dropout_backward(dy, pos, g, eo, 0.3, 11, 12)
    f = lambda eo_, g_, sh_: (oracle.combine_dropout(eo_, pos, g_, 0.3, 11, 12, sh_) * dy).sum()  # noqa: E731
    eps = 1e-6
    for t, j in ((0, 0), (1, 0), (4, 1)):
        u, v = g.copy(), g.copy()
        u[t, j] += eps
        v[t, j] -= eps
        assert abs((f(eo, u, sh) - f(eo, v, sh)) / (2 * eps) - dg[t, j]) < 1e-7
    for r, c in ((3, 0), (8, 15), (5, 7)):
        u, v = eo.copy(), eo.copy()
        u[r, c] += eps
        v[r, c] -= eps
        assert abs((f(u, g, sh) - f(v, g, sh)) / (2 * eps) - d_eo[r, c]) < 1e-7
    u, v = sh.copy(), sh.copy()
    u[2, 3] += eps
    v[2, 3] -= eps
    assert abs((f(eo, g, u) - f(eo, g, v)) / (2 * eps) - dsh[2, 3]) < 1e-7
    assert np.isnan(d_eo[9]).all() and dg[1, 0] == 0


def test_planted_mistakes_are_found(monkeypatch):
    """A swapped half, a mask of the wrong place and a slope without its chain factor change what the pins see."""
    rng = np.random.default_rng(7)
    a, w, d = rng.normal(size=(4, 3)), rng.normal(size=(1, 8, 3)), rng.normal(size=(4, 4))
    _, z = oracle.expert_linear(a, [0, 4], w, None, "silu", True)
    good = oracle.expert_act_backward(z, d, [0, 4], "silu", True)[0]
    swapped = oracle.expert_act_backward(np.concatenate([z[:, 4:], z[:, :4]], axis=1), d, [0, 4], "silu", True)[0]
    assert not np.allclose(good, swapped)
    monkeypatch.setitem(oracle.ACTIVATION_SLOPES, "silu", lambda x: 1 / (1 + np.exp(-x)))
    assert not np.allclose(good, oracle.expert_act_backward(z, d, [0, 4], "silu", True)[0])
    assert not np.array_equal(oracle.dropout_mask(0.5, 1, 1, 64)[8:], oracle.dropout_mask(0.5, 1, 1, 56))


# ------------------------------------------------------------------------------- the C entry points

def _linear(**kw):
    v = dict(a=FAKE, dt=MOE_BF16, a_nrows=64, src=FAKE, k=2, off=FAKE, E=4, rows=128, K=64, N=64, w=FAKE, bias=FAKE,
             bias_dt=MOE_F32, act=moe.MOE_ACT_SILU, gated=1, res=FAKE, out=FAKE, z=FAKE, ws=FAKE, ws_bytes=1 << 40)
    v.update(kw)
    return moe.lib().moe_expert_linear(*v.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(E=0), MOE_ERR_INVALID_ARG), (dict(rows=-1), MOE_ERR_INVALID_ARG), (dict(K=0), MOE_ERR_INVALID_ARG),
    (dict(N=0), MOE_ERR_INVALID_ARG), (dict(k=0), MOE_ERR_INVALID_ARG), (dict(a_nrows=-1), MOE_ERR_INVALID_ARG),
    (dict(a_nrows=0), MOE_ERR_INVALID_ARG), (dict(off=None), MOE_ERR_INVALID_ARG), (dict(act=6), MOE_ERR_INVALID_ARG),
    (dict(act=-1), MOE_ERR_INVALID_ARG), (dict(gated=2), MOE_ERR_INVALID_ARG), (dict(a=None), MOE_ERR_INVALID_ARG),
    (dict(w=None), MOE_ERR_INVALID_ARG), (dict(out=None), MOE_ERR_INVALID_ARG), (dict(a=FAKE + 8), MOE_ERR_INVALID_ARG),
    (dict(bias=FAKE + 4), MOE_ERR_INVALID_ARG), (dict(res=FAKE + 2), MOE_ERR_INVALID_ARG),
    (dict(z=FAKE + 8), MOE_ERR_INVALID_ARG), (dict(w=FAKE + 8), MOE_ERR_INVALID_ARG),
    (dict(out=FAKE + 8), MOE_ERR_INVALID_ARG), (dict(dt=MOE_FP8_E4M3), MOE_ERR_UNSUPPORTED),
    (dict(bias_dt=MOE_FP8_E4M3), MOE_ERR_UNSUPPORTED), (dict(dt=MOE_F32, bias_dt=MOE_BF16), MOE_ERR_UNSUPPORTED),
    (dict(K=60), MOE_ERR_UNSUPPORTED), (dict(N=60), MOE_ERR_UNSUPPORTED), (dict(E=1025), MOE_ERR_UNSUPPORTED),
    (dict(K=1 << 20), MOE_ERR_UNSUPPORTED), (dict(N=1 << 24), MOE_ERR_UNSUPPORTED),
    (dict(a_nrows=1 << 20, K=2048), MOE_ERR_UNSUPPORTED), (dict(rows=2 ** 31 - 2 ** 16, N=8), MOE_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31 - 2 ** 16 - 1, N=1 << 20), MOE_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31 - 2 ** 16 - 1, N=88), MOE_ERR_UNSUPPORTED)])
def test_linear_refusals(bad, status):
    assert _linear(**bad) == status


def test_linear_without_rows():
    assert _linear(rows=0) == MOE_OK and _linear(rows=0, a=None, w=None, out=None) == MOE_OK
    assert moe.moe_workspace_bytes(moe.MOE_OP_EXPERT_LINEAR, 0, 64, 64, 4, 0, MOE_BF16) == 0


def test_linear_workspace():
    """Every size has an answer, and a smaller workspace than that is refused."""
    for dt in (MOE_BF16, MOE_F32):
        for rows in (1, 2, 17, 100, 4096, 2 ** 31 - 2 ** 16 - 1):
            for K, Nw in ((8, 8), (14336, 4096), (4096, 14336), (2 ** 20 - 8, 8)):
                for E in (1, 8, 1024):
                    need = moe.moe_workspace_bytes(moe.MOE_OP_EXPERT_LINEAR, rows, K, Nw, E, 0, dt)
                    assert 0 <= need < 2 ** 40
                    if need and rows < 10000:
                        kw = dict(dt=dt, rows=rows, K=K, N=Nw, E=E, gated=0, src=None)
                        assert _linear(ws_bytes=need - 1, **kw) == MOE_ERR_WORKSPACE
                        assert _linear(ws=None, **kw) == MOE_ERR_WORKSPACE
                        assert _linear(ws=FAKE + 8, **kw) == MOE_ERR_INVALID_ARG


def _act(**kw):
    v = dict(z=FAKE, d=FAKE, dt=MOE_BF16, off=FAKE, E=4, rows=1280, N=64, act=moe.MOE_ACT_SILU, gated=0, dz=FAKE, db=FAKE,
             db_dt=MOE_F32, h=FAKE, ws=FAKE, ws_bytes=1 << 40)
    v.update(kw)
    return moe.lib().moe_expert_act_backward(*v.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(E=0), MOE_ERR_INVALID_ARG), (dict(rows=-1), MOE_ERR_INVALID_ARG), (dict(N=0), MOE_ERR_INVALID_ARG),
    (dict(off=None), MOE_ERR_INVALID_ARG), (dict(act=9), MOE_ERR_INVALID_ARG), (dict(gated=-1), MOE_ERR_INVALID_ARG),
    (dict(z=None), MOE_ERR_INVALID_ARG), (dict(z=None, act=0), MOE_ERR_INVALID_ARG),
    (dict(z=None, act=0, gated=1, h=None), MOE_ERR_INVALID_ARG), (dict(d=None), MOE_ERR_INVALID_ARG),
    (dict(dz=None, db=None, h=None), MOE_ERR_INVALID_ARG), (dict(db=FAKE + 4), MOE_ERR_INVALID_ARG),
    (dict(z=FAKE + 4), MOE_ERR_INVALID_ARG), (dict(d=FAKE + 8), MOE_ERR_INVALID_ARG),
    (dict(dz=FAKE + 8), MOE_ERR_INVALID_ARG), (dict(h=FAKE + 8), MOE_ERR_INVALID_ARG),
    (dict(ws=FAKE + 8), MOE_ERR_INVALID_ARG), (dict(dt=MOE_FP8_E4M3), MOE_ERR_UNSUPPORTED),
    (dict(db_dt=MOE_FP8_E4M3), MOE_ERR_UNSUPPORTED), (dict(N=60), MOE_ERR_UNSUPPORTED),
    (dict(E=1025), MOE_ERR_UNSUPPORTED), (dict(N=1 << 24), MOE_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31 - 2 ** 16), MOE_ERR_UNSUPPORTED), (dict(ws=None), MOE_ERR_WORKSPACE),
    (dict(ws_bytes=0), MOE_ERR_WORKSPACE)])
def test_act_backward_refusals(bad, status):
    assert _act(**bad) == status


def test_act_backward_workspace():
    assert _act(rows=0, db=None) == MOE_OK
    for rows in (1, 31, 300, 65536, 2 ** 31 - 2 ** 16 - 1):
        for Nw in (8, 520, 4096, 1 << 24):
            need = moe.moe_workspace_bytes(moe.MOE_OP_ACT_BACKWARD, rows, 0, Nw, 16, 0, 0)
            # a partial row is written for every expert and every range of at least 4 rows, but for the few rows that
            # one launch sums
            if rows <= 300 and Nw <= 520:
                assert need == 0
                continue
            assert 17 * Nw * 4 <= need <= (rows // 4 + 17) * Nw * 4
            if Nw < 1 << 24 and Nw % 8 == 0:
                assert _act(rows=rows, N=Nw, E=16, ws_bytes=need - 1) == MOE_ERR_WORKSPACE


def _cd(**kw):
    v = dict(eo=FAKE, eo_dt=MOE_BF16, rows=32, N=16, H=64, k=2, pos=FAKE, gate=FAKE, sh=FAKE, res=FAKE, p=0.1, rng=FAKE, y=FAKE,
             y_dt=MOE_F32)
    v.update(kw)
    return moe.lib().moe_combine_dropout(*v.values(), None)


def _cdb(**kw):
    v = dict(dy=FAKE, dy_dt=MOE_F32, dt=MOE_BF16, rows=32, N=16, H=64, k=2, pos=FAKE, gate=FAKE, eo=FAKE, p=0.1, rng=FAKE,
             d_eo=FAKE, dg=FAKE, dsh=FAKE)
    v.update(kw)
    return moe.lib().moe_combine_dropout_backward(*v.values(), None)


@pytest.mark.parametrize("f", [_cd, _cdb])
def test_combine_dropout_refusals(f):
    inv, un = MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED
    for bad in (dict(rows=-1), dict(N=-1), dict(H=0), dict(k=0), dict(p=-0.1), dict(p=1.001), dict(p=float("nan")), dict(rng=None),
                dict(rng=FAKE + 4), dict(pos=None)):
        assert f(**bad) == inv, bad
    for bad in (dict(k=33), dict(H=60), dict(N=1 << 24)):
        assert f(**bad) == un, bad
    assert f(N=0) == MOE_OK


def test_combine_dropout_pointers_and_types():
    inv, un = MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED
    for bad in (dict(eo=None), dict(y=None), dict(eo=FAKE + 8), dict(y=FAKE + 8), dict(sh=FAKE + 8), dict(res=FAKE + 8)):
        assert _cd(**bad) == inv, bad
    assert _cd(eo_dt=MOE_FP8_E4M3) == un and _cd(y_dt=MOE_FP8_E4M3) == un
    for bad in (dict(dy=None), dict(d_eo=None), dict(eo=None), dict(dy=FAKE + 8), dict(d_eo=FAKE + 8), dict(eo=FAKE + 8),
                dict(dsh=FAKE + 8)):
        assert _cdb(**bad) == inv, bad
    assert _cdb(dt=MOE_FP8_E4M3) == un and _cdb(dt=MOE_F32, dy_dt=MOE_BF16) == un


def test_dropout_refusals():
    f = moe.lib().moe_dropout
    inv, un = MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED
    assert f(FAKE, MOE_BF16, -1, 0.1, FAKE, None, FAKE, MOE_BF16, None) == inv
    assert f(FAKE, MOE_BF16, 8, 1.5, FAKE, None, FAKE, MOE_BF16, None) == inv
    assert f(FAKE, MOE_BF16, 8, 0.5, None, None, FAKE, MOE_BF16, None) == inv
    assert f(None, MOE_BF16, 8, 0.5, FAKE, None, FAKE, MOE_BF16, None) == inv
    assert f(FAKE, MOE_BF16, 8, 0.5, FAKE, None, None, MOE_BF16, None) == inv
    assert f(FAKE + 2, MOE_BF16, 8, 0.5, FAKE, None, FAKE, MOE_BF16, None) == inv
    assert f(FAKE, MOE_BF16, 8, 0.5, FAKE, FAKE + 2, FAKE, MOE_BF16, None) == inv
    assert f(FAKE, MOE_FP8_E4M3, 8, 0.5, FAKE, None, FAKE, MOE_BF16, None) == un
    assert f(FAKE, MOE_BF16, 8, 0.5, FAKE, None, FAKE, MOE_FP8_E4M3, None) == un
    assert f(FAKE, MOE_BF16, 1 << 41, 0.5, FAKE, None, FAKE, MOE_BF16, None) == un
    assert f(None, MOE_BF16, 0, 0.5, FAKE, None, None, MOE_BF16, None) == MOE_OK


# ------------------------------------------------------------------------------- the bindings

def test_linear_binding_refusals():
    bf = torch.bfloat16
    a, w = torch.zeros(6, 16, dtype=bf), torch.zeros(2, 8, 16, dtype=bf)
    off, slot = torch.zeros(3, dtype=torch.int32), torch.zeros(12, dtype=torch.int32)
    good = dict(a=a, w=w, offsets=off, src_slot=slot, k=2)
    for bad in (dict(a=a.half()), dict(a=a[0]), dict(w=w[0]), dict(w=w[:, :, :8]), dict(w=w.float()),
                dict(w=torch.zeros(2, 7, 16, dtype=bf), gated=True), dict(bias=torch.zeros(2, 7)),
                dict(bias=torch.zeros(2, 8).half()), dict(offsets=None), dict(offsets=off[:2]), dict(offsets=off.long()),
                dict(src_slot=slot.long()), dict(rows=13), dict(rows=-1), dict(rows=7, src_slot=None),
                dict(residual=torch.zeros(12, 8)), dict(residual=torch.zeros(11, 8, dtype=bf)),
                dict(out=torch.zeros(12, 8)), dict(z=torch.zeros(12, 16, dtype=bf)),
                dict(out=torch.zeros(12, 8, dtype=bf, device="meta")),
                dict(ws=torch.zeros(8, dtype=torch.uint8, device="meta"))):
        with pytest.raises(ValueError):
            moe.moe_expert_linear(**{**good, **bad})


def test_act_backward_binding_refusals():
    bf = torch.bfloat16
    d, z, off = torch.zeros(6, 8, dtype=bf), torch.zeros(6, 16, dtype=bf), torch.zeros(3, dtype=torch.int32)
    good = dict(d_out=d, z=z, offsets=off, act=moe.MOE_ACT_SILU, gated=True)
    for bad in (dict(d_out=d.half()), dict(d_out=d[0]), dict(z=z.float()), dict(z=z[:, :8]), dict(offsets=off.long()),
                dict(E=3), dict(offsets=None, E=2), dict(dz=z.float()), dict(db=torch.zeros(2, 8)),
                dict(db=torch.zeros(2, 16).half()), dict(h=z), dict(ws=torch.zeros(8, dtype=torch.uint8, device="meta"))):
        with pytest.raises(ValueError):
            moe.moe_expert_act_backward(**{**good, **bad})


def test_dropout_binding_refusals():
    eo, pos, g = torch.zeros(12, 16), torch.zeros(12, dtype=torch.int32), torch.zeros(6, 2)
    rng, dy = torch.zeros(2, dtype=torch.int64), torch.zeros(6, 16)
    good = dict(expert_out=eo, send_pos=pos, topk_gate=g, p=0.1, rng=rng)
    for bad in (dict(expert_out=eo.half()), dict(expert_out=eo[0]), dict(send_pos=pos[:11]), dict(send_pos=pos.long()),
                dict(topk_gate=g.double()), dict(topk_gate=g[0]), dict(topk_gate=None), dict(topk_gate=None, k=0),
                dict(topk_gate=None, k=5), dict(rng=rng[:1]), dict(rng=rng.int()), dict(rng=rng.to("meta")),
                dict(shared_out=dy[:5]), dict(shared_out=dy.bfloat16()), dict(residual=dy.bfloat16(), y=dy),
                dict(residual=dy[:, :8]), dict(y=dy.half())):
        with pytest.raises(ValueError):
            moe.moe_combine_dropout(**{**good, **bad})
    good = dict(dy=dy, send_pos=pos, topk_gate=g, expert_out=eo, p=0.1, rng=rng)
    for bad in (dict(dy=dy[0]), dict(dy=dy.half()), dict(dy=dy.bfloat16()), dict(expert_out=eo[:, :8]),
                dict(expert_out=None), dict(expert_out=None, d_expert_out=eo, d_gate=g), dict(send_pos=pos[:3]),
                dict(rng=rng.float()), dict(d_expert_out=eo[:11]), dict(d_gate=g[:5]), dict(d_shared=dy.bfloat16())):
        with pytest.raises(ValueError):
            moe.moe_combine_dropout_backward(**{**good, **bad})
    for bad in (dict(x=dy.half()), dict(rng=rng[:1]), dict(residual=dy.bfloat16()), dict(residual=dy[:3]),
                dict(y=dy[:3]), dict(y=dy.half())):
        with pytest.raises(ValueError):
            moe.moe_dropout(**{**dict(x=dy, p=0.1, rng=rng, y=dy), **bad})


def test_host_tensors_are_refused():
    dy, rng = torch.zeros(6, 16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_dropout(dy, 0.1, rng)


# ------------------------------------------------------------------------------- the layers

def test_layers_refuse_dropout_without_a_state_and_stay_as_they_were():
    from combine_grouped_gemm_amd.layer import BiasedMoELayer, MoELayer
    N, H, E, k, I = 6, 128, 4, 2, 128
    bf = torch.bfloat16
    layer = MoELayer(N, H, E, k, I, "bf16", torch.zeros(E, 2 * I, H, dtype=bf), torch.zeros(E, H, I, dtype=bf),
                     w_r=torch.zeros(E, H, dtype=bf))
    biased = BiasedMoELayer(N, H, E, k, I, torch.zeros(E, I, H, dtype=bf), torch.zeros(E, H, I, dtype=bf),
                            w_r=torch.zeros(E, H, dtype=bf))
    x, rng = torch.zeros(N, H, dtype=bf), torch.zeros(2, dtype=torch.int64)
    layer.drop_p, layer.keep8, biased.drop_p, biased.saved = 0.125, True, 0.125, True
    for bad in (dict(dropout=-0.1, rng=rng), dict(dropout=1.5, rng=rng), dict(dropout=0.1), dict(dropout=0.1, rng=rng[:1]),
                dict(dropout=0.1, rng=rng.int()), dict(residual=x.float()), dict(residual=x[:5]),
                dict(dropout=0.1, rng=rng.to("meta")), dict(dropout=float("nan"), rng=rng)):
        for lay in (layer, biased):
            with pytest.raises(ValueError):
                lay.forward(x, **bad)
    assert layer.drop_p == 0.125 and layer.keep8 and layer.rng_used is None and biased.drop_p == 0.125 and biased.saved


def test_biased_layer_refusals():
    from combine_grouped_gemm_amd.layer import BiasedMoELayer
    bf = torch.bfloat16
    good = dict(N=6, H=128, E=4, k=2, I=64, w1=torch.zeros(4, 64, 128, dtype=bf), w2=torch.zeros(4, 128, 64, dtype=bf),
                b1=torch.zeros(4, 64), b2=torch.zeros(4, 128, dtype=bf))
    BiasedMoELayer(**good)
    for bad in (dict(act=6), dict(act=-1), dict(gated=True), dict(w1=good["w1"].float()), dict(w2=good["w2"][:, :64]),
                dict(w1=good["w1"].half(), w2=good["w2"].half()), dict(b1=torch.zeros(4, 128)), dict(b2=torch.zeros(4, 128).half()),
                dict(w_r=torch.zeros(4, 128)), dict(bias=torch.zeros(4, dtype=bf))):
        with pytest.raises(ValueError):
            BiasedMoELayer(**{**good, **bad})
    layer = BiasedMoELayer(**good)
    x = torch.zeros(6, 128, dtype=bf)
    with pytest.raises(ValueError, match="logits"):
        layer.forward(x)
    for bad in (dict(x=x[:5]), dict(x=x.float()), dict(z=torch.zeros(6, 5)), dict(z=torch.zeros(6, 4, dtype=bf))):
        with pytest.raises(ValueError):
            layer.forward(**{**dict(x=x, z=torch.zeros(6, 4)), **bad})
    with pytest.raises(ValueError, match="multiples of 128"):
        layer.backward(x, x)
    fits = BiasedMoELayer(6, 128, 4, 2, 128, torch.zeros(4, 128, 128, dtype=bf), torch.zeros(4, 128, 128, dtype=bf))
    with pytest.raises(ValueError, match="save_for_backward"):
        fits.backward(x, x)


@pytest.mark.parametrize("act", sorted(set(oracle.ACTIVATIONS) - {"none"}))
def test_slopes_of_nan_are_nan(act):
    x = np.array([np.nan, 1.0])
    assert np.isnan(oracle.ACTIVATION_SLOPES[act](x)).tolist() == [True, False] and np.isnan(oracle.ACTIVATIONS[act](x[:1])).all()


def test_a_dropped_expert_output_does_not_count_in_the_gates_gradient():
    """y holds nothing of a dropped element's sum, so the gates' gradient takes nothing of what its rows held."""
    rng = np.random.default_rng(8)
    N, k, H = 4, 2, 32
    eo, g, dy = rng.normal(size=(N * k, H)), rng.random((N, k)), rng.normal(size=(N, H))
    pos = np.arange(N * k)
    gone = (oracle.dropout_mask(0.5, 3, 4, N * H) == 0).reshape(N, H).repeat(k, axis=0)
    bad = eo.copy()
    bad[gone] = np.where(rng.random(gone.sum()) < 0.5, np.nan, np.inf)
    assert np.isfinite(oracle.combine_dropout(bad, pos, g, 0.5, 3, 4)).all()
    want, got = (oracle.combine_dropout_backward(dy, pos, g, v, 0.5, 3, 4)[1] for v in (eo, bad))
    assert np.allclose(got, want, rtol=1e-13, atol=0)


def test_a_planted_missing_scale_shows_along_the_gradient():
    """Along a unit direction of a returned gradient the value moves by the gradient's norm; with a mask that does not
    scale (planted here) it moves by 4/3 of it."""
    rng = np.random.default_rng(9)
    N, k, E, H, I = 12, 2, 3, 16, 8
    idx = np.stack([rng.permutation(E)[:k] for _ in range(N)])
    _, off, pos, slot = oracle.dispatch_layout(idx, E)
    x, g, dy = rng.normal(size=(N, H)), rng.random((N, k)), rng.normal(size=(N, H))
    w1, w2, b2 = rng.normal(size=(E, I, H)), rng.normal(size=(E, H, I)), rng.normal(size=(E, H))
    h, _ = oracle.expert_linear(x, off, w1, None, "silu", tokens=slot // k)

    def value(b):
        eo, _ = oracle.expert_linear(h, off, w2, b)
        return (oracle.combine_dropout(eo, pos, g, 0.25, 5, 6) * dy).sum()

    eo, _ = oracle.expert_linear(h, off, w2, b2)
    d_eo, _, _ = oracle.combine_dropout_backward(dy, pos, g, eo, 0.25, 5, 6)
    for scale, ratio in ((1.0, 1.0), (3 / 4, 4 / 3)):
        db = scale * np.stack([d_eo[off[e]:off[e + 1]].sum(axis=0) for e in range(E)])
        norm = np.linalg.norm(db)
        want = (value(b2 + 1e-4 * db / norm) - value(b2 - 1e-4 * db / norm)) / 2e-4
        assert abs(want / norm - ratio) < 1e-7

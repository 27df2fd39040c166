"""GPU parity of the experts' product with bias, activation and residual, and of its activation's and biases' gradients,
with float64 forms."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U32 = 2.0 ** -24
ACT = {"none": 0, "relu": 1, "relu2": 2, "gelu": 3, "gelu_tanh": 4, "silu": 5}
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _return_cached_blocks():
    """The allocator's cached blocks go back afterwards: a test elsewhere counts the bytes it hands out."""
    yield
    torch.cuda.empty_cache()


def _t(shape, seed, dt, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale).to(F32).to(dt)


def _offsets(rows, E, seed):
    """Ragged segments over all rows: some empty, some of one row."""
    rng = np.random.default_rng(seed)
    cut = np.sort(rng.integers(0, rows + 1, E - 1)) if E > 1 else np.zeros(0, int)
    if E > 3 and rows > 3:
        cut[1] = cut[0]
        cut[2] = min(cut[1] + 1, rows)
        cut = np.sort(cut)
    return torch.tensor([0, *cut.tolist(), rows], dtype=torch.int32)


# Phi of values that are rounded to bf16 is a polynomial within 1.2e-5 of the tail (pinned by a test of its
# coefficients against the scaled error function): what it adds to |x| Phi(x) and to the slope's Phi(x)
TAIL = {BF: 1.2e-5, F32: 0.0}


def _act_terms(act, z, ez, dt):
    """(act, its slope, the largest error of act at z + an error below ez, computed in fp32).

    The slope of every activation moves by at most 2 per unit of z (relu2 exactly, the others by less), so
    the product of ez with |slope| + 2 ez covers a moved argument.  An exponential's argument y carries a
    relative 2^-24 for each of its (at most 6) operations and its hardware or library value a few ulp: a
    relative error below (6 |y| + 16) 2^-24 of the sigmoid or of erfc and of what it multiplies; y is the
    argument of the exponential that act contains."""
    f, s = oracle.ACTIVATIONS[act](z), oracle.ACTIVATION_SLOPES[act](z)
    y = {"silu": np.abs(z), "gelu": z * z, "gelu_tanh": 1.6 * np.abs(z) * (1 + 0.05 * z * z)}.get(act, 0 * z)
    tail = TAIL[dt] * np.abs(f) if act == "gelu" else 0.0
    return f, s, (np.abs(s) + 2 * ez) * ez + (6 * y + 16) * U32 * np.abs(f) + tail + 1e-30


def _half_step(dt, v):
    return torch.finfo(dt).eps / 2 * v + (2.0 ** -133 if dt == BF else 2.0 ** -149)


def _linear_reference(a, off, w, bias, act, gated, residual, tokens, dt):
    """(out, its bound before rounding, z, its bound before rounding) in float64."""
    x = f64(a) if tokens is None else f64(a)[tokens]
    rows, K = x.shape
    E, Nw, _ = w.shape
    N = Nw // 2 if gated else Nw
    z, mag = np.full((rows, Nw), np.nan), np.full((rows, Nw), np.nan)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        xe, we = torch.from_numpy(x[r]).to(DEV), w[e].double().to(DEV)   # (64-bit products on the GPU)
        z[r], mag[r] = (xe @ we.T).cpu().numpy(), (xe.abs() @ we.abs().T).cpu().numpy()
        if bias is not None:
            z[r] += f64(bias[e])
            mag[r] += np.abs(f64(bias[e]))
    # an fp32 sum of K products and a bias in any order, doubled for second order
    ez = 2 * (K + 16) * U32 * mag + 1e-37
    f, _, ef = _act_terms(act, z[:, :N], ez[:, :N], dt)
    if gated:
        u, eu = z[:, N:], ez[:, N:]
        out, eo = f * u, ef * (np.abs(u) + eu) + np.abs(f) * eu + U32 * np.abs(f * u)
    else:
        out, eo = f, ef
    if residual is not None:
        eo = eo + U32 * (np.abs(out) + np.abs(f64(residual)) + eo)
        out = out + f64(residual)
    return out, eo, z, ez


def _check(name, got, ref, err, dt, rows=slice(None)):
    got = f64(got)
    lim = err + _half_step(dt, np.abs(ref) + err)
    bad = ~(np.abs(got - ref) <= lim)
    bad[np.isnan(ref)] = False
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / lim)))


def _run_linear(rows, E, K, N, dt, act="silu", gated=False, bias="f32", residual=False, k=0, want_z=True, seed=0,
                offsets=None, dense=False):
    say(f"linear rows={rows} E={E} K={K} N={N} {dt} {act} gated={gated} bias={bias} res={residual} k={k} seed={seed}")
    Nw = 2 * N if gated else N
    off = _offsets(rows, E, seed + 1) if offsets is None else offsets
    w = _t((E, Nw, K), seed + 2, dt, 1 / np.sqrt(K))
    b = None if bias is None else _t((E, Nw), seed + 3, F32 if bias == "f32" else dt, 0.5)
    res = _t((rows, N), seed + 4, dt) if residual else None
    tokens = slot = None
    if k:
        n = max(1, rows // k)
        slot = torch.from_numpy(np.random.default_rng(seed + 5).integers(0, n * k, rows)).to(torch.int32)
        tokens = (slot // k).numpy()
        a = _t((n, K), seed + 6, dt)
    else:
        a = _t((rows, K), seed + 6, dt)
    out = torch.full((rows, N), float("nan"), dtype=dt, device=DEV)
    z = torch.full((rows, Nw), float("nan"), dtype=dt, device=DEV) if want_z else None
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    moe.moe_expert_linear(d(a), d(w), bias=d(b), offsets=None if dense else d(off), act=ACT[act], gated=gated,
                          src_slot=d(slot), k=max(k, 1), residual=d(res), out=out, z=z)
    sync()
    ref, eo, zr, ez = _linear_reference(a, off, w, b, act, gated, res, tokens, dt)
    _check("out", out, ref, eo, dt)
    if want_z:
        _check("z", z, zr, ez, dt)
    # rows of no expert stay as they were
    gap = np.isnan(zr[:, 0])
    assert np.isnan(f64(out)[gap]).all()
    return out


SIZES = [(1, 1, 8, 8), (1, 8, 64, 264), (2, 3, 72, 40), (7, 2, 136, 8), (16, 1, 4104, 64), (17, 5, 24, 136), (31, 8, 256, 128),
         (33, 1, 520, 1016), (64, 64, 64, 72), (65, 4, 200, 264), (129, 3, 1000, 136), (257, 2, 64, 520), (300, 40, 96, 328),
         (700, 5, 264, 264), (1100, 2, 128, 1032), (130, 1024, 16, 24), (520, 1, 1032, 2056)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,E,K,N", SIZES)
def test_sizes(rows, E, K, N, gated, dt):
    _run_linear(rows, E, K, N, dt, gated=gated, seed=rows)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,E,K,Nw,k,dt", [
    # 320 x 256 tiles: whole ones, ragged experts of every row-block count, one column block more than whole
    (4000, 1, 2048, 2304, 0, BF), (5000, 8, 1032, 4112, 0, BF), (4100, 1, 1032, 4112, 3, BF),
    # 128 x 256 tiles, alone and with K in parts
    (3000, 1, 1024, 2304, 0, BF), (1100, 4, 1032, 4112, 2, BF), (512, 1, 14336, 4096, 0, BF),
    # K in parts under 320 x 256 tiles
    (1024, 1, 14336, 4096, 0, BF), (900, 2, 14336, 4112, 2, BF),
    # 64 x 64 tiles with K in 4, 8 and 16 parts; a last part of one partial stage
    (600, 1, 8200, 1040, 0, BF), (64, 1, 4104, 272, 2, BF), (33, 1, 3336, 48, 0, BF),
    # fp32: 128 x 128 tiles, alone and with K in parts; 32 x 64 ones, alone and with K in parts
    (3000, 4, 520, 2064, 0, F32), (512, 1, 4096, 4096, 0, F32), (700, 3, 264, 2064, 2, F32), (1000, 1, 14336, 1040, 0, F32),
    (200, 1, 4104, 528, 2, F32), (33, 1, 3336, 48, 0, F32)])
def test_every_kernel(rows, E, K, Nw, k, dt, gated):
    """Sizes that take each of the tile kernels, with residual, kept z and a gated or plain epilogue."""
    _run_linear(rows, E, K, Nw // 2 if gated else Nw, dt, "gelu" if gated else "silu", gated, "f32", True, k, seed=rows)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,E,K,Nw,k,dt", [
    # 16 weight rows by eight waves (up to 128 groups of 32 weight rows): up to 16 and up to 32 rows of a at a time
    (16, 1, 8200, 2064, 0, BF), (31, 1, 8200, 2064, 2, BF), (57, 5, 1032, 400, 0, BF), (29, 1, 2056, 2064, 0, F32),
    # 32 by four
    (1, 1, 14336, 4112, 0, BF), (32, 1, 4096, 4112, 3, BF), (57, 5, 1032, 1040, 0, BF), (3, 9, 4104, 2064, 2, BF),
    (1, 1, 4096, 4112, 0, F32), (45, 3, 2056, 4112, 2, F32)])
def test_few_rows(rows, E, K, Nw, k, dt, gated):
    """Few rows an expert: either shape of the kernel that streams the weights, K that ends inside a stage."""
    _run_linear(rows, E, K, Nw // 2 if gated else Nw, dt, "gelu_tanh" if gated else "silu", gated, "f32", True, k, seed=rows)


def test_few_rows_of_one_expert():
    """All rows on one of many experts: 32 at a time, the last of them fewer."""
    off = torch.tensor([0, 0, 0, 117, 117, 117, 117, 117, 117], dtype=torch.int32)
    for dt in (BF, F32):
        _run_linear(117, 8, 1032, 528, dt, "gelu", False, "f32", True, seed=117, offsets=off)


def test_operands_past_32_bits():
    """Rows of a and of out whose byte offsets pass 2^32."""
    rows, n = 300000, 40
    for K, N in ((8200, 8), (8, 8200)):
        say(f"linear rows={rows} K={K} N={N}")
        a, w = torch.randn(rows, K, device=DEV, dtype=BF), torch.randn(2, N, K, device=DEV, dtype=BF)
        off = torch.tensor([0, rows - 100, rows], dtype=torch.int32, device=DEV)
        out, _ = moe.moe_expert_linear(a, w, offsets=off, act=ACT["relu"])
        few, _ = moe.moe_expert_linear(a[-n:], w[1:], act=ACT["relu"])
        sync()
        # other tiles sum K in another order: two fp32 sums of K products each, then a rounding each
        x64, w64 = a[-n:].double(), w[1].double()
        err = 4 * (K + 16) * U32 * (x64.abs() @ w64.abs().T) + 2 * 2.0 ** -8 * few.double().abs()
        assert ((out[-n:].double() - few.double()).abs() <= err).all()
        del a, out
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", sorted(ACT))
def test_activations(act, gated, dt):
    _run_linear(70, 3, 48, 72, dt, act=act, gated=gated, residual=True, seed=1)
    _run_linear(5, 2, 4096, 32, dt, act=act, gated=gated, bias="dt", seed=2)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,E,K,N,k", [(1, 4, 64, 72, 1), (2, 8, 512, 264, 2), (40, 8, 136, 136, 4), (333, 6, 520, 264, 3),
                                          (1500, 4, 72, 264, 2)])
def test_gathered(rows, E, K, N, k, dt):
    for gated, res, bias in ((False, True, "dt"), (True, False, None)):
        _run_linear(rows, E, K, N, dt, "gelu", gated, bias, res, k, seed=3)


@pytest.mark.parametrize("dt", [F32, BF])
def test_without_offsets_bias_or_kept_z(dt):
    for rows in (1, 3, 50, 400):
        _run_linear(rows, 1, 264, 520, dt, "none", bias=None, want_z=False, residual=True, dense=True, seed=4)
        _run_linear(rows, 1, 264, 520, dt, "relu", bias="f32", dense=True, seed=5)


@pytest.mark.parametrize("dt", [F32, BF])
def test_rows_outside_the_experts_stay(dt):
    """Rows before the first and behind the last expert, and experts without rows at either end."""
    for off in ([3, 3, 9, 9, 20], [0, 0, 0, 0, 0], [0, 40, 40, 41, 41], [5, 5, 5, 5, 6]):
        _run_linear(41, 4, 72, 40, dt, seed=6, offsets=torch.tensor(off, dtype=torch.int32))


def test_offsets_out_of_range_are_clamped():
    """Offsets past the rows are clamped: nothing outside the arrays is touched."""
    a, w = _t((30, 64), 1, BF).to(DEV), _t((2, 64, 64), 2, BF, 0.1).to(DEV)
    ref, _ = moe.moe_expert_linear(a, w, offsets=torch.tensor([0, 12, 30], dtype=torch.int32, device=DEV))
    got, _ = moe.moe_expert_linear(a, w, offsets=torch.tensor([-7, 12, 4000], dtype=torch.int32, device=DEV))
    sync()
    assert torch.equal(ref, got)
    slot = torch.tensor([-5, 10 ** 9] + list(range(28)), dtype=torch.int32, device=DEV)
    got, _ = moe.moe_expert_linear(a, w, offsets=torch.tensor([0, 12, 30], dtype=torch.int32, device=DEV), src_slot=slot)
    want, _ = moe.moe_expert_linear(a[torch.tensor([0, 29] + list(range(28)), device=DEV)].contiguous(), w,
                                    offsets=torch.tensor([0, 12, 30], dtype=torch.int32, device=DEV))
    sync()
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_not_finite_values_stay_in_their_rows(rows):
    """A NaN or infinity in a row of a reaches that row alone; one in a weight row that column of that expert."""
    a, w = _t((rows, 136), 1, BF), _t((2, 72, 136), 2, BF, 0.1)
    off = torch.tensor([0, rows - 1, rows], dtype=torch.int32)
    clean, _ = moe.moe_expert_linear(a.to(DEV), w.to(DEV), offsets=off.to(DEV))
    a[1, 135] = float("nan")
    w[1, 40, 0] = float("inf")
    got, _ = moe.moe_expert_linear(a.to(DEV), w.to(DEV), offsets=off.to(DEV))
    sync()
    clean, got = clean.cpu(), got.cpu()
    bad = torch.zeros(rows, 72, dtype=torch.bool)
    bad[1] = True
    bad[rows - 1, 40] = True
    assert not torch.isfinite(got[bad]).any() and torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,E", [(2, 2), (50, 3), (600, 3)])
def test_in_place_residual_repeats_and_workspace(rows, E, dt):
    """out may be residual; the same inputs give the same bits with other work between; a workspace that held
    anything serves."""
    a, w, res = _t((rows, 1032), 1, dt).to(DEV), _t((E, 264, 1032), 2, dt, 0.03).to(DEV), _t((rows, 264), 3, dt).to(DEV)
    off = _offsets(rows, E, 4).to(DEV)
    want, _ = moe.moe_expert_linear(a, w, offsets=off, residual=res)
    other, _ = moe.moe_expert_linear(a + 1, w, offsets=off, residual=res)
    ws = torch.full((max(moe.moe_workspace_bytes(moe.MOE_OP_EXPERT_LINEAR, rows, 1032, 264, E, 0, moe._dt(a)), 16),), 255,
                    dtype=torch.uint8, device=DEV)
    again, _ = moe.moe_expert_linear(a, w, offsets=off, residual=res, ws=ws)
    buf = res.clone()
    moe.moe_expert_linear(a, w, offsets=off, residual=buf, out=buf)
    sync()
    assert torch.equal(want, again) and torch.equal(want, buf) and not torch.equal(want, other)


def test_no_rows():
    w = _t((3, 64, 32), 1, BF).to(DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    out, z = moe.moe_expert_linear(torch.empty(0, 32, dtype=BF, device=DEV), w, offsets=off, want_z=True)
    assert out.shape == (0, 64) and z.shape == (0, 64)
    dz, db, h = moe.moe_expert_act_backward(out, z=z, offsets=off, act=ACT["silu"], want_h=True,
                                            db=torch.full((3, 64), 7.0, device=DEV))
    sync()
    assert dz.shape == (0, 64) and not db.any()


@pytest.mark.parametrize("rows,K,N", [(4, 64, 72), (300, 136, 264), (700, 136, 264)])
def test_other_stream_and_captured(rows, K, N):
    """On a second stream, and captured and replayed on new inputs with eager work between."""
    a, w, off = _t((rows, K), 1, BF).to(DEV), _t((2, N, K), 2, BF, 0.1).to(DEV), _offsets(rows, 2, 3).to(DEV)
    b = _t((2, N), 4, F32).to(DEV)
    d = _t((rows, N), 5, BF).to(DEV)
    kw = dict(bias=b, offsets=off, act=ACT["gelu_tanh"])
    ws = torch.empty(max(moe.moe_workspace_bytes(moe.MOE_OP_EXPERT_LINEAR, rows, K, N, 2, 0, moe.MOE_BF16), 256),
                     dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(moe.moe_workspace_bytes(moe.MOE_OP_ACT_BACKWARD, rows, 0, N, 2, 0, 0), dtype=torch.uint8, device=DEV)
    want = moe.moe_expert_linear(a, w, want_z=True, **kw)
    sync()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.moe_expert_linear(a, w, want_z=True, **kw)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, z = want[0].clone(), want[1].clone()
    dz, db, h = moe.moe_expert_act_backward(d, z=z, offsets=off, act=ACT["gelu_tanh"], want_h=True)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_expert_linear(a, w, out=out, z=z, ws=ws, **kw)
        moe.moe_expert_act_backward(d, z=z, offsets=off, act=ACT["gelu_tanh"], dz=dz, db=db, h=h, ws=ws2)
    for _ in range(3):
        a.normal_()
        d.normal_()
        ws.fill_(255)
        ws2.fill_(255)
        graph.replay()
        sync()
        o2, z2 = moe.moe_expert_linear(a, w, want_z=True, **kw)
        r2 = moe.moe_expert_act_backward(d, z=z2, offsets=off, act=ACT["gelu_tanh"], want_h=True)
        sync()
        assert torch.equal(out, o2) and torch.equal(z, z2)
        assert all(torch.equal(x, y) for x, y in zip((dz, db, h), r2))


# ------------------------------------------------------------------------------- the activation's gradient

def _run_act(rows, E, N, dt, act, gated, seed=0, db_dtype=F32, offsets=None):
    say(f"act backward rows={rows} E={E} N={N} {dt} {act} gated={gated} db={db_dtype}")
    Nw = 2 * N if gated else N
    off = _offsets(rows, E, seed + 1) if offsets is None else offsets
    z, d = _t((rows, Nw), seed + 2, dt, 2.0), _t((rows, N), seed + 3, dt)
    nan = lambda c: torch.full((rows, c), float("nan"), dtype=dt, device=DEV)  # noqa: E731
    dz, h = nan(Nw), nan(N)
    _, db, _ = moe.moe_expert_act_backward(d.to(DEV), z=z.to(DEV), offsets=off.to(DEV), act=ACT[act], gated=gated, dz=dz,
                                           h=h, db=torch.full((E, Nw), float("nan"), dtype=db_dtype, device=DEV))
    sync()
    zz, dd = f64(z), f64(d)
    rz, rb, rh = oracle.expert_act_backward(zz, dd, off.tolist(), act, gated)
    f, s, ef = _act_terms(act, zz[:, :N], 0.0 * zz[:, :N], dt)
    # the slope: an exponential of argument y as above, times factors up to 1 + |y| + 2.4 z^2 in the tails
    g = zz[:, :N]
    y = {"silu": np.abs(g), "gelu": g * g, "gelu_tanh": 1.6 * np.abs(g) * (1 + 0.05 * g * g)}.get(act, 0 * g)
    sg = {"silu": 1 / (1 + np.exp(-g)), "gelu": np.abs(oracle.ACTIVATIONS["gelu"](g) / np.where(g == 0, 1, g)) + np.exp(-g * g / 2),
          "gelu_tanh": 1 / (1 + np.exp(-1.5957691 * (g + 0.044715 * g ** 3)))}.get(act, np.abs(s))
    # a logistic value or an exponential below 2^-126 is 0 on the GPU (the exponential in its denominator passes
    # 2^128, or the reciprocal's result is subnormal), so sg is off by up to 2^-126 there
    es = (((6 * y + 24) * U32 + (TAIL[dt] if act == "gelu" else 0.0)) * sg + 2.0 ** -126) * (1 + y + np.abs(g) * 1.6 * (1 + 0.15 * g * g))
    u = np.abs(zz[:, N:]) if gated else 1.0
    e1 = (es + 3 * U32 * np.abs(s)) * np.abs(dd) * u
    ez = np.concatenate([e1, np.abs(dd) * (ef + 2 * U32 * np.abs(f))], axis=1) if gated else e1
    inside = np.zeros(rows, bool)
    for e in range(E):
        inside[int(off[e]):int(off[e + 1])] = True
    rz2, rh2 = np.where(inside[:, None], rz, np.nan), np.where(inside[:, None], rh, np.nan)
    _check("dz", dz, rz2, ez, dt)
    _check("h", h, rh2, ef * u + 2 * U32 * np.abs(rh), dt)
    assert np.isnan(f64(dz)[~inside]).all() and np.isnan(f64(h)[~inside]).all()
    off = off.tolist()
    eb = np.stack([ez[off[e]:off[e + 1]].sum(axis=0) + 2 * (off[e + 1] - off[e] + 8) * U32 * np.abs(
        rz[off[e]:off[e + 1]]).sum(axis=0) for e in range(E)])
    _check("db", db, rb, eb, db_dtype)
    # each output alone gives the same bits
    kw = dict(z=z.to(DEV), offsets=torch.tensor(off, dtype=torch.int32, device=DEV), act=ACT[act], gated=gated)
    one = moe.moe_expert_act_backward(d.to(DEV), want_dz=False, db_dtype=db_dtype, **kw)
    two = moe.moe_expert_act_backward(d.to(DEV), want_db=False, **kw)
    sync()
    assert one[0] is None and torch.equal(one[1], db) and two[1] is None
    assert torch.equal(two[0][torch.from_numpy(inside)], dz[torch.from_numpy(inside)])


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", sorted(ACT))
def test_act_backward(act, gated, dt):
    _run_act(60, 4, 40, dt, act, gated)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,E,N", [(1, 1, 8), (1, 5, 1032), (3, 1, 520), (40, 40, 72), (257, 3, 136), (301, 1024, 16),
                                      (2000, 6, 264), (5000, 1, 8), (4100, 2, 4104), (9000, 30, 512),
                                      # one launch: 129 and 512 rows of few experts, its largest row and most workgroups
                                      (129, 2, 72), (512, 1, 2048), (512, 7, 40), (64, 1, 16392), (300, 19, 1032),
                                      # two: one row, one expert, some columns more
                                      (513, 7, 40), (300, 20, 1032), (512, 1, 4104)])
def test_act_backward_sizes(rows, E, N, dt):
    _run_act(rows, E, N, dt, "silu", True, seed=rows)
    _run_act(rows, E, N, dt, "gelu_tanh", False, seed=rows, db_dtype=BF)


def test_act_backward_rows_outside_the_experts():
    for off in ([3, 3, 9, 9, 20], [0, 0, 0, 0, 0], [0, 40, 40, 41, 41], [5, 5, 5, 5, 6]):
        _run_act(41, 4, 40, BF, "silu", True, offsets=torch.tensor(off, dtype=torch.int32))


@pytest.mark.parametrize("dt", [F32, BF])
def test_bias_gradient_alone(dt):
    """The bias gradient of a product without activation: z is not needed, dz is d_out."""
    for rows, E, N in ((1, 1, 8), (37, 3, 264), (3000, 7, 520)):
        say(f"bias gradient rows={rows} E={E} N={N} {dt}")
        off, d = _offsets(rows, E, 2), _t((rows, N), 3, dt)
        dz, db, h = moe.moe_expert_act_backward(d.to(DEV), offsets=off.to(DEV))
        sync()
        off = off.tolist()
        ref = np.stack([f64(d)[off[e]:off[e + 1]].sum(axis=0) for e in range(E)])
        mag = np.stack([np.abs(f64(d))[off[e]:off[e + 1]].sum(axis=0) for e in range(E)])
        assert h is None and torch.equal(dz.cpu(), d)
        assert np.all(np.abs(f64(db) - ref) <= (rows + 8) * U32 * mag)


def test_relu_at_zero_and_special_values():
    """Slope 0 at 0 and -0; a NaN pre-activation keeps to its element and its column's sum."""
    z = torch.tensor([[0.0, -0.0, 1.0, -1.0, float("nan"), float("inf"), float("-inf"), 2.0]], device=DEV)
    d = torch.ones(1, 8, device=DEV)
    dz, db, h = moe.moe_expert_act_backward(d, z=z, act=ACT["relu"], want_h=True)
    dz2, _, _ = moe.moe_expert_act_backward(d, z=z, act=ACT["relu2"])
    sync()
    assert dz[0].tolist()[:4] == [0, 0, 1, 0] and dz[0, 5] == 1 and dz[0, 6] == 0 and db[0, 7] == 1
    assert h[0].tolist()[:4] == [0, 0, 1, 0] and torch.isnan(h[0, 4]) and h[0, 5] == float("inf") and h[0, 6] == 0
    assert dz2[0].tolist()[:4] == [0, 0, 2, 0]


def test_bias_gradient_of_many_rows():
    """300000 rows of ones: every partial sum on the way counts."""
    d = torch.ones(300000, 16, dtype=BF, device=DEV)
    off = torch.tensor([0, 1, 200001, 200001, 300000], dtype=torch.int32, device=DEV)
    _, db, _ = moe.moe_expert_act_backward(d, offsets=off, want_dz=False)
    sync()
    assert [db[e].unique().tolist() for e in range(4)] == [[1.0], [200000.0], [0.0], [99999.0]]


@pytest.mark.parametrize("gated", [False, True])
def test_act_backward_of_large_calls(gated):
    """From 256 MB on dz and h are stored past the caches: the same bits as for a few rows at a time."""
    rows, N = (17000, 4104) if gated else (34000, 4104)
    say(f"act backward of large calls gated={gated}")
    z = torch.randn(rows, 2 * N if gated else N, device=DEV).to(BF)
    d = torch.randn(rows, N, device=DEV).to(BF)
    off = torch.tensor([0, 5000, rows], dtype=torch.int32, device=DEV)
    kw = dict(act=ACT["silu"], gated=gated, want_h=True)
    dz, db, h = moe.moe_expert_act_backward(d, z=z, offsets=off, **kw)
    sync()
    sums = torch.zeros(2, z.shape[1], dtype=torch.float64, device=DEV)
    for a in range(0, rows, 1000):
        dz1, db1, h1 = moe.moe_expert_act_backward(d[a:a + 1000], z=z[a:a + 1000], **kw)
        sync()
        assert torch.equal(dz1, dz[a:a + 1000]) and torch.equal(h1, h[a:a + 1000])
        sums[int(a >= 5000)] += db1[0].double()
    mag = torch.stack([dz[:5000].abs().double().sum(dim=0), dz[5000:].abs().double().sum(dim=0)])
    # two fp32 sums of the same values in other orders: at most rows + 8 roundings of the magnitudes' sum each
    assert ((db.double() - sums).abs() <= 2 * (rows + 8) * U32 * mag).all()


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("act", sorted(set(ACT) - {"none"}))
def test_a_nan_pre_activation_reaches_dz_db_and_h(act, rows, dt):
    """A NaN in z is not hidden by the slope: its element of dz and h and its column of its expert's db are NaN, nothing
    else is."""
    z, d = _t((rows, 24), 1, dt), torch.ones(rows, 24, dtype=dt)
    z[rows - 1, 5] = float("nan")
    off = torch.tensor([0, rows - 1, rows], dtype=torch.int32)
    dz, db, h = moe.moe_expert_act_backward(d.to(DEV), z=z.to(DEV), offsets=off.to(DEV), act=ACT[act], want_h=True)
    sync()
    at = torch.zeros(rows, 24, dtype=torch.bool)
    at[rows - 1, 5] = True
    assert torch.equal(torch.isnan(dz).cpu(), at) and torch.equal(torch.isnan(h).cpu(), at)
    assert torch.isnan(db).nonzero().tolist() == [[1, 5]]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_large_finite_pre_activations(act, dt):
    """Far from 0 these activations are x or 0 and their slopes 1 or 0, also where a power of x passes 2^128."""
    v = torch.tensor([100.0, 1e10, 3e13, 2e19, 3e38, -100.0, -1e10, -3e13, -2e19, -3e38, 1e25, -1e25, 1e37, -1e37, 50.0, -50.0])
    z, d = v.to(dt).reshape(1, 16).to(DEV), torch.full((1, 16), 0.5, dtype=dt, device=DEV)
    dz, db, h = moe.moe_expert_act_backward(d, z=z, act=ACT[act], want_h=True)
    u = torch.ones(1, 16, dtype=dt, device=DEV)
    gz, gb, gh = moe.moe_expert_act_backward(d, z=torch.cat([z, u], dim=1), act=ACT[act], gated=True, want_h=True)
    a = torch.zeros(1, 16, dtype=dt, device=DEV)
    a[0, 0] = 1
    w = torch.zeros(1, 16, 16, dtype=dt, device=DEV)
    w[0, :, 0] = z[0]
    out, _ = moe.moe_expert_linear(a, w, act=ACT[act])
    sync()
    up = (v > 0).reshape(1, 16)
    for got in (dz, db, gz[:, :16], gb[:, :16]):    # 50 below 0 act is below 1e-19, its slope below 1e-17
        assert ((got.cpu().double() - 0.5 * up).abs() <= 1e-17).all()
    for got in (h, gh, out, gz[:, 16:].double() * 2):
        assert torch.equal(got.cpu().double()[up], z.cpu().double()[up]) and (got.cpu().double()[~up].abs() < 1e-19).all()


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,E,N,gated", [(3, 1, 8, False), (300, 4, 520, True), (300, 4, 520, False), (5000, 6, 264, True),
                                            (70000, 3, 2056, False)])
def test_act_backward_in_place(rows, E, N, gated, dt):
    """dz may be z, and h d_out."""
    off = _offsets(rows, E, 3).to(DEV)
    z, d = _t((rows, 2 * N if gated else N), 1, dt).to(DEV), _t((rows, N), 2, dt).to(DEV)
    kw = dict(offsets=off, act=ACT["gelu"], gated=gated)
    want = moe.moe_expert_act_backward(d, z=z, want_h=True, **kw)
    got = moe.moe_expert_act_backward(d, z=z, dz=z, h=d, **kw)
    sync()
    assert got[0] is z and got[2] is d and all(torch.equal(a, b) for a, b in zip(want, got))

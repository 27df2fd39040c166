"""GPU parity of combine with dropout and residual, its gradient, and dropout of rows, with the oracle's float64 forms and
its generator in Python integers."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U32 = 2.0 ** -24
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _return_cached_blocks():
    """The allocator's cached blocks go back afterwards: a test elsewhere counts the bytes it hands out."""
    yield
    torch.cuda.empty_cache()


def _t(shape, seed, dt, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale).to(F32).to(dt)


def _state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


def _pos(N, k, rows, seed, drop=True):
    rng = np.random.default_rng(seed)
    p = rng.permutation(rows)[:N * k]
    if drop and N * k > 3:
        p[rng.integers(0, N * k, max(1, N * k // 9))] = -1
    return torch.from_numpy(p).to(torch.int32)


def _half(dt, v):
    return torch.finfo(dt).eps / 2 * v + (2.0 ** -133 if dt == BF else 2.0 ** -149)


# p = 2^-16 / 2 + a little: the smallest that drops at all; rounding up to 1 drops everything
PS = [0.0, 0.1, 0.5, 0.9, 1.0, 0.8e-5, 1 - 0.7e-5]
SEEDS = [(0, 0), (1, 2), (-1, -1), (2 ** 40 + 5, 2 ** 33 + 9), (-2 ** 62, 77)]


@pytest.mark.parametrize("N,k,H,dt,ydt,shared,res,gated", [
    (1, 1, 8, BF, BF, False, False, True), (1, 2, 4096, BF, F32, True, True, True), (3, 3, 1032, F32, F32, False, True, True),
    (17, 8, 264, BF, BF, True, True, True), (16, 2, 72, F32, BF, True, False, False), (5, 9, 136, BF, BF, False, True, True),
    (9, 32, 40, F32, F32, True, True, True), (40, 4, 2056, BF, F32, False, False, False), (1200, 2, 16, BF, BF, True, True, True),
    (1030, 5, 24, F32, F32, False, True, True)])
def test_combine_dropout(N, k, H, dt, ydt, shared, res, gated):
    for i, p in enumerate(PS):
        seed, off = SEEDS[i % len(SEEDS)]
        say(f"combine dropout N={N} k={k} H={H} {dt} {ydt} p={p}")
        rows = N * k + 3
        eo, g = _t((rows, H), 1, dt), torch.softmax(_t((N, k), 2, F32), dim=1)
        pos = _pos(N, k, rows, 3)
        sh, r = (_t((N, H), 4, dt) if shared else None), (_t((N, H), 5, ydt) if res else None)
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        y = moe.moe_combine_dropout(d(eo), d(pos), d(g) if gated else None, p, _state(seed, off), shared_out=d(sh),
                                    residual=d(r), y_dtype=ydt, k=None if gated else k)
        sync()
        gg = f64(g) if gated else np.ones((N, k))
        args = [f64(eo), pos.numpy(), gg, p, seed, off]
        ref = oracle.combine_dropout(*args, None if sh is None else f64(sh), None if r is None else f64(r))
        mag = oracle.combine_dropout(np.abs(args[0]), args[1], gg, p, seed, off, None if sh is None else np.abs(f64(sh)),
                                     None if r is None else np.abs(f64(r)))
        # k products and k + 2 sums of at most mag each, the scale's own rounding and its product
        err = (k + 5) * U32 * mag * 1.01
        assert y.dtype == ydt and np.all(np.abs(f64(y) - ref) <= err + _half(ydt, np.abs(ref) + err))
        if r is not None:   # what is dropped leaves the residual digit for digit
            gone = oracle.dropout_mask(p, seed, off, N * H).reshape(N, H) == 0
            assert np.array_equal(f64(y)[gone], f64(r)[gone])


@pytest.mark.parametrize("N,k,H,dt,dydt,gated", [
    (1, 1, 8, BF, BF, True), (1, 2, 4096, BF, F32, True), (3, 3, 1032, F32, F32, True), (17, 8, 264, BF, BF, True),
    (16, 2, 72, F32, F32, False), (5, 9, 136, BF, BF, True), (9, 32, 40, F32, F32, True), (40, 4, 2056, BF, F32, False),
    (1200, 2, 16, BF, BF, True), (2, 7, 16392, BF, BF, True)])
def test_combine_dropout_backward(N, k, H, dt, dydt, gated):
    for i, p in enumerate(PS[:5]):
        seed, off = SEEDS[i % len(SEEDS)]
        say(f"combine dropout backward N={N} k={k} H={H} {dt} {dydt} p={p}")
        rows = N * k + 3
        eo, dy, g = _t((rows, H), 1, dt), _t((N, H), 2, dydt), torch.softmax(_t((N, k), 3, F32), dim=1)
        pos = _pos(N, k, rows, 4)
        keep = torch.full((rows, H), 7.0, dtype=dt, device=DEV)
        d_eo, dg, dsh = moe.moe_combine_dropout_backward(
            dy.to(DEV), pos.to(DEV), g.to(DEV) if gated else None, eo.to(DEV), p, _state(seed, off), d_expert_out=keep,
            d_gate=torch.full((N, k), float("nan"), device=DEV), want_shared=True, k=None if gated else k)
        sync()
        gg = f64(g) if gated else np.ones((N, k))
        r_eo, r_g, r_sh = oracle.combine_dropout_backward(f64(dy), pos.numpy(), gg, f64(eo), p, seed, off)
        _, mag, _ = oracle.combine_dropout_backward(np.abs(f64(dy)), pos.numpy(), gg, np.abs(f64(eo)), p, seed, off)
        named = ~np.isnan(r_eo[:, 0])
        e = 4 * U32 * np.abs(r_eo[named])
        assert np.all(np.abs(f64(d_eo)[named] - r_eo[named]) <= e + _half(dt, np.abs(r_eo[named]) + e))
        assert np.all(f64(d_eo)[~named] == 7.0)
        assert np.all(np.abs(f64(dg) - r_g) <= (H + 8) * U32 * mag)
        e = 3 * U32 * np.abs(r_sh)
        assert np.all(np.abs(f64(dsh) - r_sh) <= e + _half(dt, np.abs(r_sh) + e))
        # without the expert outputs: the same rows, no gate gradient
        again, none, _ = moe.moe_combine_dropout_backward(
            dy.to(DEV), pos.to(DEV), g.to(DEV) if gated else None, None, p, _state(seed, off),
            d_expert_out=torch.full((rows, H), 7.0, dtype=dt, device=DEV), k=k)
        sync()
        assert none is None and torch.equal(again, d_eo)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2047, 2048, 2055, 40001])
@pytest.mark.parametrize("dt,ydt", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
def test_dropout_rows(n, dt, ydt):
    for i, p in enumerate(PS):
        seed, off = SEEDS[i % len(SEEDS)]
        x, r = _t((n,), 1, dt), _t((n,), 2, ydt)
        y = moe.moe_dropout(x.to(DEV), p, _state(seed, off), y_dtype=ydt)
        z = moe.moe_dropout(x.to(DEV), p, _state(seed, off), residual=r.to(DEV))
        sync()
        m = oracle.dropout_mask(p, seed, off, n)
        ref = f64(x) * m
        e = 2 * U32 * np.abs(ref)
        assert np.all(np.abs(f64(y) - ref) <= e + _half(ydt, np.abs(ref) + e))
        tot = ref + f64(r)
        e = 2 * U32 * np.abs(ref) + U32 * (np.abs(tot) + np.abs(ref))
        assert np.all(np.abs(f64(z) - tot) <= e + _half(ydt, np.abs(tot) + e))


def test_slots_without_a_row():
    """Slots whose row lies outside the expert outputs are skipped, in either direction; with no rows at all y is the
    residual alone."""
    N, k, H = 40, 3, 72
    eo, g, res, dy = (_t(s, i, BF).to(DEV) for i, s in enumerate(((N * k, H), (N, k), (N, H), (N, H))))
    g = g.float()
    pos = torch.arange(N * k, dtype=torch.int32, device=DEV)
    bad = pos.clone()
    bad[::7], bad[3::7], bad[5::7] = N * k, 2 ** 31 - 1, -2 ** 31
    none = torch.where(bad == pos, pos, torch.full_like(pos, -1))
    rng = _state(2, 3)
    a, b = (moe.moe_combine_dropout(eo, q, g, 0.2, rng, residual=res) for q in (bad, none))
    ga, gb = (moe.moe_combine_dropout_backward(dy, q, g, eo, 0.2, rng, d_expert_out=torch.zeros_like(eo)) for q in (bad, none))
    alone = moe.moe_combine_dropout(eo[:0], torch.full_like(pos, -1), g, 0.2, rng, residual=res)
    _, dg, dsh = moe.moe_combine_dropout_backward(dy, pos, g, eo[:0], 0.2, rng, want_shared=True)
    sync()
    assert torch.equal(a, b) and torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1]) and torch.equal(alone, res)
    assert not dg.any() and torch.equal(dsh, moe.moe_dropout(dy, 0.2, rng))


def test_dropped_infinities_and_nan_are_gone():
    x = torch.full((4096,), float("inf"), device=DEV)
    x[::2] = float("nan")
    y = moe.moe_dropout(x, 0.5, _state(3, 4))
    all_gone = moe.moe_dropout(x, 1.0, _state(3, 4))
    sync()
    gone = torch.from_numpy(oracle.dropout_mask(0.5, 3, 4, 4096) == 0)
    y = y.cpu()
    assert (y[gone] == 0).all() and not torch.isfinite(y[~gone]).any() and not all_gone.any()
    # rows of experts and gradients alike
    N, k, H = 8, 2, 64
    eo = torch.full((N * k, H), float("nan"), device=DEV)
    pos = torch.arange(N * k, dtype=torch.int32, device=DEV)
    out = moe.moe_combine_dropout(eo, pos, None, 0.5, _state(3, 4), k=k)
    d_eo, _, d_sh = moe.moe_combine_dropout_backward(torch.full((N, H), float("nan"), device=DEV), pos, None, None, 0.5,
                                                     _state(3, 4), d_expert_out=eo, want_shared=True, k=k)
    sync()
    gone = torch.from_numpy(oracle.dropout_mask(0.5, 3, 4, N * H) == 0).reshape(N, H)
    assert (out.cpu()[gone] == 0).all() and (d_sh.cpu()[gone] == 0).all()
    assert (d_eo.cpu()[gone.repeat_interleave(k, dim=0)] == 0).all()


def test_in_place():
    x, r, rng = _t((999,), 1, BF).to(DEV), _t((999,), 2, BF).to(DEV), _state(5, 6)
    want = moe.moe_dropout(x, 0.3, rng, residual=r)
    a, b = r.clone(), x.clone()
    moe.moe_dropout(x, 0.3, rng, residual=a, y=a)
    moe.moe_dropout(b, 0.3, rng, residual=r, y=b)
    eo, pos, g = _t((12, 40), 3, BF).to(DEV), torch.arange(12, dtype=torch.int32, device=DEV), torch.ones(6, 2, device=DEV)
    res = _t((6, 40), 4, BF).to(DEV)
    w2 = moe.moe_combine_dropout(eo, pos, g, 0.3, rng, residual=res)
    moe.moe_combine_dropout(eo, pos, g, 0.3, rng, residual=res, y=res)
    sync()
    assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(res, w2)


def test_forward_and_backward_agree_and_offsets_differ():
    """The gradient of dropout is dropout of the gradient: the same elements stay."""
    rng = _state(9, 1)
    x = torch.ones(100000, device=DEV)
    y, dy = moe.moe_dropout(x, 0.2, rng), moe.moe_dropout(2 * x, 0.2, rng)
    rng[1] += 1
    z = moe.moe_dropout(x, 0.2, rng)
    sync()
    assert torch.equal(dy, 2 * y) and not torch.equal(y, z)
    # 100000 draws each: the share dropped, and the share dropped in both, within 5 standard deviations
    for share, p in (((y == 0).float().mean(), 0.2), (((y == 0) & (z == 0)).float().mean(), 0.04)):
        assert abs(share.item() - p) < 5 * (p * (1 - p) / 100000) ** 0.5


def test_far_counters():
    """Elements past 2^32 of a batch take the counter's high word."""
    n = 2 ** 32 + 4096
    x = torch.ones(n, dtype=BF, device=DEV)
    moe.moe_dropout(x, 0.5, _state(1, 2), y=x)
    sync()
    tail, head = x[n - 64:].cpu(), x[:64].cpu()
    del x
    torch.cuda.empty_cache()
    words = [w for i in range(n // 8 - 8, n // 8) for w in oracle.philox((i & 0xFFFFFFFF, i >> 32, 2, 0), (1, 0))]
    num = np.array([v for w in words for v in (w & 0xFFFF, w >> 16)])
    assert np.array_equal(f64(tail) != 0, num >= 32768)
    assert np.array_equal(f64(head) != 0, oracle.dropout_numbers(1, 2, 64) >= 32768)


def test_far_rows():
    """Rows whose elements lie past 2^31: the row offsets and the counters are 64-bit."""
    N, k, H = 300000, 1, 8192
    eo = torch.ones(N, H, dtype=BF, device=DEV)
    pos = torch.arange(N - 1, -1, -1, dtype=torch.int32, device=DEV)
    y = moe.moe_combine_dropout(eo, pos, torch.full((N, 1), 2.0, device=DEV), 0.25, _state(8, 8))
    d_eo, dg, _ = moe.moe_combine_dropout_backward(y, pos, torch.full((N, 1), 2.0, device=DEV), eo, 0.25, _state(8, 8))
    sync()
    t = N - 2
    i0 = t * H // 8
    words = [w for i in range(i0, i0 + H // 8) for w in oracle.philox((i, 0, 8, 0), (8, 0))]
    keep = np.array([v for w in words for v in (w & 0xFFFF, w >> 16)]) >= 16384
    row = f64(y[t])
    v = float(torch.tensor(8 / 3).to(BF))       # 2 * 4 / 3, rounded
    assert np.array_equal(row, np.where(keep, v, 0))
    d = np.float32(v) * np.float32(4 / 3)
    assert np.array_equal(f64(d_eo[1]), np.where(keep, float(torch.tensor(2 * float(d)).to(BF)), 0))
    assert abs(dg[t, 0].item() - keep.sum() * float(d)) <= H * U32 * keep.sum() * float(d)


def test_captured():
    """A captured call reads the generator's state when it replays: every replay draws anew."""
    N, k, H = 50, 2, 264
    eo, g = _t((N * k, H), 1, BF).to(DEV), torch.ones(N, k, device=DEV)
    pos, res = _pos(N, k, N * k, 2).to(DEV), _t((N, H), 3, BF).to(DEV)
    rng = _state(1, 0)
    y = moe.moe_combine_dropout(eo, pos, g, 0.3, rng, residual=res)
    outs = moe.moe_combine_dropout_backward(y, pos, g, eo, 0.3, rng, d_expert_out=torch.zeros_like(eo), want_shared=True)
    z = moe.moe_dropout(res, 0.3, rng)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_combine_dropout(eo, pos, g, 0.3, rng, residual=res, y=y)
        moe.moe_combine_dropout_backward(y, pos, g, eo, 0.3, rng, d_expert_out=outs[0], d_gate=outs[1], d_shared=outs[2])
        moe.moe_dropout(res, 0.3, rng, y=z)
    seen = []
    for i in range(4):
        rng[1] += 1
        eo.normal_()
        graph.replay()
        sync()
        y2 = moe.moe_combine_dropout(eo, pos, g, 0.3, rng, residual=res)
        o2 = moe.moe_combine_dropout_backward(y2, pos, g, eo, 0.3, rng, d_expert_out=torch.zeros_like(eo), want_shared=True)
        z2 = moe.moe_dropout(res, 0.3, rng)
        sync()
        assert torch.equal(y, y2) and torch.equal(z, z2) and all(torch.equal(a, b) for a, b in zip(outs, o2))
        assert not any(torch.equal(z, w) for w in seen)
        seen.append(z.clone())


def test_other_stream():
    x, rng = _t((5000,), 1, F32).to(DEV), _state(2, 3)
    want = moe.moe_dropout(x, 0.4, rng)
    sync()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.moe_dropout(x, 0.4, rng)
    side.synchronize()
    assert torch.equal(want, got)


def _numbers(seed, offset, at, n):
    """The numbers of elements at .. at + n - 1 (at a multiple of 8)."""
    words = [w for i in range(at // 8, (at + n + 7) // 8) for w in oracle.philox((i & 0xFFFFFFFF, i >> 32, offset, 0), (seed, 0))]
    return np.array([v for w in words for v in (w & 0xFFFF, w >> 16)])[:n]


def test_rows_of_more_groups_than_a_launch_has_lanes():
    """2^35 elements and some more: lanes take a second group, and the last elements follow the last whole one."""
    n = 2 ** 35 + 2 ** 12 + 5
    say(f"dropout n={n}")
    x = torch.ones(n, dtype=BF, device=DEV)
    moe.moe_dropout(x, 0.5, _state(1, 2), y=x)
    sync()
    starts = [0, 2 ** 34, 2 ** 35 - 4096, 2 ** 35 - 2048, 2 ** 35, n // 8 * 8 - 64]
    parts = [x[a:a + 69].cpu() for a in starts]
    del x
    torch.cuda.empty_cache()
    for a, part in zip(starts, parts):
        assert np.array_equal(f64(part) * 0.5, (_numbers(1, 2, a, len(part)) >= 32768).astype(float)), a


def test_combine_of_more_columns_than_a_launch_has_lanes():
    """Tokens times columns past what one pass of a launch covers: the workgroups of a token take further columns."""
    N, H = 11300000, 2056   # three passes of 128 lanes a token: 2^32 lanes and some more
    say(f"combine dropout N={N} H={H}")
    eo = torch.ones(3, H, dtype=BF, device=DEV)
    eo[1], eo[2] = 2, 4
    pos = (torch.arange(N, device=DEV) % 3).to(torch.int32)
    y = torch.zeros(N, H, dtype=BF, device=DEV)
    moe.moe_combine_dropout(eo, pos, None, 0.5, _state(1, 2), y=y, k=1)
    sync()
    rows = [0, 1, N // 2, N - 7, N - 1]
    got = [y[t].cpu() for t in rows]
    del y
    torch.cuda.empty_cache()
    for t, row in zip(rows, got):
        assert np.array_equal(f64(row), np.where(_numbers(1, 2, t * H, H) >= 32768, 2.0 * 2 ** (t % 3), 0.0)), t


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N,k,H", [(8, 2, 64), (5, 9, 264), (3, 4, 16392)])
def test_dropped_expert_outputs_do_not_reach_the_gates_gradient(N, k, H, dt):
    """Infinities and NaN where y dropped the sum: the gates' gradient is that of zeros there, bit for bit; where it did
    not, they show."""
    eo, g, dy = _t((N * k, H), 1, dt).to(DEV), torch.rand(N, k, device=DEV), _t((N, H), 2, dt).to(DEV)
    pos = torch.arange(N * k, dtype=torch.int32, device=DEV)
    gone = torch.from_numpy(oracle.dropout_mask(0.5, 3, 4, N * H) == 0).reshape(N, H).repeat_interleave(k, dim=0).to(DEV)
    bad = torch.where(gone, torch.full_like(eo, float("inf")), eo)
    bad[:, ::3] = torch.where(gone, torch.full_like(eo, float("nan")), eo)[:, ::3]
    zero = torch.where(gone, torch.zeros_like(eo), eo)
    got, want, plain = (moe.moe_combine_dropout_backward(dy, pos, g, v, 0.5, _state(3, 4)) for v in (bad, zero, eo))
    kept = int((~gone[1]).nonzero()[0])
    bad[1, kept] = float("nan")
    _, dg, _ = moe.moe_combine_dropout_backward(dy, pos, g, bad, 0.5, _state(3, 4))
    sync()
    assert all(torch.equal(a, b) and torch.equal(b, c) for a, b, c in zip(got[:2], want[:2], plain[:2]))
    assert torch.isnan(dg.reshape(-1)).nonzero().tolist() == [[1]]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N,k,H", [(6, 2, 72), (5, 9, 136), (3, 32, 2056), (2, 17, 16392)])
def test_shared_gradient_in_place(N, k, H, dt):
    """d_shared may be dy, also where a token's slots take several passes over it."""
    eo, dy, g = _t((N * k, H), 1, dt).to(DEV), _t((N, H), 2, dt).to(DEV), torch.rand(N, k, device=DEV)
    pos = torch.arange(N * k, dtype=torch.int32, device=DEV)
    want = moe.moe_combine_dropout_backward(dy, pos, g, eo, 0.4, _state(3, 4), want_shared=True)
    got = moe.moe_combine_dropout_backward(dy, pos, g, eo, 0.4, _state(3, 4), d_shared=dy)
    sync()
    assert got[2] is dy and all(torch.equal(a, b) for a, b in zip(want, got))

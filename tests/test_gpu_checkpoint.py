"""GPU parity of the activations kept in 8 bits with the oracle: codes and values bit for bit, the
SwiGLU backward from them within bounds derived from its fp32 arithmetic."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(autouse=True, scope="module")
def _return_cached_blocks():
    """The allocator's cached blocks go back afterwards: a test elsewhere counts the bytes it hands out, and
    an unsplit block of these sizes would count as more."""
    yield
    torch.cuda.empty_cache()
U32 = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16]


def _values(rows, cols, dt, seed=0):
    """Rows over many binades, with zeros, signed zeros, ties of the code grid and block maxima at and
    next to 448 times a power of two."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * np.exp2(rng.integers(-30, 31, size=(rows, 1)).astype(np.float64))
    flat = x.reshape(-1, 32)
    for i in range(0, len(flat), 7):
        kind = (i // 7) % 7
        if kind == 0:
            flat[i] = 0.0
            flat[i, 3] = -0.0
        elif kind == 1:   # maxima of exactly 448 and ties halfway between codes
            flat[i] = rng.integers(-56, 57, 32) * 4.0 + rng.integers(0, 2, 32) * 2.0
            flat[i, 0] = 448.0
        elif kind == 2:   # just above: the next scale
            flat[i, 0] = 450.0
        elif kind == 3:   # subnormal codes
            flat[i] = rng.integers(-40, 41, 32) * 2.0 ** -10
            flat[i, 0] = 448.0
        elif kind == 4:   # below the smallest scale's codes
            flat[i] = rng.normal(size=32) * 2.0 ** -124
        elif kind == 5:
            flat[i, 1] = 2.0 ** 127 * 1.5
    return torch.from_numpy(x).to(torch.float32).to(dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (257, 1056), (1000, 64), (33, 4096)])
def test_codes_and_values(rows, cols, dt):
    say(f"keep {rows}x{cols} {dt}")
    x = _values(rows, cols, dt)
    q, s = moe.moe_quantize_mxfp8(x.to(DEV))
    v32, v16 = moe.moe_dequantize_mxfp8(q, s, dtype=torch.float32), moe.moe_dequantize_mxfp8(q, s)
    sync()
    rq, rs = oracle.mx_quantize(f64(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    ref = oracle.mx_dequantize(rq, rs)
    assert np.array_equal(f64(v32), ref) and np.array_equal(f64(v16), ref)


def test_not_finite():
    """A block with a NaN or an infinity reads back as NaN; its neighbours are not touched."""
    say("keep: not finite")
    for dt in TYPES:
        x = _values(8, 128, dt, seed=2)
        x[0, 5], x[1, 40], x[2, 127] = float("nan"), float("inf"), -float("inf")
        q, s = moe.moe_quantize_mxfp8(x.to(DEV))
        got = f64(moe.moe_dequantize_mxfp8(q, s, dtype=torch.float32))
        rq, rs = oracle.mx_quantize(f64(x))
        assert np.array_equal(s.cpu().numpy(), rs) and (rs == 255).sum() == 3
        assert np.array_equal(got, oracle.mx_dequantize(rq, rs), equal_nan=True)


def test_every_scale_and_code():
    """All 256 codes under every scale byte of the format, in both types."""
    say("keep: every code")
    codes = np.tile(np.arange(256, dtype=np.uint8), (238, 1))
    scales = np.repeat(np.arange(10, 248, dtype=np.uint8)[:, None], 8, axis=1)
    # (the two types' range ends below 2^128: the largest scale's codes of 256 and more are infinities)
    with np.errstate(over="ignore"):
        ref = oracle.mx_dequantize(codes, scales).astype(np.float32).astype(np.float64)
    for dt in TYPES:
        got = moe.moe_dequantize_mxfp8(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), dtype=dt)
        assert np.array_equal(f64(got), ref, equal_nan=True)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols,k", [(1, 32, 1), (129, 160, 3), (70, 7168, 8), (500, 64, 2)])
def test_expert_ordered_rows(rows, cols, k, dt):
    """Rows scattered by a layout with dropped slots: bit for bit the values; unnamed rows, and rows
    behind the last, stay as they were."""
    say(f"keep rows {rows}x{cols} k={k}")
    rng = np.random.default_rng(rows)
    x = _values(rows, cols, dt, seed=3)
    pos = rng.permutation(rows * k).astype(np.int32)
    pos[rng.random(rows * k) < 0.2] = -1
    out = torch.full((rows * k + 3, cols), 7.5, dtype=dt, device=DEV)
    q, s = moe.moe_quantize_mxfp8(x.to(DEV))
    moe.moe_dequantize_mxfp8(q, s, out=out, send_pos=torch.from_numpy(pos).to(DEV), k=k)
    sync()
    ref = np.full((rows * k + 3, cols), 7.5)
    vals = oracle.mx_dequantize(*oracle.mx_quantize(f64(x)))
    for slot, r in enumerate(pos):
        if r >= 0:
            ref[r] = vals[slot // k]
    assert np.array_equal(f64(out), ref)


def _swiglu_case(N, k, I, dt, seed, drop):
    rng = np.random.default_rng(seed)
    rows = N * max(k, 1)
    au = torch.from_numpy(rng.normal(size=(rows, 2 * I)) * 2.5).to(torch.float32)
    au[:, ::19] *= 12      # far into the logistic's tails
    q, s = oracle.mx_quantize(f64(au.to(dt)))
    dh = torch.from_numpy(rng.normal(size=(rows, I)) / 64).to(torch.float32).to(dt)
    pos = g = None
    if k:
        pos = rng.permutation(rows).astype(np.int32)
        if drop:
            pos[rng.random(rows) < 0.15] = -1
        g = rng.random((N, k)).astype(np.float32)
    return q, s, dh, pos, g


# rows of one token, below and above 4096 slots, every share of a workgroup; odd widths
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N,k,I", [(1, 1, 32), (1, 0, 96), (7, 3, 256), (33, 4, 288), (300, 2, 1056), (11, 0, 14336),
                                   (1500, 3, 320), (5000, 0, 64)])
def test_swiglu_backward(N, k, I, dt):
    say(f"kept swiglu N={N} k={k} I={I} {dt}")
    for drop in ((False, True) if k else (False,)):
        q, s, dh, pos, g = _swiglu_case(N, k, I, dt, N + I, drop)
        rows = len(q)
        dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        d_au = torch.full((rows, 2 * I), 3.0, dtype=dt, device=DEV)
        h = torch.full((rows, I), 3.0, dtype=dt, device=DEV)
        _, _, dg = moe.moe_swiglu_backward_mxfp8(dev(q), dev(s), dh.to(DEV), dev(pos), dev(g), d_au=d_au, h=h)
        sync()
        au, d = oracle.mx_dequantize(q, s), f64(dh)
        r_au, r_h, r_dg = oracle.kept_swiglu_backward(au, d, pos, g)
        named = np.ones(rows, bool) if pos is None else np.isin(np.arange(rows), pos)
        gr = np.ones(rows)
        if pos is not None:
            gr = np.zeros(rows)
            gr[pos[pos >= 0]] = g.reshape(-1)[pos >= 0]
        a, u = np.abs(au[:, :I]), np.abs(au[:, I:])
        sg = 1 / (1 + np.exp(-au[:, :I]))
        # the logistic: its exponent's argument rounds by 2^-24 |a| and carries the constant's
        # rounding, exponential and reciprocal within 2^-23 each, the sum within 2^-24; then at
        # most 6 products; doubled.  (Below 2^-126 the hardware exponential and reciprocal give 0.)
        eps = 2 * U32 * (1.5 * a + 6 + 6)
        tiny = 2.0 ** -120 * (1 + a) * (1 + u)
        half = torch.finfo(dt).eps / 2
        gd = (gr[:, None] * np.abs(d))
        b_h = gr[:, None] * a * sg * u * eps + tiny
        b_au = np.concatenate([gd * u * (sg + 2 * a * sg) * eps + tiny, gd * a * sg * eps + tiny], axis=1)
        for got, ref, b in ((f64(d_au), r_au, b_au), (f64(h), r_h, b_h)):
            assert np.all((np.abs(got - ref) <= b + half * (np.abs(ref) + b))[named])
            assert (got[~named] == 3.0).all()
        if g is None:
            assert dg is None
            continue
        # the dot product: every term as h, and at most I / 16 + 16 additions
        row_b = (np.abs(d) * (a * sg * u * (eps + 2 * U32 * (I / 16 + 16)) + tiny)).sum(axis=1)
        got = f64(dg).reshape(-1)
        for slot, r in enumerate(pos):
            if r < 0:
                assert got[slot] == 0.0
            else:
                assert abs(got[slot] - r_dg[slot]) <= row_b[r]


def test_positions_out_of_range_are_dropped():
    """A position behind the last row is a dropped slot: nothing is written for it."""
    say("kept swiglu: positions out of range")
    q, s, dh, pos, g = _swiglu_case(6, 2, 64, torch.bfloat16, 5, False)
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    pos[3] = 12
    pos[7] = 2 ** 31 - 1
    d_au = torch.zeros(12, 128, dtype=torch.bfloat16, device=DEV)
    _, _, dg = moe.moe_swiglu_backward_mxfp8(dev(q), dev(s), dh.to(DEV), dev(pos), dev(g), d_au=d_au)
    sync()
    gone = ~np.isin(np.arange(12), pos)
    assert gone.sum() == 2 and not f64(d_au)[gone].any()
    assert f64(dg).reshape(-1)[3] == 0 and f64(dg).reshape(-1)[7] == 0


def test_captured_and_on_another_stream():
    """Quantize, dequantize and the SwiGLU backward in one captured graph, replayed on new inputs; the
    same calls on a stream of their own."""
    say("keep: graph and stream")
    rows, I = 700, 256
    au = torch.empty(rows, 2 * I, dtype=torch.bfloat16, device=DEV)
    dh = torch.empty(rows, I, dtype=torch.bfloat16, device=DEV)
    au.normal_()
    dh.normal_()
    q, s = moe.moe_quantize_mxfp8(au)
    v = moe.moe_dequantize_mxfp8(q, s)
    d_au, h, _ = moe.moe_swiglu_backward_mxfp8(q, s, dh)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_quantize_mxfp8(au, q, s)
        moe.moe_dequantize_mxfp8(q, s, out=v)
        moe.moe_swiglu_backward_mxfp8(q, s, dh, d_au=d_au, h=h)
    side = torch.cuda.Stream()
    for i in range(3):
        au.normal_()
        dh.normal_()
        graph.replay()
        sync()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q2, s2 = moe.moe_quantize_mxfp8(au)
            v2 = moe.moe_dequantize_mxfp8(q2, s2)
            d2, h2, _ = moe.moe_swiglu_backward_mxfp8(q2, s2, dh)
        sync()
        for x, y in ((q, q2), (s, s2), (v, v2), (d_au, d2), (h, h2)):
            assert torch.equal(x, y)


def _gate_up_inputs(N, H, E, k, I, seed, hot=False):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((N, E)), axis=1)[:, :k]
    if hot:   # one expert with every token, one with none
        idx = np.where(idx == E - 1, 1, idx)
        idx[:, 0] = 0
        for t in range(N):
            if len(set(idx[t])) < k:
                idx[t] = [0] + [e for e in rng.permutation(E) if e not in (0, E - 1)][:k - 1]
    n_e, off, sp, ss = oracle.dispatch_layout(idx.astype(np.int32), E)
    t = lambda *s: torch.from_numpy(rng.normal(size=s)).to(torch.bfloat16).to(DEV)  # noqa: E731
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)  # noqa: E731
    std = H ** -0.5
    return t(N, H), t(E, 2 * I, H) * std, t(1, 2 * I, H) * std, dev(off), dev(ss), n_e


# tiles of every shape: one row, 1 x 4 and 2 x 2 layouts, experts of 257..320 rows (320-row tiles), a hot
# and an empty expert, column blocks that end inside a tile
@pytest.mark.parametrize("N,H,E,k,I,hot", [(1, 128, 4, 1, 128, False), (5, 256, 3, 2, 128, False),
                                           (200, 256, 8, 3, 256, False), (300, 512, 4, 2, 384, True),
                                           (1100, 256, 8, 2, 128, False), (600, 128, 5, 2, 640, True)])
def test_gate_up_keeps_the_codes_of_its_bf16_rows(N, H, E, k, I, hot):
    """h and the codes are bit for bit those of the GEMM that writes bf16 pre-activations and the
    quantizer, with and without the shared expert; rows behind the last are left as they were."""
    say(f"gate/up with kept codes N={N} H={H} E={E} k={k} I={I} hot={hot}")
    x, w13, sw, off, ss, n_e = _gate_up_inputs(N, H, E, k, I, N + I, hot)
    rows = N * k
    au = torch.empty(rows + N, 2 * I, dtype=torch.bfloat16, device=DEV)
    h = moe.moe_expert_gate_up_gathered_shared(x, ss, k, off, w13, sw, au=au)
    q, s = moe.moe_quantize_mxfp8(au)
    h2, q2, s2 = moe.moe_expert_gate_up_mxfp8(x, ss, k, off, w13, sw)
    sync()
    assert torch.equal(h, h2) and torch.equal(q, q2) and torch.equal(s, s2)
    h3 = torch.full((rows, I), 3.0, dtype=torch.bfloat16, device=DEV)
    q3 = torch.full((rows, 2 * I), 5, dtype=torch.uint8, device=DEV)
    s3 = torch.full((rows, 2 * I // 32), 6, dtype=torch.uint8, device=DEV)
    short = off.clone()
    last = int(off[-1]) - int(n_e[-1])
    short[-1] = last            # the last expert's rows count for nobody
    moe.moe_expert_gate_up_mxfp8(x, ss, k, short, w13, rows=rows, h=h3, au_q=q3, au_scale=s3)
    sync()
    assert torch.equal(h3[:last], h[:last]) and torch.equal(q3[:last], q[:last]) and torch.equal(s3[:last], s[:last])
    assert (h3[last:] == 3).all() and (q3[last:] == 5).all() and (s3[last:] == 6).all()


# the same on sizes that take each tile shape: 64 weight rows (one round of tiles), 128 (few tiles; many tiles with few
# rows an expert), and 256 (even experts, experts of 257..320 rows, a hot and an empty one)
@pytest.mark.parametrize("N,H,E,k,I,hot", [(97, 1152, 6, 2, 384, False), (161, 384, 3, 2, 128, True),
                                           (513, 640, 16, 4, 512, False), (450, 256, 8, 2, 1024, True),
                                           (90, 512, 33, 4, 1152, False), (2, 256, 200, 8, 2176, False),
                                           (1100, 256, 8, 2, 2048, False), (600, 128, 5, 2, 2560, True),
                                           (300, 512, 4, 2, 4096, True), (200, 256, 3, 3, 8192, False)])
def test_gate_up_kept_codes_of_every_tile_shape(N, H, E, k, I, hot):
    test_gate_up_keeps_the_codes_of_its_bf16_rows(N, H, E, k, I, hot)


def test_gate_up_kept_codes_shared_rows_only():
    """No routed rows: the shared expert's alone, without a slot table."""
    say("gate/up with kept codes: shared rows only")
    for N, I in ((70, 256), (700, 4096)):
        x, w13, sw, off, ss, _ = _gate_up_inputs(N, 256, 2, 1, I, 7)
        au = torch.empty(2 * N, 2 * I, dtype=torch.bfloat16, device=DEV)
        h = moe.moe_expert_gate_up_gathered_shared(x, ss, 1, off, w13, sw, au=au)
        q, s = moe.moe_quantize_mxfp8(au)
        h2, q2, s2 = moe.moe_expert_gate_up_mxfp8(x, ss[:0], 1, torch.zeros_like(off), w13, sw, rows=0)
        sync()
        assert torch.equal(h[N:], h2) and torch.equal(q[N:], q2) and torch.equal(s[N:], s2)


def test_gate_up_kept_codes_not_finite():
    """A token with a NaN gives NaN blocks in its own rows only."""
    say("gate/up with kept codes: NaN")
    x, w13, sw, off, ss, _ = _gate_up_inputs(40, 128, 4, 2, 128, 1)
    x[7, 3] = float("nan")
    _, q, s = moe.moe_expert_gate_up_mxfp8(x, ss, 2, off, w13, sw)
    sync()
    mine = np.concatenate([ss.cpu().numpy() // 2 == 7, np.arange(40) == 7])
    assert (s.cpu().numpy()[mine] == 255).all() and (s.cpu().numpy()[~mine] != 255).all()

"""GPU parity of the balance loss, its counts and the logits' gradient with the float64 oracle."""
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


def _case(N, E, k, S=1, seed=0, mask=False, bias=False, bad_ids=False):
    rng = np.random.default_rng(seed)
    z = (rng.normal(size=(N, E)) + 0.5 * rng.normal(size=E)).astype(np.float32)
    b = rng.normal(size=E).astype(np.float32) if bias else None
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    if bad_ids:
        idx[rng.random(idx.shape) < 0.1] = -1
        idx[rng.random(idx.shape) < 0.1] = E
    seq = None
    if S > 1:
        seq = np.sort(rng.integers(0, N + 1, S + 1)).astype(np.int32)
        seq[1] = seq[2] if S > 2 else seq[1]     # an empty sequence
    m = (rng.random(N) < 0.8).astype(np.uint8) if mask else None
    return dict(z=z, topk_idx=idx, bias=b, seq_start=seq, mask=m)


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _loss(c, alpha, **kw):
    return moe.moe_balance_loss(_dev(c["z"]), _dev(c["topk_idx"]), alpha, bias=_dev(c["bias"]),
                                seq_start=_dev(c["seq_start"]), token_mask=_dev(c["mask"]), **kw)


def _grad(c, alpha, counts, tokens, **kw):
    return moe.moe_balance_loss_backward(_dev(c["z"]), _dev(c["topk_idx"]), alpha, counts, tokens, bias=_dev(c["bias"]),
                                         seq_start=_dev(c["seq_start"]), token_mask=_dev(c["mask"]), **kw)


def _prob_rel(c):
    """Relative bound of one probability: the argument z - max rounds by 2^-24 |z - max|, which the
    exponential carries as a relative error; exponential, reciprocal and product within 2 ulp each,
    the sum of at most 16 terms a lane and a 6-step tree; doubled for second order."""
    zb = oracle.biased_logits(c["z"], c["bias"])
    zb = np.where(np.isfinite(zb), zb, 0.0)
    return 2 * U32 * (float((zb.max(axis=1) - zb.min(axis=1)).max()) + 6 + 22) if zb.size else 0.0


def _check(c, alpha=0.03, d_loss=1.7, dz_dtype=torch.float32, gates=False):
    N, E = c["z"].shape
    k = c["topk_idx"].shape[1]
    loss, counts, prob, tokens = _loss(c, alpha)
    g = dg = None
    if gates:
        rng = np.random.default_rng(7)
        g = np.exp(rng.normal(size=(N, k)))
        g = (g / g.sum(axis=1, keepdims=True)).astype(np.float32)
        dg = rng.normal(size=(N, k)).astype(np.float32)
    dl = torch.full((1,), d_loss, device=DEV)
    dz = _grad(c, alpha, counts, tokens, d_loss=dl, topk_gate=_dev(g), d_gate=_dev(dg), dz_dtype=dz_dtype)
    sync()
    rl, rc, rp, rt = oracle.balance_loss(alpha=alpha, **c)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    rel = _prob_rel(c)
    # a mean of positive terms: at most N / 512 + 2 passes of a chunk, 5 steps across a wave's groups,
    # 16 waves, 8 partials a row and 64 rows, each adding once: N / 512 + 95 roundings
    mean_rel = rel + 2 * U32 * (N / 512 + 4 + 32 + 26)
    assert np.all(np.abs(f64(prob) - rp) <= mean_rel * rp + 1e-37)
    # the loss adds at most 2^16 positive shares: 256 a thread and an 8-step tree, 6 products
    assert abs(float(loss) - rl) <= (mean_rel + 2 * U32 * (256 + 8 + 10)) * rl + 1e-37
    rdz = oracle.balance_loss_backward(alpha=alpha, d_loss=float(dl), gates=g, dg=dg, **c)
    # p (a - sum p a) with a about the even load: a within 8 roundings, p within rel, the sum of
    # products within rel + a 22-step sum
    zb = oracle.biased_logits(c["z"], c["bias"])
    bound = np.zeros((N, E))
    starts = [0, N] if c["seq_start"] is None else np.clip(c["seq_start"], 0, N)
    for s, (lo, hi) in enumerate(zip(starts, starts[1:])):
        if rt[s] == 0 or lo >= hi:
            continue
        p = oracle._row_softmax(zb[lo:hi])
        a = float(dl) * alpha / len(rt) * np.abs(E * rc[s] - k * rt[s]) / (k * float(rt[s]) ** 2)
        bound[lo:hi] = p * (a[None, :] + (p @ a)[:, None]) * (2 * rel + 2 * U32 * 32)
        # the oracle's own float64 roundings: it takes a in full, not about the even load, so where
        # the loads are even (true gradient 0) p (a - sum p a) leaves up to E + 16 roundings of p a
        full = float(dl) * alpha / len(rt) * E * rc[s] / (k * float(rt[s]) ** 2)
        bound[lo:hi] += p * (full[None, :] + (p @ full)[:, None]) * (E + 16) * 2.0 ** -53
    if gates:
        g64, d64 = g.astype(np.float64), dg.astype(np.float64)
        zb4 = 4 * (k + 2) * U32 * g64 * (np.abs(d64) + np.abs(g64 * d64).sum(axis=1, keepdims=True))
        for t in range(N):
            for j, e in enumerate(c["topk_idx"][t]):
                if 0 <= e < E:
                    bound[t, e] += zb4[t, j]
        bound += 2 * U32 * (k + 1) * np.abs(rdz) + 2 * bound   # (the parts are added in fp32)
    step = torch.finfo(dz_dtype).eps / 2
    assert dz.dtype == dz_dtype and np.all(np.abs(f64(dz) - rdz) <= bound + step * (np.abs(rdz) + bound) + 1e-37)


# experts: odd, below and above a wave, every group width; tokens: one, odd, several chunks
@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (1, 4, 2), (3, 6, 6), (65, 8, 2), (700, 13, 3), (129, 16, 4), (77, 30, 5),
                                   (500, 32, 4), (33, 60, 4), (257, 64, 8), (40, 100, 32), (300, 128, 6), (513, 160, 6),
                                   (90, 201, 8), (2100, 256, 8), (50, 333, 8), (31, 512, 9), (17, 1000, 8),
                                   (20, 1021, 10)])
def test_sizes(N, E, k):
    say(f"balance N={N} E={E} k={k}")
    _check(_case(N, E, k, seed=N + E))
    _check(_case(N, E, k, seed=N + E + 1, mask=True, bias=True, bad_ids=True), dz_dtype=torch.bfloat16, gates=True)


@pytest.mark.parametrize("N,E,S", [(100, 8, 3), (1000, 24, 40), (37, 60, 90), (2500, 256, 7), (9000, 5, 300)])
def test_sequences(N, E, S):
    """Packed sequences, empty ones and tokens outside all of them."""
    say(f"balance sequences N={N} E={E} S={S}")
    for mask in (False, True):
        _check(_case(N, E, 2, S=S, seed=S, mask=mask, bias=True), gates=mask)


@pytest.mark.parametrize("N,E,ones", [(3000, 32, 64), (700, 4, 39), (5000, 100, 20)])
def test_uneven_sequences(N, E, ones):
    """Sequences of one token, then one of all the others: a chunk meets many sequences and a sequence
    many chunks."""
    say(f"balance uneven sequences N={N} E={E} ones={ones}")
    c = _case(N, E, 2, seed=ones, mask=True)
    for seq in ([*range(ones + 1), N], [0, *range(N - ones, N + 1)]):
        c["seq_start"] = np.array(seq, np.int32)
        _check(c, gates=True)


def test_nothing_counts():
    """No tokens at all, a mask that leaves none, and no sequence with a token: loss 0, gradient 0."""
    say("balance: nothing counts")
    c = _case(40, 12, 2, seed=3)
    c["mask"] = np.zeros(40, np.uint8)
    _check(c)
    c = _case(40, 12, 2, seed=4)
    c["seq_start"] = np.array([7, 7, 7], np.int32)
    _check(c, gates=True)
    z, idx = torch.empty(0, 12, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    loss, counts, prob, tokens = moe.moe_balance_loss(z, idx, 0.1)
    dz = moe.moe_balance_loss_backward(z, idx, 0.1, counts, tokens)
    sync()
    assert float(loss) == 0 and not counts.any() and not prob.any() and not tokens.any() and dz.shape == (0, 12)


def test_infinite_and_nan_logits():
    """-inf logits (masked experts, a whole row of them) and the type's lowest value have no
    probability; NaN and +inf in uncounted tokens do nothing; in a counted token they show."""
    say("balance: infinities and NaN")
    c = _case(64, 24, 3, S=4, seed=5, mask=True)
    c["z"][:, 5] = -np.inf
    c["z"][:, 6] = np.finfo(np.float32).min
    c["z"][11] = -np.inf
    on = np.flatnonzero(c["mask"])
    off = np.flatnonzero(c["mask"] == 0)
    loss, counts, prob, tokens = _loss(c, 0.1)
    dz = _grad(c, 0.1, counts, tokens)
    c["z"][off[0]] = np.nan
    c["z"][off[1], 3] = np.inf
    loss2, counts2, prob2, tokens2 = _loss(c, 0.1)
    dz2 = _grad(c, 0.1, counts2, tokens2)
    sync()
    # finite logits within 12 of each other: each probability within 2^-23 (12 + 28), the sums of 64
    # tokens and 24 experts within 2^-23 70
    rl = oracle.balance_loss(alpha=0.1, **c)[0]
    assert abs(float(loss) - rl) <= 2 * U32 * 110 * rl
    assert torch.equal(loss, loss2) and torch.equal(prob, prob2) and torch.equal(dz, dz2)
    assert torch.isfinite(dz).all() and not dz[:, 5].any() and not dz[11].any()
    inside = [t for t in on if c["seq_start"][0] <= t < c["seq_start"][-1]]
    c["z"][inside[0], 2] = np.nan
    loss3 = _loss(c, 0.1)[0]
    sync()
    assert torch.isnan(loss3).all()


def test_same_bits_and_offset_views():
    """Repeats give the same bits; z and dz that start off a 16-byte boundary give the same values."""
    say("balance: repeats, unaligned rows")
    c = _case(3000, 64, 4, S=5, seed=6)
    a, b = _loss(c, 0.1), _loss(c, 0.1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = _grad(c, 0.1, a[1], a[3])
    assert torch.equal(g, _grad(c, 0.1, a[1], a[3]))
    zo = torch.empty(3000 * 64 + 1, device=DEV)[1:].view(3000, 64)
    zo.copy_(_dev(c["z"]))
    do = torch.empty(3000 * 64 + 1, device=DEV)[1:].view(3000, 64)
    args = dict(seq_start=_dev(c["seq_start"]))
    loss, counts, prob, tokens = moe.moe_balance_loss(zo, _dev(c["topk_idx"]), 0.1, **args)
    moe.moe_balance_loss_backward(zo, _dev(c["topk_idx"]), 0.1, counts, tokens, dz=do, **args)
    sync()
    assert torch.equal(counts, a[1])
    assert np.all(np.abs(f64(prob) - f64(a[2])) <= 2e-5 * f64(a[2]))
    assert np.abs(f64(do) - f64(g)).max() <= 1e-5 * np.abs(f64(g)).max()


def test_two_streams_and_a_captured_graph():
    """Two calls in flight on two streams with workspaces of their own, and a captured pair of calls
    replayed on new inputs with eager work between."""
    say("balance: streams and a graph")
    c1, c2 = _case(4000, 128, 4, seed=8), _case(3500, 96, 3, seed=9)
    ref1, ref2 = _loss(c1, 0.1), _loss(c2, 0.1)
    sync()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        o1 = _loss(c1, 0.1)
    with torch.cuda.stream(s2):
        o2 = _loss(c2, 0.1)
    sync()
    assert all(torch.equal(x, y) for x, y in zip(ref1 + ref2, o1 + o2))
    z, idx = _dev(c1["z"]), _dev(c1["topk_idx"])
    ws = torch.empty(moe.moe_workspace_bytes(moe.MOE_OP_BALANCE_LOSS, 4000, 0, 0, 128, 1, 0), dtype=torch.uint8,
                     device=DEV)
    out = moe.moe_balance_loss(z, idx, 0.1, ws=ws)
    dz = moe.moe_balance_loss_backward(z, idx, 0.1, out[1], out[3])
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_balance_loss(z, idx, 0.1, out=out, ws=ws)
        moe.moe_balance_loss_backward(z, idx, 0.1, out[1], out[3], dz=dz)
    for seed in (20, 21, 22):
        n = _case(4000, 128, 4, seed=seed)
        z.copy_(_dev(n["z"]))
        idx.copy_(_dev(n["topk_idx"]))
        ws.fill_(255)
        graph.replay()
        sync()
        want = _loss(n, 0.1)
        assert all(torch.equal(x, y) for x, y in zip(want, out))
        assert torch.equal(dz, _grad(n, 0.1, want[1], want[3]))


def test_one_chunk_of_one_listed_sequence():
    """A batch small enough for one launch whose only sequence is listed: a part of the batch, all of
    it, none of it, and outside it."""
    say("balance: one listed sequence")
    for lo, hi in ((3, 20), (0, 25), (9, 9), (40, 50), (-5, 7), (20, 3)):
        c = _case(25, 60, 4, seed=30)
        c["seq_start"] = np.array([lo, hi], np.int32)
        if lo <= hi:
            _check(c, gates=True)
        else:   # (not a valid list: no token)
            loss, counts, _, tokens = _loss(c, 0.1)
            sync()
            assert float(loss) == 0 and not counts.any() and not tokens.any()

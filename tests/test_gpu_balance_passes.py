"""GPU parity of the balance loss where a group of lanes works on several tokens one after the other, of loads whose
counts need more than 24 bits, and of batches without tokens or with an expert named twice by a token."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from oracle import moe_oracle as oracle
from tests.gpu_util import f64, say, sync
from tests.test_gpu_balance import DEV, U32, _case, _check, _dev, _prob_rel, _return_cached_blocks  # noqa: F401

pytestmark = pytest.mark.gpu


# the gradient's 2048 workgroups hold 8192 tokens with more than 128 experts and 262144 with up to eight, the loss's
# 512 chunks of two passes 16384 with more than 128: larger batches, of one sequence and of many (empty ones, and
# tokens before the first and behind the last), with 16-byte rows and without
@pytest.mark.parametrize("N,E,k,S", [(8200, 160, 6, 1), (9001, 160, 6, 37), (16500, 201, 8, 5), (33000, 256, 4, 700),
                                     (33100, 132, 2, 1), (270000, 4, 3, 11)])
def test_several_tokens_a_group(N, E, k, S):
    say(f"balance, several tokens a group: N={N} E={E} k={k} S={S}")
    _check(_case(N, E, k, S=S, seed=N + S, mask=S != 1, bias=E % 4 != 0, bad_ids=True), gates=S != 700,
           dz_dtype=torch.bfloat16 if k == 6 else torch.float32)


def test_sequences_that_end_inside_a_workgroup():
    """Sequences of one to nine tokens, an empty one after every third: the coefficients change from token to
    token, and some tokens of a group belong to no sequence."""
    say("balance, several tokens a group: short sequences")
    N, E = 8400, 132
    c = _case(N, E, 3, seed=40, mask=True)
    rng = np.random.default_rng(41)
    cuts = np.cumsum(rng.integers(1, 10, 1500))
    cuts = cuts[cuts < N - 30] + 3
    c["seq_start"] = np.sort(np.concatenate([cuts, cuts[::3]])).astype(np.int32)
    _check(c, gates=True)


@pytest.mark.parametrize("E,k,T,odd", [(5, 5, 3500001, False), (7, 7, 5000001, True), (160, 6, 3000001, True), (160, 6, 8000001, True),
                                       (3, 3, 100000007, True), (1024, 2, 1048575, True)])
def test_loads_beyond_24_bits(E, k, T, odd):
    """Counts of millions of tokens: the difference of an expert's load and the even one keeps every digit.  All
    experts chosen by every token: no gradient at all; loads next to the even one: the gradient of that difference."""
    say(f"balance, large counts: E={E} k={k} T={T}")
    N, alpha = 9, 1e9
    c = _case(N, E, k, seed=E)
    counts = np.full((1, E), k * T // E, np.int64)
    if odd:
        counts[0] += np.arange(E) % 3 - 1
    dz = moe.moe_balance_loss_backward(_dev(c["z"]), _dev(c["topk_idx"]), alpha, _dev(counts.astype(np.int32)),
                                       torch.tensor([T], dtype=torch.int32, device=DEV))
    sync()
    diff = [E * int(n) - k * T for n in counts[0]]
    if not odd:
        assert not any(diff) and not dz.any()
        return
    a = alpha / k / float(T) ** 2 * np.array(diff, np.float64)
    p = oracle._row_softmax(c["z"])
    ref = p * (a[None, :] - (p @ a)[:, None])
    # (as in the parity tests: a within 8 roundings, p within its bound, a sum of at most 22 steps)
    bound = p * (np.abs(a)[None, :] + (p @ np.abs(a))[:, None]) * (2 * _prob_rel(c) + 2 * U32 * 32)
    assert np.all(np.abs(f64(dz) - ref) <= bound + U32 * (np.abs(ref) + bound) + 1e-37)


@pytest.mark.parametrize("S", [1, 2, 70])
def test_no_tokens_and_several_sequences(S):
    say(f"balance, no tokens: S={S}")
    z, idx = torch.empty(0, 12, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    seq = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    out = (torch.full((1,), 7.0, device=DEV), torch.full((S, 12), 7, dtype=torch.int32, device=DEV),
           torch.full((S, 12), 7.0, device=DEV), torch.full((S,), 7, dtype=torch.int32, device=DEV))
    moe.moe_balance_loss(z, idx, 0.1, seq_start=seq, out=out)
    dz = moe.moe_balance_loss_backward(z, idx, 0.1, out[1], out[3], seq_start=seq)
    sync()
    assert not any(t.any() for t in out) and dz.shape == (0, 12)


def test_an_expert_named_twice():
    """A token whose slots name one expert several times counts it as often, and every slot's gradient arrives."""
    say("balance: the same expert twice")
    for E, k in ((6, 4), (40, 8), (256, 8)):
        c = _case(300, E, k, S=3, seed=E, mask=True)
        c["topk_idx"][::2, 1] = c["topk_idx"][::2, 0]
        c["topk_idx"][::3] = c["topk_idx"][::3, :1]
        _check(c, gates=True)

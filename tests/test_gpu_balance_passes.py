"""GPU parity of the balance loss where a group of lanes works on several tokens one after the other, and of
batches without tokens or with an expert named twice by a token."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from tests.gpu_util import say, sync
from tests.test_gpu_balance import DEV, _case, _check, _return_cached_blocks  # noqa: F401

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

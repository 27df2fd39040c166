"""Repeats of the gate/up GEMM that keeps its codes: the same inputs give the same bits."""
import pytest
import torch

import combine_grouped_gemm_amd as moe
from tests.gpu_util import say, sync
from tests.test_gpu_checkpoint import _gate_up_inputs, _return_cached_blocks  # noqa: F401

pytestmark = pytest.mark.gpu


def test_kept_codes_repeat_themselves():
    """The gate/up with kept codes gives the same bits on every call, with other inputs in between (every tile shape:
    128-row tiles of 64 and 128 weight rows, 256 x 256, 320 x 256)."""
    for N, H, E, k, I in ((97, 1152, 6, 2, 384), (509, 1024, 16, 4, 512), (1100, 256, 8, 2, 2048), (580, 256, 4, 2, 4096)):
        say(f"gate/up with kept codes, repeats: N={N} H={H} E={E} k={k} I={I}")
        a, b = (_gate_up_inputs(N, H, E, k, I, seed)[:5] for seed in (1, 2))
        run = lambda t: moe.moe_expert_gate_up_mxfp8(t[0], t[4], k, t[3], t[1], t[2])  # noqa: E731
        first = run(a)
        for _ in range(3):
            run(b)
            again = run(a)
            sync()
            assert all(torch.equal(x, y) for x, y in zip(first, again))

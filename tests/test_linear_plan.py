"""Launch limits and the choice of a kernel of the expert product, on the CPU."""
import random

import pytest

import combine_grouped_gemm_amd as moe
from combine_grouped_gemm_amd import MOE_BF16, MOE_ERR_UNSUPPORTED, MOE_F32
from tests.linear_plan import plans

FAKE = 4096   # a non-null, 16-byte aligned host integer: never dereferenced on these paths


def _linear(rows, K, N, E, f32, gated):
    dt = MOE_F32 if f32 else MOE_BF16
    return moe.lib().moe_expert_linear(FAKE, dt, 0, None, 1, FAKE, E, rows, K, N, FAKE, None, MOE_F32, 0, int(gated), None,
                                       FAKE, None, FAKE, 1 << 60, None)


@pytest.mark.parametrize("rows,K,N,E,f32,gated", [
    (2 ** 30, 8, 8, 1, False, False),            # 2^24 tiles of 64 x 64, 256 lanes each
    (2 ** 30, 8, 8, 1, False, True), (2 ** 30, 8, 8, 7, False, False), (2 ** 31 - 2 ** 16 - 1, 8, 8, 1024, True, False),
    (2 ** 30, 8, 24, 3, False, False), (2 ** 30 - 64, 64, 8, 1024, False, False)])
def test_launches_of_2_to_the_32_work_items_are_refused(rows, K, N, E, f32, gated):
    """A launch takes fewer than 2^32 work-items: larger ones are refused before they reach it."""
    plan, = plans([(rows, K, N, E, f32, gated)])
    assert plan.groups * plan.threads >= 2 ** 32 and not plan.fits
    assert _linear(rows, K, N, E, f32, gated) == MOE_ERR_UNSUPPORTED


def test_what_fits_stays_below_the_limit():
    """Sizes over the whole range: what is let through is a launch below 2^32 work-items, and what is not passes a
    documented limit."""
    rng = random.Random(1)
    pick = lambda lo, hi: int(round(2 ** rng.uniform(lo, hi)))  # noqa: E731
    sizes = [(min(pick(0, 31), 2 ** 31 - 2 ** 16 - 1), 8 * pick(0, 16.9), 8 * pick(0, 20.9), pick(0, 10), rng.random() < 0.5,
              rng.random() < 0.5) for _ in range(20000)]
    most = 0
    for s, p in zip(sizes, plans(sizes)):
        if p.fits:
            most = max(most, p.groups * p.threads)
            assert p.groups * p.threads < 2 ** 32, s
        else:
            rows, _, N, E = s[:4]
            assert (rows // 32 + E + 1) * (N // 32 + 1) >= 2 ** 27 - 1 or p.groups * p.threads >= 2 ** 32, s
        assert p.split * 8 <= max(s[1] * (4 if s[4] else 2) / 128 + 1, 8), s   # (every part of K has stages)
    assert most > 2 ** 30


def _sizes(test, names):
    """The parametrized sizes of a GPU test."""
    mark, = [m for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names]
    return mark.args[1]


def _take(cases, gated):
    import torch
    return plans([(rows, K, Nw // 2 if gated else Nw, E, dt == torch.float32, gated) for rows, E, K, Nw, k, dt in cases])


@pytest.mark.parametrize("gated", [False, True])
def test_the_gpu_tests_of_every_kernel_take_it(gated):
    """The sizes by which the GPU tests reach each kernel, whole K and K in parts, still do."""
    from tests import test_gpu_bias_experts as t
    got = [(p.kind, p.split > 1) for p in _take(_sizes(t.test_every_kernel, "rows,E,K,Nw,k,dt"), gated)]
    assert got == [("320", False)] * 3 + [("128", False)] * 2 + [("128", True)] + [("320", True)] * 2 + [("64", True)] * 3 + [
        ("128", False), ("128", True), ("32", False)] + [("32", True)] * 3
    tall = _take(_sizes(t.test_every_kernel, "rows,E,K,Nw,k,dt")[:1], gated)[0]
    assert tall.tile_rows == 192   # (320-row tiles made shorter to fill a round)
    few = _sizes(t.test_few_rows, "rows,E,K,Nw,k,dt")
    assert {p.kind for p in _take(few, gated)} == {"few"}
    # 16 weight rows a workgroup up to 128 groups of 32, else 32
    groups = [min(E, rows) * -(-Nw // 32) for rows, E, K, Nw, k, dt in few]
    assert [n <= 128 for n in groups] == [True] * 4 + [False] * 6


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_the_small_sizes_take_64_row_tiles_whole(gated, f32):
    """64 x 64 tiles (bf16) and 32 x 64 (fp32) with K whole are reached by the general sizes."""
    from tests import test_gpu_bias_experts as t
    kinds = {(p.kind, p.split) for p in plans([(rows, K, N, E, f32, gated) for rows, E, K, N in t.SIZES])}
    assert ("32" if f32 else "64", 1) in kinds and ("few", 1) in kinds


def test_the_gpu_tests_of_many_experts_take_tiles():
    import torch
    from tests import test_gpu_many_experts as t
    got = plans([(rows, K, N, E, dt == torch.float32, gated) for rows, E, K, N, dt, gated, _, _ in t.CASES])
    assert [(p.kind, p.split) for p in got] == [c[6:] for c in t.CASES] and all(c[1] > 64 for c in t.CASES)

"""GPU parity of the expert product's tile kernels with more than 64 experts: a lane of the tile search then stands
for a run of experts first, and for an expert of the run that holds the tile second."""
import numpy as np
import pytest
import torch

from tests.test_gpu_bias_experts import BF, F32, _return_cached_blocks, _run_linear  # noqa: F401

pytestmark = pytest.mark.gpu

# (rows, E, K, N, type, gated, kernel, parts of K); which kernel a size takes is pinned by a CPU test
CASES = [
    # a run of two experts, the last of one (65); whole runs (128); runs of five (300) and sixteen (1024)
    (4400, 65, 64, 64, BF, False, "64", 1), (4400, 65, 64, 64, F32, True, "32", 1), (4400, 128, 64, 64, BF, True, "64", 1),
    (4400, 128, 64, 64, F32, False, "32", 1), (11000, 300, 72, 72, BF, False, "64", 1),
    (36000, 1024, 64, 64, BF, False, "64", 1), (40000, 1024, 16, 24, F32, False, "32", 1),
    (36000, 1024, 64, 64, F32, True, "128", 1),
    # wider tiles
    (20000, 128, 128, 512, BF, False, "128", 1), (20000, 128, 128, 512, F32, False, "128", 1),
    (20000, 100, 264, 1032, BF, False, "320", 1), (20000, 128, 128, 512, BF, True, "320", 1),
    # K in parts
    (2152, 65, 2056, 8, BF, False, "64", 4), (2152, 65, 1032, 8, F32, True, "32", 2), (4557, 65, 8200, 72, BF, False, "128", 4)]


def _segments(kind, rows, E):
    if kind == "ragged":      # every third expert without rows, some of one row
        rng = np.random.default_rng(E)
        n = rng.integers(0, 2 * rows // E, E) * (np.arange(E) % 3 > 0)
        n[4::9] = 1
    elif kind == "last":      # all rows on the last expert
        n = np.zeros(E, int)
        n[-1] = rows
    else:                     # "runs": whole runs of experts without rows; rows before the first and behind the last expert
        run = (E + 63) // 64
        n = np.full(E, 3) * (np.arange(E) // run % 4 == 2)
        n[E // 2] += rows // 3
    off = np.concatenate([[0], np.cumsum(n)])
    if kind == "runs":
        off = off + 5
    return torch.from_numpy(np.minimum(off, rows)).to(torch.int32)


@pytest.mark.parametrize("kind", ["ragged", "last", "runs"])
@pytest.mark.parametrize("rows,E,K,N,dt,gated,kernel,parts", CASES)
def test_many_experts(rows, E, K, N, dt, gated, kernel, parts, kind):
    _run_linear(rows, E, K, N, dt, gated=gated, residual=gated, k=0 if K < 100 else 3, seed=rows,
                offsets=_segments(kind, rows, E))


def test_the_largest_launch_is_complete():
    """Rows just below the refused ones (2^32 work-items): the first, the last and those between are computed."""
    import combine_grouped_gemm_amd as moe
    from tests.gpu_util import say, sync
    rows = 2 ** 30 - 1024      # 2^24 - 16 tiles of 64 rows, 256 lanes each
    say(f"linear rows={rows} K=8 N=8")
    dev = torch.device("cuda:0")
    at = torch.tensor([0, 63, 64, 2 ** 28 + 5, 2 ** 29, rows // 3 * 2, rows - 65, rows - 64, rows - 1], device=dev)
    a = torch.zeros(rows, 8, dtype=BF, device=dev)
    rand = lambda seed, *shape: torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dev)  # noqa: E731
    a[at] = rand(1, len(at), 8).to(BF)
    w, b = rand(2, 1, 8, 8).to(BF), rand(3, 1, 8)
    out, _ = moe.moe_expert_linear(a, w, bias=b)
    want = (a[at].double() @ w[0].double().T + b.double()).float().to(BF)
    got, plain = out[at], b.to(BF)
    others = (out[1:63] == plain).all() & (out[-63:-1] == plain).all() & (out[2 ** 29 + 1:2 ** 29 + 10 ** 6] == plain).all()
    sync()
    assert others.item()
    # 8 exact products and a bias in fp32, each addition off by 2^-24 of the magnitudes' sum at most; then a rounding on
    # either side, half a step each
    mag = a[at].double().abs() @ w[0].double().abs().T + b.double().abs()
    assert ((got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 20 * 2.0 ** -24 * mag).all()
    del a, out
    torch.cuda.empty_cache()

"""GPU parity of the router's gradients from a dense logit gradient with float64 products."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
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


def _t(shape, seed, dt, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale).to(torch.float32).to(dt)


def _bound(mag, terms, ref, dt):
    """fp32 sums of `terms` products (bf16 products are exact; fp32 ones round inside an FMA), in any
    order, doubled for second order; one rounding to dt."""
    b = 2 * (terms + 2) * U32 * mag
    return b + torch.finfo(dt).eps / 2 * (np.abs(ref) + b) + 1e-37


def _wgrad(dz, x, dw_dtype):
    dw = moe.moe_router_dense_wgrad(dz.to(DEV), x.to(DEV), dw_dtype=dw_dtype)
    sync()
    a, b = f64(dz), f64(x)
    ref = a.T @ b
    assert dw.dtype == dw_dtype and np.all(np.abs(f64(dw) - ref) <= _bound(np.abs(a).T @ np.abs(b), len(a) + 64, ref, dw_dtype))


def _dgrad(dz, w, rest):
    dx = moe.moe_router_dense_dgrad(dz.to(DEV), w.to(DEV), rest=None if rest is None else rest.to(DEV))
    sync()
    a, b = f64(dz), f64(w)
    ref, mag = a @ b, np.abs(a) @ np.abs(b)
    if rest is not None:
        ref, mag = ref + f64(rest), mag + np.abs(f64(rest))
    assert np.all(np.abs(f64(dx) - ref) <= _bound(mag, len(b) + 1, ref, w.dtype))


# one token; tails of every tile size in every direction; odd expert counts; whole stages and not
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,H", [(1, 1, 8), (1, 256, 1024), (3, 8, 136), (31, 60, 520), (33, 64, 128), (100, 13, 264),
                                   (257, 72, 384), (300, 128, 640), (129, 130, 136), (65, 256, 256), (500, 201, 200),
                                   (1000, 1000, 136), (70, 1021, 512), (2050, 16, 1160)])
def test_sizes(N, E, H, dt):
    say(f"dense router gradients N={N} E={E} H={H} {dt}")
    dz, x, w = _t((N, E), 1, dt, 2.0 ** -9), _t((N, H), 2, dt), _t((E, H), 3, dt, 0.02)
    _wgrad(dz, x, torch.float32)
    _wgrad(dz, x, torch.bfloat16)
    _dgrad(dz, w, None)
    _dgrad(dz, w, _t((N, H), 4, dt, 0.01))


# the tiles and ranges of large batches: 16-byte dz rows and others, one and several row tiles, tails in every
# direction
@pytest.mark.parametrize("N,E,H", [(4200, 60, 8320), (4200, 64, 8200), (4100, 203, 8200), (4100, 136, 8200),
                                   (8200, 256, 7176), (8200, 250, 7176), (8192, 24, 7168), (3000, 512, 1032)])
def test_large_sizes(N, E, H):
    say(f"dense router gradients N={N} E={E} H={H}")
    dt = torch.bfloat16
    dz, w = _t((N, E), 1, dt, 2.0 ** -9), _t((E, H), 3, dt, 0.02)
    x = _t((N, H), 2, dt)
    _wgrad(dz, x, torch.float32)
    _dgrad(dz, w, x)


def test_many_ranges_and_repeats():
    """A batch cut into many token ranges, and the same bits on every call."""
    say("dense router gradients: token ranges")
    dz, x = _t((9000, 8), 5, torch.bfloat16, 2.0 ** -9), _t((9000, 256), 6, torch.bfloat16)
    _wgrad(dz, x, torch.float32)
    a = [moe.moe_router_dense_wgrad(dz.to(DEV), x.to(DEV)) for _ in range(3)]
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


def test_nan_stays_in_its_row():
    """A token's NaN or infinity reaches its own dx row and the columns it multiplies, nothing else:
    not the neighbouring rows that a tile reads past a row's end, nor stored columns past the data."""
    say("dense router gradients: NaN")
    for E in (8, 40, 72, 60):
        N, H = 70, 200
        dz, w = _t((N, E), 7, torch.bfloat16, 2.0 ** -9), _t((E, H), 8, torch.bfloat16, 0.02)
        x = _t((N, H), 9, torch.bfloat16)
        clean = moe.moe_router_dense_dgrad(dz.to(DEV), w.to(DEV))
        dz[17, :] = float("nan")
        dz[33, 0] = float("inf")
        got = moe.moe_router_dense_dgrad(dz.to(DEV), w.to(DEV))
        sync()
        keep = [t for t in range(N) if t not in (17, 33)]
        assert torch.isnan(got[17]).all() and torch.equal(got[keep], clean[keep])
        dz2 = _t((N, E), 7, torch.bfloat16, 2.0 ** -9)
        dw = moe.moe_router_dense_wgrad(dz2.to(DEV), x.to(DEV))
        dz2[5, 3] = float("nan")
        x[9, 100] = float("nan")
        got = moe.moe_router_dense_wgrad(dz2.to(DEV), x.to(DEV))
        sync()
        bad = torch.zeros(E, H, dtype=torch.bool)
        bad[3, :] = True
        bad[:, 100] = True
        assert torch.isnan(got.cpu()[bad]).all() and torch.equal(got.cpu()[~bad], dw.cpu()[~bad])


def test_in_place_rest_unaligned_dz_and_no_tokens():
    say("dense router gradients: in place, unaligned dz, no tokens")
    N, E, H = 200, 64, 512
    dz, w, rest = _t((N, E), 10, torch.bfloat16, 2.0 ** -9), _t((E, H), 11, torch.bfloat16, 0.02), _t((N, H), 12, torch.bfloat16)
    want = moe.moe_router_dense_dgrad(dz.to(DEV), w.to(DEV), rest=rest.to(DEV))
    buf = rest.to(DEV)
    moe.moe_router_dense_dgrad(dz.to(DEV), w.to(DEV), rest=buf, dx=buf)
    off = torch.empty(N * E + 1, dtype=torch.bfloat16, device=DEV)[1:].view(N, E)
    off.copy_(dz)
    got = moe.moe_router_dense_dgrad(off, w.to(DEV), rest=rest.to(DEV))
    sync()
    assert torch.equal(buf, want) and torch.equal(got, want)
    assert torch.equal(moe.moe_router_dense_wgrad(off, rest.to(DEV)), moe.moe_router_dense_wgrad(dz.to(DEV), rest.to(DEV)))
    dw = torch.full((E, H), 3.0, device=DEV)
    moe.moe_router_dense_wgrad(dz[:0].to(DEV), rest[:0].to(DEV), dw=dw)
    assert moe.moe_router_dense_dgrad(dz[:0].to(DEV), w.to(DEV)).shape == (0, H)
    sync()
    assert not dw.any()


def test_captured():
    """Both in one captured graph, replayed on new inputs with eager work between."""
    say("dense router gradients: graph")
    N, E, H = 600, 40, 256
    dz, x = _t((N, E), 13, torch.bfloat16, 2.0 ** -9).to(DEV), _t((N, H), 14, torch.bfloat16).to(DEV)
    w = _t((E, H), 15, torch.bfloat16, 0.02).to(DEV)
    ws = torch.empty(moe.moe_workspace_bytes(moe.MOE_OP_ROUTER_WGRAD, N, H, 0, E, 0, moe.MOE_BF16) + 256,
                     dtype=torch.uint8, device=DEV)
    dw, dx = moe.moe_router_dense_wgrad(dz, x, ws=ws), moe.moe_router_dense_dgrad(dz, w, rest=x)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_router_dense_wgrad(dz, x, dw=dw, ws=ws)
        moe.moe_router_dense_dgrad(dz, w, rest=x, dx=dx)
    for _ in range(3):
        dz.normal_()
        x.normal_()
        ws.fill_(255)
        graph.replay()
        sync()
        assert torch.equal(dw, moe.moe_router_dense_wgrad(dz, x)) and torch.equal(dx, moe.moe_router_dense_dgrad(dz, w, rest=x))

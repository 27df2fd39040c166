"""The logit gradient in three bf16 planes (an fp32 value each): what the balance loss's gradient writes, and the dense
router gradients that read it, against float64 products of the fp32 gradient."""
import numpy as np
import pytest
import torch

import combine_grouped_gemm_amd as moe
from tests.gpu_util import f64, say, sync
from tests.test_gpu_balance import _case, _dev, _loss, _return_cached_blocks  # noqa: F401
from tests.test_gpu_router_dense import DEV, _bound, _t

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _planes(dz):
    """fp32 dz as three bf16 tensors, each the rounding of what the ones before it leave."""
    out, r = [], dz.float()
    for _ in range(3):
        out.append(r.to(BF))
        r = r - out[-1].float()
    return torch.stack(out)


def _gradient(N, E, seed):
    """fp32 gradients as a training step has them: a few large entries beside small ones, every digit in use."""
    rng = np.random.default_rng(seed)
    dz = rng.normal(size=(N, E)) * 2.0 ** -20
    dz[np.arange(N), rng.integers(0, E, N)] += rng.normal(size=N) * 2.0 ** -8
    return torch.from_numpy(dz.astype(np.float32))


def _wgrad(dz, x, dw_dtype):
    dw = moe.moe_router_dense_wgrad(_planes(dz).to(DEV), x.to(DEV), dw_dtype=dw_dtype)
    sync()
    a, b = f64(dz), f64(x)
    ref = a.T @ b
    # (three terms a product, whose sizes add up to at most 1 + 2^-7 of it: inside the bound's doubling)
    assert dw.dtype == dw_dtype and np.all(np.abs(f64(dw) - ref) <= _bound(np.abs(a).T @ np.abs(b), 3 * len(a) + 64, ref,
                                                                          dw_dtype))


def _dgrad(dz, w, rest):
    dx = moe.moe_router_dense_dgrad(_planes(dz).to(DEV), w.to(DEV), rest=None if rest is None else rest.to(DEV))
    sync()
    a, b = f64(dz), f64(w)
    ref, mag = a @ b, np.abs(a) @ np.abs(b)
    if rest is not None:
        ref, mag = ref + f64(rest), mag + np.abs(f64(rest))
    assert np.all(np.abs(f64(dx) - ref) <= _bound(mag, 3 * len(b) + 1, ref, BF))


@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (7, 60, 4), (300, 8, 2), (129, 13, 3), (500, 256, 8), (40, 333, 8), (17, 1000, 8),
                                   (9001, 160, 6)])
def test_planes_of_the_gradient(N, E, k):
    """The planes' sum is the fp32 gradient bit for bit, the first plane the bf16 one."""
    say(f"planes of the logit gradient N={N} E={E} k={k}")
    c = _case(N, E, k, S=3, seed=N, mask=True, bias=True)
    _, counts, _, tokens = _loss(c, 0.03)
    rng = np.random.default_rng(1)
    g = dict(topk_gate=_dev(rng.random((N, k)).astype(np.float32)), d_gate=_dev(rng.normal(size=(N, k)).astype(np.float32)))
    for kw in ({}, g):
        a = (_dev(c["z"]), _dev(c["topk_idx"]), 0.03, counts, tokens)
        kw = dict(kw, bias=_dev(c["bias"]), seq_start=_dev(c["seq_start"]), token_mask=_dev(c["mask"]))
        f32, bf = (moe.moe_balance_loss_backward(*a, **kw, dz_dtype=t) for t in (torch.float32, BF))
        pl = moe.moe_balance_loss_backward(*a, **kw, planes=True)
        # (rows off a 16-byte boundary take other lanes, whose sums have another order: their own fp32 gradient)
        f32_off = torch.full((N * E + 1,), 7.0, device=DEV)[1:].view(N, E)
        pl_off = torch.full((3 * N * E + 1,), 7.0, dtype=BF, device=DEV)[1:].view(3, N, E)
        moe.moe_balance_loss_backward(*a, **kw, dz=f32_off)
        moe.moe_balance_loss_backward(*a, **kw, dz=pl_off)
        sync()
        assert torch.equal(pl.double().sum(0), f32.double()) and torch.equal(pl[0], bf)
        assert torch.equal(pl_off.double().sum(0), f32_off.double())


# one token; tails of every tile size in every direction; odd expert counts; whole stages and not; token ranges
@pytest.mark.parametrize("N,E,H", [(1, 1, 8), (1, 256, 1024), (3, 8, 136), (31, 60, 520), (33, 64, 128), (100, 13, 264),
                                   (257, 72, 384), (300, 128, 640), (129, 130, 136), (65, 256, 256), (500, 201, 200),
                                   (1000, 1000, 136), (70, 1021, 512), (2050, 16, 1160), (96, 32, 256)])
def test_sizes(N, E, H):
    say(f"dense router gradients, planes N={N} E={E} H={H}")
    dz, x, w = _gradient(N, E, 1), _t((N, H), 2, BF), _t((E, H), 3, BF, 0.02)
    _wgrad(dz, x, torch.float32)
    _wgrad(dz, x, BF)
    _dgrad(dz, w, None)
    _dgrad(dz, w, _t((N, H), 4, BF, 2.0 ** -14))


@pytest.mark.parametrize("N,E,H", [(4200, 60, 8320), (4100, 136, 8200), (8200, 256, 7176), (8200, 250, 7176), (8192, 24, 7168),
                                   (3000, 512, 1032)])
def test_large_sizes(N, E, H):
    say(f"dense router gradients, planes N={N} E={E} H={H}")
    dz, w, x = _gradient(N, E, 1), _t((E, H), 3, BF, 0.02), _t((N, H), 2, BF)
    _wgrad(dz, x, torch.float32)
    _dgrad(dz, w, x)


def test_nan_stays_in_its_row():
    """A token's NaN or infinity reaches its own dx row and the columns it multiplies, nothing else."""
    say("dense router gradients, planes: NaN")
    for E in (8, 40, 72, 60):
        N, H = 70, 200
        dz, w, x = _gradient(N, E, 7), _t((E, H), 8, BF, 0.02), _t((N, H), 9, BF)
        clean = moe.moe_router_dense_dgrad(_planes(dz).to(DEV), w.to(DEV))
        dw = moe.moe_router_dense_wgrad(_planes(dz).to(DEV), x.to(DEV))
        bad = dz.clone()
        bad[17, :] = float("nan")
        bad[33, 0] = float("inf")
        got = moe.moe_router_dense_dgrad(_planes(bad).to(DEV), w.to(DEV))
        sync()
        keep = [t for t in range(N) if t not in (17, 33)]
        assert torch.isnan(got[17]).all() and not torch.isfinite(got[33]).any() and torch.equal(got[keep], clean[keep])
        bad = dz.clone()
        bad[5, 3] = float("nan")
        x[9, 100] = float("nan")
        got = moe.moe_router_dense_wgrad(_planes(bad).to(DEV), x.to(DEV))
        sync()
        hit = torch.zeros(E, H, dtype=torch.bool)
        hit[3, :] = True
        hit[:, 100] = True
        assert torch.isnan(got.cpu()[hit]).all() and torch.equal(got.cpu()[~hit], dw.cpu()[~hit])


def test_in_place_rest_unaligned_planes_and_no_tokens():
    say("dense router gradients, planes: in place, unaligned, no tokens")
    N, E, H = 200, 64, 512
    dz, w, rest = _planes(_gradient(N, E, 10)).to(DEV), _t((E, H), 11, BF, 0.02).to(DEV), _t((N, H), 12, BF).to(DEV)
    want = moe.moe_router_dense_dgrad(dz, w, rest=rest)
    buf = rest.clone()
    moe.moe_router_dense_dgrad(dz, w, rest=buf, dx=buf)
    off = torch.empty(3 * N * E + 1, dtype=BF, device=DEV)[1:].view(3, N, E)
    off.copy_(dz)
    got = moe.moe_router_dense_dgrad(off, w, rest=rest)
    sync()
    assert torch.equal(buf, want) and torch.equal(got, want)
    assert torch.equal(moe.moe_router_dense_wgrad(off, rest), moe.moe_router_dense_wgrad(dz, rest))
    dw = torch.full((E, H), 3.0, device=DEV)
    moe.moe_router_dense_wgrad(dz[:, :0].contiguous(), rest[:0], dw=dw)
    assert moe.moe_router_dense_dgrad(dz[:, :0].contiguous(), w).shape == (0, H)
    sync()
    assert not dw.any()


def test_captured_and_on_another_stream():
    """Gradient in planes and both products in one captured graph, replayed on new inputs with eager work between;
    the same calls on a stream of their own."""
    say("dense router gradients, planes: graph and stream")
    N, E, H, k = 600, 40, 256, 2
    z, x = torch.randn(N, E, device=DEV), _t((N, H), 14, BF).to(DEV)
    idx = torch.randint(0, E, (N, k), device=DEV, dtype=torch.int32)
    w = _t((E, H), 15, BF, 0.02).to(DEV)

    def step(**out):
        loss, counts, _, tokens = moe.moe_balance_loss(z, idx, 0.1, out=out.get("bal"))
        dz = moe.moe_balance_loss_backward(z, idx, 0.1, counts, tokens, planes=True, dz=out.get("dz"))
        return dz, moe.moe_router_dense_wgrad(dz, x, dw=out.get("dw")), moe.moe_router_dense_dgrad(dz, w, rest=x, dx=out.get("dx"))

    bal = moe.moe_balance_loss(z, idx, 0.1)
    dz, dw, dx = step(bal=bal)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bal=bal, dz=dz, dw=dw, dx=dx)
    side = torch.cuda.Stream()
    for _ in range(3):
        z.normal_()
        x.normal_()
        graph.replay()
        sync()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = step()
        sync()
        assert all(torch.equal(a, b) for a, b in zip((dz, dw, dx), want))

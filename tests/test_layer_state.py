"""What the layer holds and keeps between calls, on the CPU: refused calls change nothing, buffers of the balance loss
are bounded (no GPU needed: nothing here is enqueued)."""
import pytest
import torch

import combine_grouped_gemm_amd as moe
import combine_grouped_gemm_amd.layer as layer_module
from combine_grouped_gemm_amd.layer import MoELayer

STATE = ("keep8", "kept_x", "kept_au", "save_au", "au_saved", "au_all", "balance", "balance_args")


def _layer(N=6, H=128, E=4, k=2, I=128, dtype="bf16", shared=False, w_r=True, **kw):
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    s = dict(shared_w13=torch.zeros(1, 2 * I, H, dtype=t), shared_w2=torch.zeros(1, H, I, dtype=t)) if shared else {}
    return MoELayer(N, H, E, k, I, dtype, torch.zeros(E, 2 * I, H, dtype=t), torch.zeros(E, H, I, dtype=t),
                    w_r=torch.zeros(E, H, dtype=t) if w_r else None, **s, **kw)


def _refused(layer, x, **kw):
    before = {n: getattr(layer, n) for n in STATE}
    with pytest.raises(ValueError):
        layer.forward(x, **kw)
    assert all(getattr(layer, n) is v for n, v in before.items())


@pytest.mark.parametrize("case", [dict(dtype="f32"), dict(gather=False), dict(shared=True, fuse_shared=False),
                                  dict(H=160), dict(H=136), dict(I=96), dict(E=1024, I=128)])
def test_layers_that_cannot_keep_8_bits_refuse_and_stay_as_they_were(case):
    layer = _layer(**case)
    layer.save_au = layer.au_saved = False
    _refused(layer, torch.zeros(6, layer.H, dtype=layer.act_dtype), save_for_backward="mxfp8")


def test_refused_forwards_leave_the_last_one_in_place():
    """A forward that is refused does not change what the next backward goes by."""
    for shared in (False, True):
        layer = _layer(shared=shared)
        layer.balance, layer.balance_args = (1, 2, 3, 4), dict(z=0)
        x = torch.zeros(6, 128, dtype=torch.bfloat16)
        _refused(layer, x, save_for_backward="fp8")
        _refused(layer, x, token_mask=torch.ones(6, dtype=torch.uint8))
        _refused(layer, torch.zeros(5, 128, dtype=torch.bfloat16), save_for_backward="mxfp8")
        _refused(layer, x.float(), save_for_backward="mxfp8")
        for bad in (dict(seq_start=torch.zeros(3, dtype=torch.int64)), dict(seq_start=torch.zeros(0, dtype=torch.int32)),
                    dict(seq_start=torch.zeros(1, dtype=torch.int32)), dict(seq_start=torch.zeros(65537, dtype=torch.int32)),
                    dict(seq_start=torch.zeros(2, 2, dtype=torch.int32)),
                    dict(token_mask=torch.ones(5, dtype=torch.uint8)), dict(token_mask=torch.ones(6))):
            _refused(layer, x, balance_alpha=0.1, save_for_backward="mxfp8", **bad)
    layer = _layer(w_r=False)
    _refused(layer, torch.zeros(6, 128, dtype=torch.bfloat16), save_for_backward="mxfp8")


def test_balance_buffers_are_bounded(monkeypatch):
    """Batches of ever other sequence counts: the buffers are those of a few capacities, each call's views fit its
    count and the workspace is large enough, and a count that came before finds its buffers again."""
    calls = []

    def record(z, idx, alpha, bias=None, seq_start=None, token_mask=None, out=None, ws=None):
        S = 1 if seq_start is None else seq_start.numel() - 1
        need = moe.moe_workspace_bytes(moe.MOE_OP_BALANCE_LOSS, z.shape[0], 0, 0, z.shape[1], S, 0)
        assert [tuple(t.shape) for t in out] == [(1,), (S, 4), (S, 4), (S,)] and ws.numel() >= need
        assert all(t.is_contiguous() for t in out)
        calls.append((S, tuple(t.data_ptr() for t in out) + (ws.data_ptr(),)))
        return out

    monkeypatch.setattr(layer_module, "moe_balance_loss", record)
    layer = _layer(N=700)
    z = torch.zeros(700, 4)
    for S in [None, *range(1, 1200), 65535, *range(1, 40)]:
        seq = None if S is None else torch.zeros(S + 1, dtype=torch.int32)
        layer.balance_step(z, 0.1, seq)
    assert len(layer.balance_bufs) <= 17
    first = {}
    for S, at in calls:
        assert first.setdefault(S, at) == at


def test_combine_alone_goes_by_its_own_arguments(monkeypatch):
    """A combine call beside a forward (a step taken alone) drops out and adds what it is given, not what the last
    forward was; a residual needs no generator's state."""
    calls = []
    monkeypatch.setattr(layer_module, "moe_combine", lambda *a, **kw: calls.append(("plain",)))
    monkeypatch.setattr(layer_module, "moe_combine_dropout",
                        lambda eo, pos, g, p, rng, sh=None, res=None, y=None, k=None: calls.append((p, rng, res)))
    layer = _layer()
    res, rng = torch.zeros(6, 128, dtype=torch.bfloat16), torch.tensor([1, 2])
    layer.combine(res)
    assert calls[-1][0] == 0.0 and calls[-1][1].shape == (2,) and calls[-1][2] is res
    layer.drop_p, layer.rng_used = 0.25, torch.tensor([3, 4])     # as a forward with dropout leaves them
    layer.combine()
    assert calls[-1] == ("plain",)
    layer.combine(res)
    assert calls[-1][0] == 0.0 and calls[-1][2] is res
    layer.combine(res, 0.5, rng)
    assert calls[-1][0] == 0.5 and calls[-1][1] is rng and calls[-1][2] is res
    before = len(calls)
    for bad in (dict(dropout=0.5), dict(dropout=1.5, rng=rng), dict(dropout=-0.5, rng=rng), dict(dropout=float("nan"), rng=rng),
                dict(residual=res.float()), dict(residual=res[:5])):
        with pytest.raises(ValueError):
            layer.combine(**bad)
    assert len(calls) == before and layer.drop_p == 0.25


def test_tensors_that_the_launches_would_refuse_leave_the_last_forward_in_place():
    """Strided or unaligned tokens, logits and residuals are refused before anything changes, in either layer."""
    from combine_grouped_gemm_amd.layer import BiasedMoELayer
    bf = torch.bfloat16
    biased = BiasedMoELayer(6, 128, 4, 2, 128, torch.zeros(4, 128, 128, dtype=bf), torch.zeros(4, 128, 128, dtype=bf),
                            w_r=torch.zeros(4, 128, dtype=bf))
    x = torch.zeros(6, 128, dtype=bf)
    strided, shifted = torch.zeros(6, 256, dtype=bf)[:, ::2], torch.zeros(6 * 128 + 1, dtype=bf)[1:].view(6, 128)
    assert strided.shape == shifted.shape == x.shape and shifted.data_ptr() % 16
    for layer, names in ((_layer(), STATE + ("drop_p", "rng_used")), (biased, ("drop_p", "rng_used", "pre", "saved"))):
        layer.drop_p, layer.rng_used = 0.125, torch.tensor([3, 4])
        layer.saved = layer.save_au = True
        before = {n: getattr(layer, n) for n in names}
        for bad in (dict(x=strided), dict(x=shifted), dict(x=x, residual=strided), dict(x=x, residual=shifted),
                    dict(x=x, z=torch.zeros(6, 8)[:, ::2])):
            with pytest.raises(ValueError):
                layer.forward(**bad, dropout=0.5, rng=torch.tensor([5, 6]))
            assert all(getattr(layer, n) is v for n, v in before.items()) and layer.rng_used.tolist() == [3, 4]


def test_biased_layer_refuses_strided_weights():
    from combine_grouped_gemm_amd.layer import BiasedMoELayer
    bf = torch.bfloat16
    good = dict(N=6, H=128, E=4, k=2, I=64, w1=torch.zeros(4, 64, 128, dtype=bf), w2=torch.zeros(4, 128, 64, dtype=bf),
                b1=torch.zeros(4, 64), b2=torch.zeros(4, 128, dtype=bf), w_r=torch.zeros(4, 128, dtype=bf),
                bias=torch.zeros(4))
    BiasedMoELayer(**good)
    for n in ("w1", "w2", "b1", "b2", "w_r", "bias"):
        t = good[n]
        with pytest.raises(ValueError, match=n):
            BiasedMoELayer(**{**good, n: torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]})

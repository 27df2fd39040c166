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

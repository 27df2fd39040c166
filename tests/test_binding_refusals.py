"""Refusals of the training operators' Python entry points that need no GPU: tensors on another device, sequence
starts that name no sequence."""
import pytest
import torch

import combine_grouped_gemm_amd as moe


def test_workspaces_of_another_device_are_refused():
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="meta")
    z, idx = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32)
    x, off = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    w, ss = torch.zeros(2, 256, 128, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    for f in (lambda: moe.moe_balance_loss(z, idx, 0.1, ws=ws), lambda: moe.moe_router_dense_wgrad(z, torch.zeros(6, 8), ws=ws),
              lambda: moe.moe_expert_gate_up_mxfp8(x, ss, 2, off, w, ws=ws)):
        with pytest.raises(ValueError, match="ws is on meta"):
            f()


def test_sequence_starts_that_name_no_sequence():
    z, idx = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32)
    c, t = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for n in (0, 1):
        seq = torch.zeros(n, dtype=torch.int32)
        with pytest.raises(ValueError, match="seq_start"):
            moe.moe_balance_loss(z, idx, 0.1, seq_start=seq)
        with pytest.raises(ValueError, match="seq_start"):
            moe.moe_balance_loss_backward(z, idx, 0.1, c, t, seq_start=seq)


def test_row_counts_below_zero():
    x, off = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    w, ss = torch.zeros(2, 256, 128, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="rows"):
        moe.moe_expert_gate_up_mxfp8(x, ss, 2, off, w, rows=-1)


FAKE = 4096   # never dereferenced on these paths


def test_planes_of_a_logit_gradient():
    """Three planes of dz go with bf16 operands only, and no other entry point takes their type."""
    bf = torch.bfloat16
    dz, x, w = torch.zeros(3, 6, 4, dtype=bf), torch.zeros(6, 8, dtype=bf), torch.zeros(4, 8, dtype=bf)
    for bad in (dict(dz=dz[:2]), dict(dz=dz.float()), dict(dz=dz[:, :5]), dict(x=x.float())):
        with pytest.raises(ValueError, match="must|goes"):
            moe.moe_router_dense_wgrad(**{**dict(dz=dz, x=x), **bad})
    for bad in (dict(dz=dz[:2]), dict(dz=dz.float()), dict(dz=dz[:, :, :3]), dict(w_r=w.float()), dict(rest=x.float())):
        with pytest.raises(ValueError, match="must|goes"):
            moe.moe_router_dense_dgrad(**{**dict(dz=dz, w_r=w), **bad})
    z, idx = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32)
    c, t = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dz[:2], dz.float(), torch.zeros(3, 6, 5, dtype=bf)):
        with pytest.raises(ValueError, match="dz"):
            moe.moe_balance_loss_backward(z, idx, 0.1, c, t, dz=bad)
    with pytest.raises(ValueError, match="dz"):
        moe.moe_balance_loss_backward(z, idx, 0.1, c, t, dz=torch.zeros(6, 4), planes=True)
    L, X3 = moe.lib(), moe.MOE_BF16X3
    un = moe.MOE_ERR_UNSUPPORTED
    assert L.moe_router_dense_wgrad(FAKE, FAKE, X3, 4096, 16, 512, FAKE, X3, FAKE, 1 << 30, None) == un
    assert L.moe_router_dense_wgrad(FAKE, FAKE, X3, 4096, 16, 516, FAKE, moe.MOE_F32, FAKE, 1 << 30, None) == un
    need = moe.moe_workspace_bytes(moe.MOE_OP_ROUTER_WGRAD, 4096, 512, 0, 16, 0, X3)
    assert need > 0 and need % (16 * 512 * 4) == 0
    assert L.moe_router_dense_wgrad(FAKE, FAKE, X3, 4096, 16, 512, FAKE, moe.MOE_F32, FAKE, need - 1, None) == moe.MOE_ERR_WORKSPACE
    assert L.moe_router_dense_dgrad(None, None, X3, 0, 16, 512, None, None, None) == moe.MOE_OK
    assert L.moe_router_dense_dgrad(FAKE, FAKE + 8, X3, 9, 16, 512, None, FAKE, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_quantize_mxfp8(FAKE, X3, 10, 96, FAKE, FAKE, None) == un
    assert L.moe_dequantize_mxfp8(FAKE, FAKE, 10, 96, 1, None, 0, FAKE, X3, None) == un
    assert L.moe_swiglu_backward_mxfp8(FAKE, FAKE, FAKE, X3, 10, 96, 10, None, None, FAKE, FAKE, None, None) == un
    assert L.moe_router_logits(FAKE, X3, 4, 256, FAKE, 8, FAKE, FAKE, 1 << 20, None) == un
    assert L.moe_permute(FAKE, X3, 4, 256, 2, FAKE, FAKE, X3, None, None) == un
    for N in (0, 1, 63, 8192, 2 ** 24 - 1, 2 ** 31 - 1):
        for E in (1, 7, 8, 160, 1024):
            for H in (8, 7168, 2 ** 20):
                assert 0 <= moe.moe_workspace_bytes(moe.MOE_OP_ROUTER_WGRAD, N, H, 0, E, 0, X3) <= 1024 * 4 * E * H + 255

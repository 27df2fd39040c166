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

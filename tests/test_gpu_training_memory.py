"""What the layer holds in device memory after the steps of either kind."""
import pytest
import torch

import workload as w
from tests.gpu_util import say, sync
from tests.test_gpu_balance import _return_cached_blocks  # noqa: F401
from tests.test_gpu_training_step import SMALL, _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["dsv3_small", "mixtral_small"])
def test_device_bytes_of_the_kept_activations(name):
    """An 8-bit forward adds the codes of the tokens and of all pre-activation rows, 33/32 byte a value, and nothing
    else; a bf16 one two bytes a pre-activation (where the layer keeps them); h and the expert outputs stay the layer's
    in both; what both kinds of step allocated stays.  The 8-bit backward holds a bf16 copy of the tokens where the
    shared expert or the router needs one, and no bf16 pre-activations."""
    cfg = SMALL[name]
    say(f"device bytes {name}")
    inp, layer, dy = _layer(cfg)
    N, H, I, rows = cfg.N, cfg.H, cfg.I, cfg.N * cfg.k + (cfg.N if layer.fuse else 0)
    codes = (N * H + rows * 2 * I) * 33 // 32
    fixed = layer.device_bytes()["activations"]
    layer.forward(inp["x"], inp["z"], save_for_backward="mxfp8")
    assert layer.device_bytes()["activations"] == fixed + codes
    if layer.fuse:   # (expert outputs and h are among the fixed ones)
        assert fixed > rows * (H + I) * 2
    layer.backward(None, dy)
    sync()
    eight = layer.device_bytes()["backward"]
    layer.forward(inp["x"], inp["z"], save_for_backward=True)
    both = layer.device_bytes()["activations"]
    assert both == fixed + codes + (rows * 2 * I * 2 if layer.fuse else 0)
    inp, other, dy = _layer(cfg)
    other.forward(inp["x"], inp["z"], save_for_backward=True)
    other.backward(inp["x"], dy)
    sync()
    assert other.device_bytes()["activations"] == both - codes
    # (bf16: the buffers of recomputed pre-activations, which the layer has in every mode)
    pre = cfg.N * cfg.k * 2 * I * 2 + (N * 2 * I * 2 if layer.shared else 0)
    assert other.device_bytes()["backward"] - eight == pre - N * H * 2


@pytest.mark.parametrize("counts", [(3, 5, 4, 8, 7, 2)])
def test_device_bytes_of_changing_sequence_counts(counts):
    """Batches of other sequence counts take the buffers of the next power of two, once."""
    cfg = w.CONFIGS["dsv3_bf16"].scaled(N=256, H=256, E=32, k=4, I=128, n_group=4, topk_group=2)
    say(f"device bytes of sequence counts {counts}")
    inp, layer, _ = _layer(cfg)
    seen = []
    for S in counts:
        seq = torch.linspace(0, cfg.N, S + 1).to(torch.int32).cuda()
        layer.forward(inp["x"], inp["z"], balance_alpha=0.1, seq_start=seq)
        sync()
        assert layer.balance[1].shape == (S, cfg.E) and int(layer.balance[1].sum()) == cfg.N * cfg.k
        seen.append(sum(layer.device_bytes().values()))
    assert seen[0] < seen[1] and seen[1] == seen[2] == seen[3] == seen[4] < seen[5]

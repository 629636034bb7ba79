"""The block norms' gradient where an input leaves the numbers' range but its
result does not."""
import pytest
import torch

import mixture_experts_layer_61_b200 as moe
import train_ref as R
from test_gpu_train_rows import gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate_mode", [0, 1, 2])
@pytest.mark.parametrize("H", [264, 4104, 8192])
def test_without_a_norm_after_the_block_dy_does_not_depend_on_y(H, gate_mode, dtype):
    """h = s r + gate y: dy = gate dh, finite where y is not."""
    T = 5
    g = gen(H)
    y, dh = randn(T, H, g=g, dtype=dtype), randn(T, H, g=g, dtype=dtype)
    y[1, 3], y[1, H - 1], y[2, 8], y[4] = float("inf"), float("-inf"), float("nan"), float("inf")
    gate = None if gate_mode == 0 else randn(*((H,) if gate_mode == 1 else (T, H)), g=g, dtype=dtype)
    nc = moe.norm_config(T, H, res_scale=0.5, gate_mode=gate_mode, dtype=dtype)
    ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
    r = moe.block_norm_grad(nc, ws, dh=dh, y=y, gate=gate)
    ref = R.f64(dh) if gate is None else R.f64(gate) * R.f64(dh)
    # one fp32 product and one rounding (none without a gate)
    R.close(r["dy"], ref, (R.HALF[dtype] + 2.0 ** -23) * ref.abs(), "dy")
    assert torch.equal(r["dresidual"], (0.5 * dh.float()).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zero_tokens_write_zeros_beside_infinite_weights(dtype):
    H = 264
    nc = moe.norm_config(0, H, gate_mode=moe.GATE_CHANNEL, dtype=dtype)
    w = torch.ones(H, dtype=dtype, device="cuda")
    w[0], w[1], w[2] = float("inf"), float("-inf"), float("nan")
    e = torch.empty((0, H), dtype=dtype, device="cuda")
    ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
    r = moe.block_norm_grad(nc, ws, h=e, dh=e, dn=e, y=e, w_post=w, gate=w, w_next=w)
    for k in ("dw_next", "dw_post", "dgate"):
        assert not r[k].any(), k

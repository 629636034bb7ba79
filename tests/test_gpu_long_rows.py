"""Rows whose bytes, as a 32-bit number, wrap to a short or negative row: the
operators without a limit on the row's length move all of them."""
import pytest
import torch

import mixture_experts_layer_61_b200 as moe

pytestmark = pytest.mark.gpu

CASES = [((1 << 30) + 4, torch.float32), (1 << 30, torch.bfloat16)]


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def one_token(H, dtype):
    """One token on one expert: the config, its alignment and a row of H values."""
    cfg = moe.config(1, H, 1, 1, 8, tile_B=1, dtype=dtype)
    al = moe.align_pad(cfg, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(1)
    return cfg, al, torch.empty((1, H), dtype=dtype, device="cuda").normal_(generator=g)


def same(out, ref):
    return torch.equal(out.view(-1), ref.view(-1))


@pytest.mark.parametrize("H,dtype", CASES)
def test_permute(H, dtype):
    cfg, al, x = one_token(H, dtype)
    assert same(moe.permute(cfg, x, al["sorted_ids"], al["scalars"]), x)


@pytest.mark.parametrize("H,dtype", CASES)
def test_combine(H, dtype):
    cfg, al, y = one_token(H, dtype)
    w = torch.full((1, 1), 0.5, device="cuda")
    assert same(moe.combine(cfg, y, al["pos"], w), y.mul_(0.5))  # halves are exact


@pytest.mark.parametrize("H,dtype", CASES)
def test_permute_grad(H, dtype):
    cfg, al, d = one_token(H, dtype)
    extra = d.flip(1)
    dx = moe.permute_grad(cfg, d, al["pos"], dx_add=extra)
    assert same(dx, d.add_(extra))  # one fp32 sum of two values, one rounding, on both sides

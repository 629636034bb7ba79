"""Refusals of the training entry points, on the CPU: every call here is turned
away by the library's argument checks (MOE_ERR_ARG) before any device call, or
by the binding's checks of its tensors."""
import ctypes
import os
import re

import pytest
import torch

import mixture_experts_layer_61_b200 as moe

ARG = -1
P = ctypes.c_void_p(4096)      # never read: the call is refused first
ODD = ctypes.c_void_p(4100)    # not on a 16-byte boundary
NONE = None
WS = 1 << 30


def cfg(**kw):
    a = dict(T=32, H=256, E=8, K=2, I=512)
    a.update(kw)
    return moe.config(**a)


def nc(**kw):
    a = dict(T=32, H=256)
    a.update(kw)
    return moe.norm_config(**a)


BAD_CFG = [dict(T=-1), dict(H=250), dict(K=9), dict(E=1025), dict(dtype=2), dict(score_fn=2), dict(renorm=3)]

CALLS = {  # name: (number of pointers after the config, pointers that may be NULL, trailing workspace)
    "moe_combine_grad": (8, (), False),
    "moe_permute_grad": (4, (2,), False),
    "moe_route_grad": (4, (), False),
    "moe_grouped_gate_up_train": (5, (), True),
    "moe_grouped_down_grad": (5, (), True),
    "moe_grouped_gate_up_grad": (4, (), True),
    "moe_grouped_down_wgrad": (4, (), True),
    "moe_grouped_gate_up_wgrad": (4, (), True),
}


def call(name, c, ptrs, ws=P):
    n, _, has_ws = CALLS[name]
    args = [ctypes.byref(c)] + list(ptrs)
    if has_ws:
        args += [ws, WS]
    return getattr(moe.lib(), name)(*args, None)


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_configurations_and_pointers(name):
    n, optional, has_ws = CALLS[name]
    for bad in BAD_CFG:
        c = cfg(**{k: v for k, v in bad.items()})
        assert call(name, c, [P] * n) == ARG, bad
    assert getattr(moe.lib(), name)(None, *([P] * n), *([P, WS] if has_ws else []), None) == ARG
    for i in range(n):
        if i in optional:
            continue
        assert call(name, cfg(), [NONE if j == i else P for j in range(n)]) == ARG, i
    if has_ws:
        assert call(name, cfg(), [P] * n, ws=NONE) == ARG
        assert call(name, cfg(), [P] * n, ws=ODD) == ARG


@pytest.mark.parametrize("name,vectors", [
    ("moe_combine_grad", (0, 1, 6)), ("moe_permute_grad", (0, 2, 3)), ("moe_grouped_gate_up_train", (0, 1, 3, 4)),
    ("moe_grouped_down_grad", (0, 1, 2, 4)), ("moe_grouped_gate_up_grad", (0, 1, 3)),
    ("moe_grouped_down_wgrad", (0, 1, 3)), ("moe_grouped_gate_up_wgrad", (0, 1, 3))])
def test_misaligned_tensors(name, vectors):
    n = CALLS[name][0]
    for i in vectors:
        assert call(name, cfg(), [ODD if j == i else P for j in range(n)]) == ARG, i


@pytest.mark.parametrize("name", [n for n in CALLS if n.startswith("moe_grouped")])
def test_products_are_bf16_on_whole_mma_steps(name):
    n = CALLS[name][0]
    assert call(name, cfg(dtype=moe.FP32), [P] * n) == ARG
    for B in (1, 8, 24, 255):
        assert call(name, cfg(tile_B=B), [P] * n) == ARG, B


def test_rows_wider_than_the_row_kernels_are_refused():
    assert call("moe_combine_grad", cfg(H=16392), [P] * 8) == ARG
    assert call("moe_combine_grad", cfg(H=8196, dtype=moe.FP32), [P] * 8) == ARG
    assert moe.lib().moe_block_norm_grad_workspace_size(ctypes.byref(nc(H=16392))) == 0


def norm(c, y=P, residual=P, w_post=NONE, gate=NONE, w_next=NONE, h=P, n=NONE):
    return moe.lib().moe_block_norm(ctypes.byref(c), y, residual, w_post, gate, w_next, h, n, None)


def combine_norm(c, k, y=P, pos=P, w=P, shared=NONE, residual=P, w_post=NONE, gate=NONE, w_next=NONE, y_out=NONE, h=P,
                 n=NONE):
    return moe.lib().moe_combine_norm(ctypes.byref(c), ctypes.byref(k), y, pos, w, shared, residual, w_post, gate,
                                      w_next, y_out, h, n, None)


def norm_grad(c, h=P, dh=P, dn=P, y=P, w_post=NONE, gate=NONE, w_next=P, dres=P, dy=P, dgate=NONE, dw_post=NONE,
              dw_next=P, ws=P):
    return moe.lib().moe_block_norm_grad(ctypes.byref(c), h, dh, dn, y, w_post, gate, w_next, dres, dy, dgate, dw_post,
                                         dw_next, ws, WS, None)


BAD_NORM = [dict(T=-1), dict(H=0), dict(H=252), dict(H=16392), dict(H=8196, dtype=moe.FP32), dict(dtype=2),
            dict(gate_mode=3), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
            dict(res_scale=float("nan")), dict(res_scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_NORM)
def test_bad_norm_configurations(bad):
    c = nc(**bad)
    assert norm(c) == ARG and norm_grad(c) == ARG and combine_norm(cfg(), c) == ARG
    assert moe.lib().moe_block_norm_grad_workspace_size(ctypes.byref(c)) == 0


def test_norm_arguments_that_do_not_belong_together():
    c, g = nc(), nc(gate_mode=moe.GATE_CHANNEL)
    assert norm(c, y=NONE, residual=NONE) == ARG                # nothing to norm
    assert norm(c, y=NONE, w_post=P) == ARG                     # a norm after a block that is not there
    assert norm(g, y=NONE, gate=P) == ARG
    assert norm(c, gate=P) == ARG and norm(g) == ARG            # a gate against its mode
    assert norm(c, w_next=P) == ARG and norm(c, n=P) == ARG     # n with w_next and only then
    assert norm(c, h=NONE) == ARG                               # no output
    for k in ("y", "residual", "w_post", "w_next", "h"):
        kw = {k: ODD}
        if k == "w_next":
            kw["n"] = P
        assert norm(c, **kw) == ARG, k
    assert combine_norm(cfg(), c, y=NONE) == ARG and combine_norm(cfg(), c, pos=NONE) == ARG
    assert combine_norm(cfg(), c, w=NONE) == ARG and combine_norm(cfg(), c, shared=ODD) == ARG
    assert combine_norm(cfg(), c, y_out=ODD) == ARG
    for other in (nc(T=31), nc(H=264), nc(dtype=moe.FP32)):     # another layer's norm
        assert combine_norm(cfg(), other) == ARG


def test_norm_gradient_arguments_that_do_not_belong_together():
    c, g = nc(), nc(gate_mode=moe.GATE_CHANNEL)
    assert norm_grad(c, dn=NONE) == ARG and norm_grad(c, w_next=NONE) == ARG
    assert norm_grad(c, h=NONE) == ARG                          # n's gradient needs h
    assert norm_grad(c, dh=NONE, dn=NONE, w_next=NONE, dw_next=NONE) == ARG
    assert norm_grad(c, dw_post=P) == ARG                       # a gradient of a weight that is not there
    assert norm_grad(c, dn=NONE, w_next=NONE) == ARG            # dw_next without w_next
    assert norm_grad(c, y=NONE) == ARG and norm_grad(c, dy=NONE) == ARG
    assert norm_grad(c, gate=P, dgate=P) == ARG and norm_grad(g) == ARG
    assert norm_grad(g, gate=P) == ARG and norm_grad(g, dgate=P) == ARG
    assert norm_grad(c, y=NONE, dy=NONE, w_post=P) == ARG       # a norm after a block that is not there
    assert norm_grad(c, y=NONE, dy=NONE, dres=NONE) == ARG      # no output
    assert norm_grad(c, ws=NONE) == ARG
    for k in ("h", "dh", "dn", "y", "w_next", "dres", "dy", "dw_next", "ws"):
        assert norm_grad(c, **{k: ODD}) == ARG, k


def test_zero_tokens_is_a_no_op_without_pointers():
    for name in ("moe_combine_grad", "moe_permute_grad", "moe_route_grad"):
        assert call(name, cfg(T=0), [NONE] * CALLS[name][0]) == 0
    for name in ("moe_grouped_gate_up_train", "moe_grouped_down_grad", "moe_grouped_gate_up_grad"):
        assert call(name, cfg(T=0), [NONE] * CALLS[name][0]) == 0
        assert call(name, cfg(T=0), [NONE] * CALLS[name][0], ws=NONE) == 0
    for name in ("moe_grouped_down_wgrad", "moe_grouped_gate_up_wgrad"):  # these write zeros: somewhere
        assert call(name, cfg(T=0), [NONE] * 4) == ARG
    assert norm(nc(T=0), y=NONE, residual=NONE, h=NONE) == 0
    assert combine_norm(cfg(T=0), nc(T=0), y=NONE, pos=NONE, w=NONE, residual=NONE, h=NONE) == 0


def test_norm_config_matches_the_header():
    with open(moe.HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} moe_norm_config_t;", text).group(1)
    assert re.findall(r"(int|float)\s+(\w+);", body) == [
        ("float" if t is ctypes.c_float else "int", n) for n, t in moe.NormConfig._fields_]


def test_binding_refuses_tensors_that_do_not_fit():
    c = cfg()
    x = torch.zeros((32, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.permute_grad(c, x, torch.zeros(64, dtype=torch.int32))
    with pytest.raises(ValueError, match="needs y or residual"):
        moe.block_norm(nc())

    class Fake:
        """Stands in for a CUDA tensor of another type, shape, layout or device."""
        is_cuda = True

        def __init__(self, shape, dtype, index=0, contiguous=True):
            self.shape, self.dtype, self.device, self._c = shape, dtype, torch.device("cuda", index), contiguous

        def is_contiguous(self):
            return self._c

    import unittest.mock as mock
    with mock.patch.object(torch.cuda, "current_device", lambda: 0):
        good = Fake((32, 256), torch.bfloat16)
        moe._arg("x", good, (32, 256), torch.bfloat16)
        moe._arg("x", None, (32, 256), torch.bfloat16)
        for bad in (Fake((32, 255), torch.bfloat16), Fake((32, 256), torch.float16), Fake((256, 32), torch.bfloat16),
                    Fake((32, 256), torch.bfloat16, contiguous=False), Fake((32, 256), torch.bfloat16, index=1)):
            with pytest.raises(ValueError):
                moe._arg("x", bad, (32, 256), torch.bfloat16)


WRAPPING = [(1 << 30, moe.FP32), ((1 << 30) + 4, moe.FP32), (1 << 30, moe.BF16), ((1 << 30) + 8, moe.BF16)]


@pytest.mark.parametrize("H,dtype", WRAPPING)
def test_row_bytes_past_32_bits_are_refused(H, dtype):
    """Rows whose bytes, as a 32-bit number, wrap to a short or negative row."""
    c = nc(T=1, H=H, dtype=dtype)
    assert norm(c) == ARG and norm_grad(c) == ARG
    k = cfg(T=1, E=1, K=1, H=H, I=8, dtype=dtype)
    assert combine_norm(k, c) == ARG
    assert call("moe_combine_grad", k, [P] * 8) == ARG


@pytest.mark.parametrize("name", [n for n in CALLS if n.startswith("moe_grouped")])
@pytest.mark.parametrize("size", [dict(H=(1 << 30) + 8, I=8), dict(H=8, I=(1 << 29) + 8), dict(H=8, I=(1 << 30) - 8)])
def test_products_whose_tile_coordinates_would_pass_32_bits_are_refused(name, size):
    assert call(name, cfg(T=1, E=1, K=1, **size), [P] * CALLS[name][0]) == ARG

"""Forms of the training calls that the header allows beside the binding's usual
ones: outputs left out, results over their inputs, max-value padding, rows and
weights whose element offsets pass 2^31."""
import ctypes

import pytest
import torch

import mixture_experts_layer_61_b200 as moe
import train_ref as R
from test_gpu_train_products import BF, HALF, Case, dot
from test_gpu_train_rows import gen, norm_inputs, randn, routing

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return None if t is None else t.data_ptr()


def grad_call(nc, ws, h, dh, dn, y, wp, gate, wn, dres, dy, dgate, dwp, dwn):
    rc = moe.lib().moe_block_norm_grad(ctypes.byref(nc), *(ptr(t) for t in (h, dh, dn, y, wp, gate, wn, dres, dy, dgate,
                                                                            dwp, dwn, ws)), ws.numel(), stream())
    assert rc == 0, rc


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(3, 264), (331, 4104), (200, 8192)])
@pytest.mark.parametrize("gate_mode", [0, 1, 2])
def test_norm_gradient_over_its_inputs_and_without_optional_outputs(T, H, gate_mode, dtype):
    wp, gate, wn, y = norm_inputs(T, H, dtype, True, gate_mode, True)
    g = gen(21)
    h, dh, dn = (randn(T, H, g=g, dtype=dtype) for _ in range(3))
    nc = moe.norm_config(T, H, res_scale=0.7, gate_mode=gate_mode, dtype=dtype)
    ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
    want = moe.block_norm_grad(nc, ws, h=h, dh=dh, dn=dn, y=y, w_post=wp, gate=gate, w_next=wn)

    def dgate():
        return None if gate is None else torch.full_like(want["dgate"], 5.0)

    # dy over dn, dresidual over dh
    d2, n2, dg = dh.clone(), dn.clone(), dgate()
    sums = torch.full((2, H), 5.0, device="cuda")
    grad_call(nc, ws, h, d2, n2, y, wp, gate, wn, d2, n2, dg, sums[0], sums[1])
    assert torch.equal(d2, want["dresidual"]) and torch.equal(n2, want["dy"])
    assert torch.equal(sums[0], want["dw_post"]) and torch.equal(sums[1], want["dw_next"])
    assert dg is None or torch.equal(dg, want["dgate"])
    # no weights' gradients, no dresidual
    dy, dg = torch.empty_like(y), dgate()
    grad_call(nc, ws, h, dh, dn, y, wp, gate, wn, None, dy, dg, None, None)
    assert torch.equal(dy, want["dy"]) and (dg is None or torch.equal(dg, want["dgate"]))
    # one of the two
    only = torch.full((H,), 5.0, device="cuda")
    grad_call(nc, ws, h, dh, dn, y, wp, gate, wn, None, dy, dgate(), only, None)
    assert torch.equal(only, want["dw_post"])
    grad_call(nc, ws, h, dh, dn, y, wp, gate, wn, None, dy, dgate(), None, only)
    assert torch.equal(only, want["dw_next"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norms_without_h_and_over_the_residual(dtype):
    T, H = 37, 1000
    cfg, _, ids, w, al = routing(T, 5, 3, 2, dyn=True, dtype=dtype, H=H)
    yp = randn(moe.padded_rows_max(cfg), H, g=gen(3), dtype=dtype)
    wp, gate, wn, res = norm_inputs(T, H, dtype, True, 1, True)
    nc = moe.norm_config(T, H, res_scale=0.5, gate_mode=1, dtype=dtype)
    h, n, y = moe.combine_norm(cfg, nc, yp, al["pos"], w, None, res, wp, gate, wn, save_y=True)
    n2 = torch.full_like(n, 5.0)
    args = (ptr(yp), ptr(al["pos"]), ptr(w), None, ptr(res), ptr(wp), ptr(gate), ptr(wn))
    rc = moe.lib().moe_combine_norm(ctypes.byref(cfg), ctypes.byref(nc), *args, None, None, ptr(n2), stream())
    assert rc == 0 and torch.equal(n2, n)
    over = res.clone()
    h2, n2, _ = moe.combine_norm(cfg, nc, yp, al["pos"], w, None, over, wp, gate, wn, h=over)
    assert torch.equal(h2, h) and torch.equal(n2, n)
    n3 = torch.full_like(n, 5.0)
    hb, nb = moe.block_norm(nc, residual=res, y=y, w_post=wp, gate=gate, w_next=wn)
    rc = moe.lib().moe_block_norm(ctypes.byref(nc), ptr(y), ptr(res), ptr(wp), ptr(gate), ptr(wn), None, ptr(n3),
                                  stream())
    assert rc == 0 and torch.equal(n3, nb)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,K,B", [(1, 4, 2, 16), (50, 6, 2, 16), (130, 3, 3, 5)])
def test_max_value_padding(T, E, K, B, dtype):
    """Every expert as long as the longest: the combine's gradient zeroes all the padding, the permute's reads none."""
    H = 200
    cfg, _, ids, w, al = routing(T, E, K, 4, B, dtype=dtype, H=H, pad_mode=moe.MAXVALUE)
    g = gen(22)
    Pm, P = moe.padded_rows_max(cfg), int(al["scalars"][0])
    y, dout = randn(Pm, H, g=g, dtype=dtype), randn(T, H, g=g, dtype=dtype)
    y[al["sorted_ids"] < 0] = float("nan")
    buf = torch.full_like(y, 7.0)
    dy, dw = moe.combine_grad(cfg, dout, y, al["pos"], w, al["sorted_ids"], al["scalars"], dy_perm=buf)
    rows, rdw, mag = R.combine_grad(R.f64(dout), R.f64(y), al["pos"].cpu(), R.f64(w))
    R.close(dw, rdw, R.rounded(rdw, torch.float32, mag), "dw")
    ref = torch.zeros((P, H), dtype=torch.float64)
    ref[al["pos"].cpu().long()] = rows.view(T * K, H)
    R.close(dy[:P], ref, (R.HALF[dtype] + 2.0 ** -23) * ref.abs(), "dy_perm")
    assert (dy[P:] == 7.0).all()
    dx = moe.permute_grad(cfg, y, al["pos"])
    ref, mag = R.combine(torch.nan_to_num(R.f64(y)), al["pos"].cpu(), torch.ones((T, K), dtype=torch.float64))
    R.close(dx, ref, R.rounded(ref, dtype, mag), "dx")


def test_products_with_row_offsets_past_2_31():
    """140000 tokens, pre-activations of 16384: their elements pass 2^31."""
    T, H, E, I = 140000, 64, 3, 8192
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ids[100000:] = 2
    c = Case(T, H, E, 1, I, ids=ids)
    assert c.P * 2 * I > 2 ** 31
    g = c.g
    big = lambda n: torch.empty((c.Pm, n), dtype=BF, device="cuda").normal_(generator=g)
    x, dy = big(H), big(H)
    for t in (x, dy):
        t[~c.real] = 0
    w13, w2 = randn(E, 2 * I, H, g=g, dtype=BF, std=H ** -0.5), randn(E, H, I, g=g, dtype=BF, std=I ** -0.5)
    h13, act = moe.grouped_gate_up_train(c.cfg, x, w13, c.off, c.ws)
    keep = h13[c.P - 64:c.P].clone()
    dh = moe.grouped_down_grad(c.cfg, dy, w2, h13, c.off, c.ws, dh13=h13)
    dx = moe.grouped_gate_up_grad(c.cfg, dh, w13, c.off, c.ws)
    dw2 = moe.grouped_down_wgrad(c.cfg, dy, act, c.off, c.ws)
    dw13 = moe.grouped_gate_up_wgrad(c.cfg, dh, x, c.off, c.ws)
    moe.check_status(c.ws)
    s = slice(c.P - 64, c.P)  # the farthest rows, of expert 2
    v, m = (t.cpu() for t in dot(x[s], w13[2].t()))
    acc = R.product_bound(H, m)
    R.close(keep, v, HALF * (v.abs() + acc) + acc, "h13")
    da, m = (t.cpu() for t in dot(dy[s], w2[2]))
    acc = R.product_bound(H, m)
    gt = R.f64(keep[:, :I])
    e = R.silu(gt).abs() * (acc + (da.abs() + acc) * 2.0 ** -20 * (1 + gt.abs()))
    ref = da * R.silu(gt)
    R.close(dh[s, I:], ref, HALF * (ref.abs() + e) + e, "du")
    v, m = (t.cpu() for t in dot(dh[s], w13[2]))
    acc = R.product_bound(2 * I, m)
    R.close(dx[s], v, HALF * (v.abs() + acc) + acc, "dx_perm")
    a, b = c.seg[2], c.seg[3]
    cols = slice(I - 16, I)
    for out, d, r in ((dw2[2][:, cols], dy[a:b], act[a:b, cols]),
                      (dw13[2][-16:], dh[a:b, -16:], x[a:b])):
        v, m = (t.cpu() for t in dot(d.t(), r))
        acc = R.product_bound(b - a, m)
        R.close(out, v, HALF * (v.abs() + acc) + acc, "weight gradient")
    assert not dw2[1].any() and not dw13[1].any()


def test_weights_with_offsets_past_2_31():
    """260 experts of 4096 x 2048: the weights' elements, and their gradients', pass 2^31."""
    T, H, E, I = 300, 2048, 260, 2048
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    ids[:40] = 0
    c = Case(T, H, E, 1, I, ids=ids)
    assert E * 2 * I * H > 2 ** 31
    g = c.g
    x, dy, dh = c.rows(H), c.rows(H, 0.1), c.rows(2 * I, 0.1)
    w13 = torch.zeros((E, 2 * I, H), dtype=BF, device="cuda")
    for e in (0, E - 1):
        w13[e] = randn(2 * I, H, g=g, dtype=BF, std=H ** -0.5)
    h13, _ = moe.grouped_gate_up_train(c.cfg, x, w13, c.off, c.ws)
    dx = moe.grouped_gate_up_grad(c.cfg, dh, w13, c.off, c.ws)
    dw13 = moe.grouped_gate_up_wgrad(c.cfg, dh, x, c.off, c.ws)
    moe.check_status(c.ws)
    for out, d, w in ((h13, x, w13.transpose(1, 2)), (dx, dh, w13)):
        v, m = c.each(lambda e, s: dot(d[s], w[e]), out.shape[1])
        acc = R.product_bound(w.shape[1], m)
        R.close(out[:c.P], v, HALF * (v.abs() + acc) + acc)
    a, b = c.seg[E - 1], c.seg[E]
    v, m = (t.cpu() for t in dot(dh[a:b].t(), x[a:b]))
    acc = R.product_bound(b - a, m)
    R.close(dw13[E - 1], v, HALF * (v.abs() + acc) + acc, "dw13")
    assert not dw13[1:E - 1].any()

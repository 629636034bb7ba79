"""The row-wise training operators on the GPU against their 64-bit closed
forms: combine, permute and gate gradients, the block norms and their
gradient; the error bounds are train_ref's."""
import itertools

import numpy as np
import pytest
import torch

import mixture_experts_layer_61_b200 as moe
import train_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, g, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def routing(T, E, K, seed, B=16, dyn=False, dtype=torch.bfloat16, H=64, I=64, **kw):
    """A config and the library's own routing of random logits."""
    cfg = moe.config(T, H, E, K, I, tile_B=B, dtype=dtype, **kw)
    logits = torch.randn((T, E), generator=gen(seed), device="cuda")
    k = torch.randint(0, K + 1, (T,), generator=gen(seed + 1), device="cuda", dtype=torch.int32) if dyn else None
    ids, w = moe.route(cfg, logits, k=k)
    return cfg, logits, ids, w, moe.align_pad(cfg, ids)


SHAPES = [  # T, H, E, K, B, dyn
    (1, 8, 1, 1, 16, False), (1, 4096, 8, 2, 16, False), (33, 264, 5, 3, 1, True), (64, 256, 8, 2, 16, False),
    (257, 1000, 64, 8, 16, True), (40, 4104, 33, 16, 128, True), (19, 7168, 256, 8, 16, False),
    (5, 16384, 16, 4, 16, False), (300, 72, 1024, 16, 32, True)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,E,K,B,dyn", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_combine_grad(T, H, E, K, B, dyn, dt, in_place):
    dtype = DT[dt]
    if dt == "fp32" and H > 8192:
        H = 8192
    cfg, _, ids, w, al = routing(T, E, K, T + H, B, dyn, dtype, H)
    g = gen(7)
    Pm = moe.padded_rows_max(cfg)
    P = int(al["scalars"][0])
    dout, y = randn(T, H, g=g, dtype=dtype), randn(Pm, H, g=g, dtype=dtype)
    real = al["sorted_ids"] >= 0
    y[~real] = float("nan")  # padding slots and rows past P are never read
    ref_rows, ref_dw, mag = R.combine_grad(R.f64(dout), R.f64(y), al["pos"].cpu(), R.f64(w))
    buf = y if in_place else torch.full_like(y, 7.0)
    tail = buf[P:].clone()
    dy, dw = moe.combine_grad(cfg, dout, y, al["pos"], w, al["sorted_ids"], al["scalars"], dy_perm=buf)
    R.close(dw, ref_dw, R.rounded(ref_dw, torch.float32, mag), "dw")
    ref = torch.zeros((P, H), dtype=torch.float64)
    pos = al["pos"].cpu().long()
    ref[pos[pos >= 0]] = ref_rows.view(T * K, H)[pos >= 0]
    # one product, one rounding (and the product's own in fp32)
    R.close(dy[:P], ref, (R.HALF[dtype] + 2.0 ** -23) * ref.abs(), "dy_perm")
    assert torch.equal(torch.nan_to_num(dy[P:].float(), nan=-1.0), torch.nan_to_num(tail.float(), nan=-1.0))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,E,K,B,dyn", SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_permute_grad(T, H, E, K, B, dyn, dt, add):
    dtype = DT[dt]
    cfg, _, ids, w, al = routing(T, E, K, T + H, B, dyn, dtype, H)
    g = gen(8)
    dx_perm = randn(moe.padded_rows_max(cfg), H, g=g, dtype=dtype)
    dx_perm[al["sorted_ids"] < 0] = float("nan")
    extra = randn(T, H, g=g, dtype=dtype) if add else None
    dx = moe.permute_grad(cfg, dx_perm, al["pos"], dx_add=extra)
    ones = torch.ones((T, K), dtype=torch.float64)
    rows = torch.nan_to_num(R.f64(dx_perm))
    ref, mag = R.combine(rows, al["pos"].cpu(), ones, R.f64(extra))
    R.close(dx, ref, R.rounded(ref, dtype, mag), "dx")


@pytest.mark.parametrize("score_fn,renorm", list(itertools.product([0, 1], [0, 1])))
@pytest.mark.parametrize("T,E,K,dyn", [(1, 1, 1, False), (1, 8, 2, False), (70, 8, 8, True), (333, 64, 8, True),
                                       (129, 256, 8, False), (65, 1024, 16, True), (4, 37, 5, True)])
def test_route_grad(T, E, K, dyn, score_fn, renorm):
    cfg, logits, ids, w, _ = routing(T, E, K, 3 * T + E, dyn=dyn, score_fn=score_fn, renorm=renorm)
    dw = torch.randn((T, K), generator=gen(9), device="cuda")
    dw[ids < 0] = float("nan")  # an empty slot's gradient is not read
    out = moe.route_grad(cfg, logits, ids, dw, dlogits=torch.full((T, E), 5.0, device="cuda"))
    ref, mag = R.gate_grad(R.f64(logits), ids.cpu(), R.f64(dw), score_fn, renorm)
    R.close(out, ref, R.rounded(ref, torch.float32, mag), "dlogits")


def test_route_grad_extremes():
    """Saturated sigmoids keep their small complement; infinite logits that are not selected, repeated and
    out-of-range ids."""
    cfg = moe.config(3, 64, 4, 2, 64, score_fn=1, renorm=0)
    l = torch.tensor([[30.0, -30.0, 0.0, 1.0], [20.0, 15.0, -80.0, 2.0], [0.5, 1.0, 2.0, 3.0]], device="cuda")
    ids = torch.tensor([[0, 1], [2, 1], [3, 3]], dtype=torch.int32, device="cuda")
    dw = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]], device="cuda")
    ref, mag = R.gate_grad(R.f64(l), ids.cpu(), R.f64(dw), 1, 0)
    R.close(moe.route_grad(cfg, l, ids, dw), ref, R.rounded(ref, torch.float32, mag))
    bad = ids.clone()
    bad[0, 1], bad[1, 0] = 4, -7
    ref, mag = R.gate_grad(R.f64(l), torch.where((bad < 0) | (bad > 3), -1, bad).cpu(), R.f64(dw), 1, 0)
    R.close(moe.route_grad(cfg, l, bad, dw), ref, R.rounded(ref, torch.float32, mag))
    for renorm in (0, 1):
        c = moe.config(1, 64, 4, 2, 64, renorm=renorm)
        l = torch.tensor([[1.0, float("-inf"), 0.0, -1e30]], device="cuda")
        i = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
        d = torch.tensor([[1.0, -1.0]], device="cuda")
        ref, mag = R.gate_grad(R.f64(l), i.cpu(), R.f64(d), 0, renorm)
        R.close(moe.route_grad(c, l, i, d), ref, R.rounded(ref, torch.float32, mag))


# ----------------------------------------------------------------- block norms
NORM_SHAPES = [(1, 8), (1, 4096), (7, 264), (333, 1000), (150, 7168), (3, 2056), (2, 16384), (600, 64)]
FORMS = [(p, g, n) for p in (False, True) for g in (0, 1, 2) for n in (False, True)]


def norm_inputs(T, H, dtype, post, gate_mode, nxt, seed=11):
    g = gen(seed)
    wp = (1 + 0.2 * randn(H, g=g, dtype=torch.float32)).to(dtype) if post else None
    gate = None if gate_mode == 0 else randn(*((H,) if gate_mode == 1 else (T, H)), g=g, dtype=dtype, std=0.5)
    wn = (1 + 0.2 * randn(H, g=g, dtype=torch.float32)).to(dtype) if nxt else None
    return wp, gate, wn, randn(T, H, g=g, dtype=dtype)


def check_norm(h, n, ref, dtype, residual=True):
    rh, rn, mag = ref
    R.close(h, rh, R.rounded(rh, dtype, mag), "h")
    if rn is not None:
        # n scales h's unrounded terms by rho and w: the same relative magnitudes
        s = torch.where(rh != 0, rn.abs() / rh.abs().clamp(min=1e-300), torch.zeros_like(rh))
        R.close(n, rn, R.rounded(rn, dtype, s * mag + rn.abs()), "n")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("post,gate_mode,nxt", FORMS)
def test_block_norm(T, H, post, gate_mode, nxt, dt):
    dtype = DT[dt]
    H = min(H, 8192) if dt == "fp32" else H
    wp, gate, wn, y = norm_inputs(T, H, dtype, post, gate_mode, nxt)
    res = randn(T, H, g=gen(12), dtype=dtype)
    nc = moe.norm_config(T, H, eps=1e-5, res_scale=0.7, gate_mode=gate_mode, dtype=dtype)
    h, n = moe.block_norm(nc, residual=res, y=y, w_post=wp, gate=gate, w_next=wn)
    eps, s = float(nc.eps), float(nc.res_scale)  # as the library holds them, in 32 bits
    ref = R.block_norm(R.f64(y), R.f64(res), R.f64(wp), R.f64(gate), R.f64(wn), eps, s)
    check_norm(h, n, ref, dtype)
    if nxt:  # in place, and n alone
        buf = res.clone()
        h2, n2 = moe.block_norm(nc, residual=buf, y=y, w_post=wp, gate=gate, w_next=wn, h=buf)
        assert torch.equal(h2, h) and torch.equal(n2, n)
        buf = y.clone()
        h3, _ = moe.block_norm(nc, residual=res, y=buf, w_post=wp, gate=gate, w_next=wn, h=buf)
        assert torch.equal(h3, h)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_norm_before_a_block_only(dt):
    dtype = DT[dt]
    T, H = 37, 520
    x, w = randn(T, H, g=gen(1), dtype=dtype), randn(H, g=gen(2), dtype=dtype)
    x[3] = 0  # a row of zeros: rho = eps^-1/2, n = 0
    nc = moe.norm_config(T, H, eps=1e-6, dtype=dtype)
    h, n = moe.block_norm(nc, residual=x, w_next=w)
    assert h is None
    _, ref, mag = R.block_norm(None, R.f64(x), None, None, R.f64(w), float(nc.eps), 1.0)
    R.close(n, ref, R.rounded(ref, dtype, ref.abs()), "n")
    assert not n[3].any()
    dn = randn(T, H, g=gen(3), dtype=dtype)
    r = moe.block_norm_grad(nc, moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc)), h=x, dn=dn, w_next=w)
    assert r["dy"] is None and r["dgate"] is None and r["dw_post"] is None
    want = R.block_norm_grad(R.f64(x), None, R.f64(dn), None, None, None, R.f64(w), float(nc.eps), 1.0)
    R.close(r["dresidual"], want["dresidual"], R.rounded(want["dresidual"], dtype, want["dresidual|"]), "dresidual")
    R.close(r["dw_next"], want["dw_next"], R.rounded(want["dw_next"], torch.float32, want["dw_next|"]), "dw_next")


def test_block_without_a_residual():
    T, H = 5, 264
    y, w = randn(T, H, g=gen(1), dtype=torch.bfloat16), randn(H, g=gen(2), dtype=torch.bfloat16)
    nc = moe.norm_config(T, H, res_scale=3.0)
    h, n = moe.block_norm(nc, y=y, w_post=w)
    assert n is None
    ref, _, mag = R.block_norm(R.f64(y), None, R.f64(w), None, None, float(nc.eps), 3.0)
    R.close(h, ref, R.rounded(ref, torch.bfloat16, mag), "h")
    dh = randn(T, H, g=gen(3), dtype=torch.bfloat16)
    r = moe.block_norm_grad(nc, moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc)), dh=dh, y=y, w_post=w,
                            residual=False)
    assert r["dresidual"] is None
    want = R.block_norm_grad(None, R.f64(dh), None, R.f64(y), R.f64(w), None, None, float(nc.eps), 3.0)
    R.close(r["dy"], want["dy"], R.rounded(want["dy"], torch.bfloat16, want["dy|"]), "dy")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,E,K,B,dyn", SHAPES)
@pytest.mark.parametrize("shared,post,gate_mode,nxt", [(False, False, 0, True), (True, True, 1, True),
                                                       (True, False, 2, False), (False, True, 0, False)])
def test_combine_norm(T, H, E, K, B, dyn, shared, post, gate_mode, nxt, dt):
    dtype = DT[dt]
    H = min(H, 8192) if dt == "fp32" else H
    cfg, _, ids, w, al = routing(T, E, K, T + H, B, dyn, dtype, H)
    g = gen(13)
    yp = randn(moe.padded_rows_max(cfg), H, g=g, dtype=dtype)
    yp[al["sorted_ids"] < 0] = float("nan")
    sh = randn(T, H, g=g, dtype=dtype) if shared else None
    wp, gate, wn, res = norm_inputs(T, H, dtype, post, gate_mode, nxt)
    nc = moe.norm_config(T, H, eps=1e-5, res_scale=0.5, gate_mode=gate_mode, dtype=dtype)
    h, n, y = moe.combine_norm(cfg, nc, yp, al["pos"], w, sh, res, wp, gate, wn, save_y=True)
    ry, ymag = R.combine(torch.nan_to_num(R.f64(yp)), al["pos"].cpu(), R.f64(w), R.f64(sh))
    R.close(y, ry, R.rounded(ry, dtype, ymag), "y")
    # the combine's own output, bit for bit
    assert torch.equal(y, moe.combine(cfg, yp, al["pos"], w, sh))
    rh, rn, mag = R.block_norm(ry, R.f64(res), R.f64(wp), R.f64(gate), R.f64(wn), float(nc.eps), 0.5)
    # z's terms: the combine's, scaled as y is (a row of zeros has none)
    zs = torch.where(ry != 0, (rh - 0.5 * R.f64(res)).abs() / ry.abs().clamp(min=1e-300), torch.zeros_like(ry))
    mag = mag + zs * ymag
    # the sum of squares is off by 2 |y| FP32 |terms|, which moves every element of the row
    row = (ry.abs() * ymag).sum(1, keepdim=True) / ry.pow(2).sum(1, keepdim=True).clamp(min=1e-300)
    mag = mag * (1 + row) if post else mag
    check_norm(h, n, (rh, rn, mag * (1 + (rh.abs() * mag).sum(1, keepdim=True) /
                                     rh.pow(2).sum(1, keepdim=True).clamp(min=1e-300))), dtype)
    h2, n2, none = moe.combine_norm(cfg, nc, yp, al["pos"], w, sh, res, wp, gate, wn)
    assert none is None and torch.equal(h2, h) and (n2 is None or torch.equal(n2, n))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("post,gate_mode,nxt", FORMS)
def test_block_norm_grad(T, H, post, gate_mode, nxt, dt):
    dtype = DT[dt]
    H = min(H, 8192) if dt == "fp32" else H
    wp, gate, wn, y = norm_inputs(T, H, dtype, post, gate_mode, nxt)
    g = gen(14)
    h, dh = randn(T, H, g=g, dtype=dtype, std=2.0), randn(T, H, g=g, dtype=dtype)
    dn = randn(T, H, g=g, dtype=dtype) if nxt else None
    nc = moe.norm_config(T, H, eps=1e-5, res_scale=0.7, gate_mode=gate_mode, dtype=dtype)
    ws = torch.full((moe.block_norm_grad_workspace_size(nc),), 0xFF, dtype=torch.uint8, device="cuda")
    for first in ((dh, None)[:1 + nxt]):  # with and without a gradient that reaches h (one of the two is needed)
        r = moe.block_norm_grad(nc, ws, h=h, dh=first, dn=dn, y=y, w_post=wp, gate=gate, w_next=wn)
        want = R.block_norm_grad(R.f64(h), R.f64(first), R.f64(dn), R.f64(y), R.f64(wp), R.f64(gate), R.f64(wn),
                                 float(nc.eps), float(nc.res_scale))
        for k, t in r.items():
            assert (t is None) == (k not in want), k
            if t is not None:
                R.close(t, want[k], R.rounded(want[k], t.dtype, want[k + "|"]), k)
    # in place: dresidual over dh, dy over y
    d2, y2 = dh.clone(), y.clone()
    a = moe.block_norm_grad(nc, ws, h=h, dh=dh, dn=dn, y=y, w_post=wp, gate=gate, w_next=wn)
    b = moe.block_norm_grad(nc, ws, h=h, dh=d2, dn=dn, y=y2, w_post=wp, gate=gate, w_next=wn, dresidual=d2, dy=y2)
    for k in a:
        assert (a[k] is None and b[k] is None) or torch.equal(a[k], b[k]), k  # also: the same from run to run


def test_zero_tokens():
    nc = moe.norm_config(0, 64, gate_mode=moe.GATE_CHANNEL)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
    r = moe.block_norm_grad(nc, ws, h=e, dh=e, dn=e, y=e, w_post=w, gate=w, w_next=w)
    assert all(not r[k].any() for k in ("dw_next", "dw_post", "dgate"))
    h, n = moe.block_norm(nc, residual=e, y=e, w_post=w, gate=w, w_next=w)
    assert h.shape == (0, 64) and n.shape == (0, 64)


def test_short_workspace_is_refused():
    nc = moe.norm_config(8, 256)
    t = torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
    with pytest.raises(moe.MoeError, match="MOE_ERR_WORKSPACE"):
        moe.block_norm_grad(nc, ws[:8 * 2 * 256 * 4 - 16], dh=t, y=t)


def test_offsets_past_32_bits():
    """Permuted rows whose element offsets pass 2^31: 70000 tokens x 4 rows of 8192 bf16."""
    T, H, E, K = 70000, 8192, 8, 4
    cfg, _, ids, w, al = routing(T, E, K, 5, H=H, I=64)
    g = gen(15)
    yp = torch.empty((moe.padded_rows_max(cfg), H), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dout = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy, dw = moe.combine_grad(cfg, dout, yp, al["pos"], w, al["sorted_ids"], al["scalars"])
    dx = moe.permute_grad(cfg, yp, al["pos"])
    pos = al["pos"].view(T, K).long()
    tok = torch.cat([torch.argmax(pos, 0), torch.arange(T - 8, T, device="cuda")])  # the farthest rows among them
    assert int(pos[tok].max()) * H > 2 ** 31
    rows, rdw, mag = R.combine_grad(R.f64(dout[tok]), R.f64(yp[pos[tok].view(-1)]),
                                    torch.arange(tok.numel() * K, dtype=torch.int32), R.f64(w[tok]))
    R.close(dw[tok], rdw, R.rounded(rdw, torch.float32, mag), "dw")
    R.close(dy[pos[tok]], rows, (R.HALF[torch.bfloat16] + 2.0 ** -23) * rows.abs(), "dy")
    s, m = R.combine(R.f64(yp[pos[tok].view(-1)]), torch.arange(tok.numel() * K, dtype=torch.int32),
                     torch.ones((tok.numel(), K), dtype=torch.float64))
    R.close(dx[tok], s, R.rounded(s, torch.bfloat16, m), "dx")


def test_side_stream_and_graph_replay():
    """The calls on another stream, captured once and replayed on new inputs, beside eager results."""
    T, H, E, K = 96, 512, 8, 2
    cfg, logits, ids, w, al = routing(T, E, K, 6, H=H)
    nc = moe.norm_config(T, H, gate_mode=moe.GATE_CHANNEL)
    g = gen(16)
    wp, gate, wn, res = norm_inputs(T, H, torch.bfloat16, True, 1, True)
    yp = randn(moe.padded_rows_max(cfg), H, g=g, dtype=torch.bfloat16)
    dh, dn = randn(T, H, g=g, dtype=torch.bfloat16), randn(T, H, g=g, dtype=torch.bfloat16)
    ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
    dy_buf = torch.zeros_like(yp)

    def step():
        h, n, y = moe.combine_norm(cfg, nc, yp, al["pos"], w, None, res, wp, gate, wn, save_y=True)
        r = moe.block_norm_grad(nc, ws, h=h, dh=dh, dn=dn, y=y, w_post=wp, gate=gate, w_next=wn)
        dy, dw = moe.combine_grad(cfg, r["dy"], yp, al["pos"], w, al["sorted_ids"], al["scalars"], dy_perm=dy_buf)
        dx = moe.permute_grad(cfg, dy, al["pos"], dx_add=r["dresidual"])
        return [h, n, y, dw, dx, moe.route_grad(cfg, logits, ids, dw)] + [r[k] for k in sorted(r)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        for t in (yp, dh, dn, res):
            t.copy_(randn(*t.shape, g=gen(seed), dtype=t.dtype))
        graph.replay()
        got = [o.clone() for o in outs]
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_permute_grad_of_rows_past_the_row_kernels():
    """The permute's gradient has no limit on the row's length."""
    T, H = 9, 40000
    cfg, _, ids, w, al = routing(T, 5, 3, 2, H=H)
    dx_perm = randn(moe.padded_rows_max(cfg), H, g=gen(3), dtype=torch.bfloat16)
    dx = moe.permute_grad(cfg, dx_perm, al["pos"])
    ref, mag = R.combine(R.f64(dx_perm), al["pos"].cpu(), torch.ones((T, 3), dtype=torch.float64))
    R.close(dx, ref, R.rounded(ref, torch.bfloat16, mag), "dx")


def test_two_norm_gradients_at_once():
    """Two streams, a workspace each: the same bits as one after the other."""
    cases = []
    for T, H, seed in ((700, 1024, 1), (300, 4096, 2)):
        wp, gate, wn, y = norm_inputs(T, H, torch.bfloat16, True, 1, True, seed)
        g = gen(seed + 10)
        h, dh, dn = (randn(T, H, g=g, dtype=torch.bfloat16) for _ in range(3))
        nc = moe.norm_config(T, H, gate_mode=1)
        ws = moe.alloc_workspace(moe.block_norm_grad_workspace_size(nc))
        cases.append(lambda nc=nc, ws=ws, h=h, dh=dh, dn=dn, y=y, wp=wp, gate=gate, wn=wn: moe.block_norm_grad(
            nc, ws, h=h, dh=dh, dn=dn, y=y, w_post=wp, gate=gate, w_next=wn))
    want = [{k: v.clone() for k, v in f().items()} for f in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for f, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[k], b[k]) for k in b)


@pytest.mark.parametrize("dt,H", [("bf16", 16384), ("bf16", 12296), ("fp32", 8192), ("fp32", 4100)])
@pytest.mark.parametrize("post,gate_mode,nxt", [(True, 2, True), (True, 1, True), (False, 0, True), (True, 2, False)])
def test_norm_gradient_of_long_rows_several_to_a_block(dt, H, post, gate_mode, nxt):
    """Rows that fill a block's shared memory (one to three at once), more rows than blocks."""
    test_block_norm_grad(331, H, post, gate_mode, nxt, dt)

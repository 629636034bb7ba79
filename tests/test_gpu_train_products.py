"""The gradients of the experts' products on the GPU (tcgen05, bf16) against
64-bit products of the same inputs, and a whole training step of the block."""
import pytest
import torch

import mixture_experts_layer_61_b200 as moe
import train_ref as R
from test_gpu_train_rows import gen, randn, routing

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = R.HALF[BF]


class Case:
    """A routing and row buffers whose padding rows are zero and whose rows past P hold NaN."""

    def __init__(self, T, H, E, K, I, B=16, dyn=False, seed=1, pad_mode=0, ids=None):
        self.cfg, _, self.ids, self.w, self.al = routing(T, E, K, seed, B, dyn, H=H, I=I, pad_mode=pad_mode)
        if ids is not None:
            self.ids = ids
            self.al = moe.align_pad(self.cfg, ids)
        self.g = gen(seed + 100)
        self.P = int(self.al["scalars"][0])
        self.Pm = moe.padded_rows_max(self.cfg)
        self.off = self.al["offsets"]
        self.seg = self.off.cpu().tolist()
        self.real = self.al["sorted_ids"] >= 0
        self.ws = moe.alloc_workspace(moe.gemm_workspace_size())

    def rows(self, width, std=1.0):
        t = randn(self.Pm, width, g=self.g, dtype=BF, std=std)
        t[~self.real] = 0
        t[self.P:] = float("nan")
        return t

    def buf(self, width):
        return torch.full((self.Pm, width), 9.0, dtype=BF, device="cuda")

    def each(self, f, width):
        """f(e, rows slice) per expert on the GPU in float64 -> [P, width] (value, magnitude) on the CPU."""
        out = torch.zeros((2, self.P, width), dtype=torch.float64)
        for e in range(self.cfg.E):
            a, b = self.seg[e], self.seg[e + 1]
            if b > a:
                v, m = f(e, slice(a, b))
                out[0, a:b], out[1, a:b] = v.cpu(), m.cpu()
        return out

    def done(self, *bufs):
        moe.check_status(self.ws)
        for t in bufs:
            assert (t[self.P:].float() == 9.0).all(), "rows past P were touched"


def dot(a, b):
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


CASES = [  # T, H, E, K, I, B, dyn, pad_mode
    (1, 8, 1, 1, 8, 16, False, 0), (1, 64, 4, 1, 64, 16, False, 0), (16, 256, 1, 1, 256, 16, False, 0),
    (40, 264, 5, 3, 136, 16, True, 0), (300, 520, 5, 3, 328, 32, True, 0), (600, 512, 2, 2, 520, 128, False, 0),
    (77, 1000, 13, 2, 72, 64, False, 0), (50, 320, 6, 2, 200, 16, False, 1), (2100, 256, 3, 2, 640, 256, False, 0),
    (200, 128, 256, 8, 64, 16, False, 0), (90, 2048, 8, 2, 1024, 16, False, 0)]


@pytest.mark.parametrize("case", CASES)
def test_gate_up_train(case):
    T, H, E, K, I, B, dyn, pm = case
    c = Case(T, H, E, K, I, B, dyn, pad_mode=pm)
    x, w13 = c.rows(H), randn(E, 2 * I, H, g=c.g, dtype=BF, std=H ** -0.5)
    h13, act = moe.grouped_gate_up_train(c.cfg, x, w13, c.off, c.ws, h13=c.buf(2 * I), act=c.buf(I))
    c.done(h13, act)
    v, m = c.each(lambda e, s: dot(x[s], w13[e].t()), 2 * I)
    acc = R.product_bound(H, m)
    R.close(h13[:c.P], v, HALF * (v.abs() + acc) + acc, "h13")
    g, u = v[:, :I], v[:, I:]
    ref = R.silu(g) * u
    # errors of g and u through silu(g) u (|silu'| <= 1.1), then the fast exponential and division:
    # 2^-20 (1 + |g|) relative (exp's argument is rounded to 2^-24 of |g| log2 e, and both are within 2^-21)
    e = 1.1 * u.abs() * acc[:, :I] + R.silu(g).abs() * acc[:, I:] + 1.1 * acc[:, :I] * acc[:, I:]
    e = e + ref.abs() * 2.0 ** -20 * (1 + g.abs())
    R.close(act[:c.P], ref, HALF * (ref.abs() + e) + e, "act")
    # the same activations as the forward without pre-activations, up to its summation order
    act2 = moe.grouped_gate_up(c.cfg, x, w13, c.off, c.ws, torch.zeros_like(act))
    R.close(act2[:c.P], ref, HALF * (ref.abs() + e) + e, "act of grouped_gate_up")


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_down_grad(case, in_place):
    T, H, E, K, I, B, dyn, pm = case
    c = Case(T, H, E, K, I, B, dyn, pad_mode=pm)
    dy, h13 = c.rows(H, 0.1), c.rows(2 * I, 2.0)
    w2 = randn(E, H, I, g=c.g, dtype=BF, std=I ** -0.5)
    if in_place:
        h13[c.P:] = 9.0
    keep = h13.clone()
    out = moe.grouped_down_grad(c.cfg, dy, w2, h13, c.off, c.ws, dh13=h13 if in_place else c.buf(2 * I))
    c.done(out)
    da, m = c.each(lambda e, s: dot(dy[s], w2[e]), I)
    acc = R.product_bound(H, m)
    g, u = R.f64(keep[:c.P, :I]), R.f64(keep[:c.P, I:])
    s = torch.sigmoid(g)
    # s within 2^-20 (1 + |g|) relative; 1 + g (1 - s) is off by |g| times s's error
    ds = 2.0 ** -20 * (1 + g.abs())
    ref = da * u * R.silu_grad(g)
    e = u.abs() * R.silu_grad(g).abs() * acc + (da.abs() + acc) * u.abs() * s * ds * (2 + 2 * g.abs())
    R.close(out[:c.P, :I], ref, HALF * (ref.abs() + e) + e, "dg")
    ref = da * R.silu(g)
    e = R.silu(g).abs() * (acc + (da.abs() + acc) * ds)
    R.close(out[:c.P, I:], ref, HALF * (ref.abs() + e) + e, "du")


def test_down_grad_far_activations():
    """Pre-activations where the exponential leaves fp32: silu' is 0 or 1 there."""
    c = Case(32, 64, 2, 1, 64)
    dy, w2 = c.rows(64), randn(2, 64, 64, g=c.g, dtype=BF)
    h13 = c.rows(128)
    far = torch.tensor([-3e38, -1000.0, -90.0, -88.0, 88.0, 90.0, 1000.0, 3e38], device="cuda").to(BF).repeat(8)
    h13[:c.P, :64] = far
    h13[:c.P, 64:] = 1.0
    h13[~c.real] = 0
    out = moe.grouped_down_grad(c.cfg, dy, w2, h13, c.off, c.ws)
    moe.check_status(c.ws)
    da, m = c.each(lambda e, s: dot(dy[s], w2[e]), 64)
    acc = R.product_bound(64, m)
    on = (R.f64(far) > 0).double()
    ref = da * on * R.f64(h13[:c.P, 64:])
    R.close(out[:c.P, :64], ref, HALF * ref.abs() + 2 * acc + 2.0 ** -100, "dg")


@pytest.mark.parametrize("case", CASES)
def test_gate_up_grad(case):
    T, H, E, K, I, B, dyn, pm = case
    c = Case(T, H, E, K, I, B, dyn, pad_mode=pm)
    dh, w13 = c.rows(2 * I, 0.1), randn(E, 2 * I, H, g=c.g, dtype=BF, std=H ** -0.5)
    dx = moe.grouped_gate_up_grad(c.cfg, dh, w13, c.off, c.ws, dx_perm=c.buf(H))
    c.done(dx)
    v, m = c.each(lambda e, s: dot(dh[s], w13[e]), H)
    acc = R.product_bound(2 * I, m)
    R.close(dx[:c.P], v, HALF * (v.abs() + acc) + acc, "dx_perm")


@pytest.mark.parametrize("case", CASES)
def test_weight_grads(case):
    T, H, E, K, I, B, dyn, pm = case
    c = Case(T, H, E, K, I, B, dyn, pad_mode=pm)
    dy, act, dh, x = c.rows(H, 0.1), c.rows(I), c.rows(2 * I, 0.1), c.rows(H)
    dw2 = moe.grouped_down_wgrad(c.cfg, dy, act, c.off, c.ws, dw2=torch.full((E, H, I), 9.0, dtype=BF, device="cuda"))
    dw13 = moe.grouped_gate_up_wgrad(c.cfg, dh, x, c.off, c.ws)
    c.done()
    for out, d, r in ((dw2, dy, act), (dw13, dh, x)):
        for e in range(E):
            a, b = c.seg[e], c.seg[e + 1]
            v, m = dot(d[a:b].t(), r[a:b])
            v, acc = v.cpu(), R.product_bound(b - a, m.cpu())
            R.close(out[e], v, HALF * (v.abs() + acc) + acc, f"expert {e}")


def test_all_tokens_on_one_expert_and_no_tokens_on_the_others():
    T, H, E, I = 100, 128, 6, 72
    ids = torch.full((T, 1), 4, dtype=torch.int32, device="cuda")
    c = Case(T, H, E, 1, I, ids=ids)
    dy, act = c.rows(H), c.rows(I)
    dw2 = moe.grouped_down_wgrad(c.cfg, dy, act, c.off, c.ws, dw2=torch.full((E, H, I), 9.0, dtype=BF, device="cuda"))
    c.done()
    assert not dw2[[0, 1, 2, 3, 5]].any()
    v, m = dot(dy[:c.P].t(), act[:c.P])
    acc = R.product_bound(c.P, m.cpu())
    R.close(dw2[4], v.cpu(), HALF * (v.cpu().abs() + acc) + acc)


def test_every_slot_empty():
    T, H, E, I = 9, 64, 4, 64
    c = Case(T, H, E, 2, I, ids=torch.full((T, 2), -1, dtype=torch.int32, device="cuda"))
    assert c.P == 0
    dh, x, dy, act = c.rows(2 * I), c.rows(H), c.rows(H), c.rows(I)
    assert not moe.grouped_gate_up_wgrad(c.cfg, dh, x, c.off, c.ws).any()
    assert not moe.grouped_down_wgrad(c.cfg, dy, act, c.off, c.ws).any()
    w13, w2 = randn(E, 2 * I, H, g=c.g, dtype=BF), randn(E, H, I, g=c.g, dtype=BF)
    outs = [moe.grouped_gate_up_grad(c.cfg, dh, w13, c.off, c.ws, dx_perm=c.buf(H)),
            moe.grouped_down_grad(c.cfg, dy, w2, dh, c.off, c.ws, dh13=c.buf(2 * I))]
    outs += moe.grouped_gate_up_train(c.cfg, x, w13, c.off, c.ws, h13=c.buf(2 * I), act=c.buf(I))
    c.done(*outs)
    dw = moe.combine_grad(c.cfg, randn(T, H, g=c.g, dtype=BF), dy, c.al["pos"], c.w, c.al["sorted_ids"],
                          c.al["scalars"])[1]
    assert not dw.any()
    assert not moe.permute_grad(c.cfg, dy, c.al["pos"]).any()


def test_zero_tokens_write_zero_weight_gradients():
    cfg = moe.config(0, 64, 4, 2, 72)
    ws = moe.alloc_workspace(moe.gemm_workspace_size())
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    e = lambda n: torch.empty((1, n), dtype=BF, device="cuda")
    dw2 = torch.full((4, 64, 72), 9.0, dtype=BF, device="cuda")
    assert not moe.grouped_down_wgrad(cfg, e(64), e(72), off, ws, dw2=dw2).any()
    assert not moe.grouped_gate_up_wgrad(cfg, e(144), e(64), off, ws).any()


def test_one_experts_nan_stays_with_it():
    """NaN and infinities in one expert's rows and weights reach no other expert: K tails (H and I not multiples
    of 64) read zeros, and a stage that reaches into the next segment does not multiply it."""
    T, H, E, I = 96, 200, 4, 136
    c = Case(T, H, E, 2, I)
    x, dy, dh, act, h13 = c.rows(H), c.rows(H), c.rows(2 * I), c.rows(I), c.rows(2 * I)
    w13, w2 = randn(E, 2 * I, H, g=c.g, dtype=BF), randn(E, H, I, g=c.g, dtype=BF)
    bad = 2
    s = slice(c.seg[bad], c.seg[bad + 1])
    for t in (x, dy, dh, act, h13):
        t[s] = float("nan")
    w13[bad], w2[bad] = float("inf"), float("-inf")
    good = torch.ones(c.P, dtype=torch.bool, device="cuda")
    good[s] = False
    others = [e for e in range(E) if e != bad]
    for rows in (*moe.grouped_gate_up_train(c.cfg, x, w13, c.off, c.ws),
                 moe.grouped_down_grad(c.cfg, dy, w2, h13, c.off, c.ws),
                 moe.grouped_gate_up_grad(c.cfg, dh, w13, c.off, c.ws)):
        assert torch.isfinite(rows[:c.P][good]).all()
    for dw in (moe.grouped_down_wgrad(c.cfg, dy, act, c.off, c.ws),
               moe.grouped_gate_up_wgrad(c.cfg, dh, x, c.off, c.ws)):
        assert torch.isfinite(dw[others]).all() and torch.isnan(dw[bad]).all()
    moe.check_status(c.ws)


def all_products(c, t):
    h13, act = moe.grouped_gate_up_train(c.cfg, t["x"], t["w13"], c.off, c.ws, h13=t["h13"], act=t["act"])
    dh = moe.grouped_down_grad(c.cfg, t["dy"], t["w2"], h13, c.off, c.ws, dh13=t["dh"])
    dx = moe.grouped_gate_up_grad(c.cfg, dh, t["w13"], c.off, c.ws, dx_perm=t["dx"])
    dw2 = moe.grouped_down_wgrad(c.cfg, t["dy"], act, c.off, c.ws)
    dw13 = moe.grouped_gate_up_wgrad(c.cfg, dh, t["x"], c.off, c.ws)
    return h13, act, dh, dx, dw2, dw13


def product_tensors(c):
    H, I, E = c.cfg.H, c.cfg.I, c.cfg.E
    return dict(x=c.rows(H), dy=c.rows(H, 0.1), w13=randn(E, 2 * I, H, g=c.g, dtype=BF, std=H ** -0.5),
                w2=randn(E, H, I, g=c.g, dtype=BF, std=I ** -0.5), h13=c.buf(2 * I), act=c.buf(I), dh=c.buf(2 * I),
                dx=c.buf(H))


def test_runs_agree_bit_for_bit_eager_captured_and_beside_another_stream():
    a, b = Case(700, 512, 4, 2, 320, seed=1), Case(500, 264, 5, 2, 200, seed=2)
    ta, tb = product_tensors(a), product_tensors(b)
    first = [t.clone() for t in all_products(a, ta)]
    other = [t.clone() for t in all_products(b, tb)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):  # two steps at once, each with its own workspace
        with torch.cuda.stream(s1):
            ra = all_products(a, ta)
        with torch.cuda.stream(s2):
            rb = all_products(b, tb)
    torch.cuda.synchronize()
    for x, y in zip(list(ra) + list(rb), first + other):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc = all_products(a, ta)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(rc, first):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    moe.check_status(a.ws)
    moe.check_status(b.ws)


@pytest.mark.parametrize("which", ["gate_up_train", "down_grad", "gate_up_grad", "down_wgrad", "gate_up_wgrad"])
def test_a_withheld_load_times_out_and_the_workspace_stays_usable(which):
    c = Case(300, 256, 4, 2, 256)
    t = product_tensors(c)
    h = c.rows(512)
    calls = {
        "gate_up_train": lambda: moe.grouped_gate_up_train(c.cfg, t["x"], t["w13"], c.off, c.ws)[0],
        "down_grad": lambda: moe.grouped_down_grad(c.cfg, t["dy"], t["w2"], h, c.off, c.ws),
        "gate_up_grad": lambda: moe.grouped_gate_up_grad(c.cfg, h, t["w13"], c.off, c.ws),
        "down_wgrad": lambda: moe.grouped_down_wgrad(c.cfg, t["dy"], c.rows(256), c.off, c.ws),
        "gate_up_wgrad": lambda: moe.grouped_gate_up_wgrad(c.cfg, h, t["x"], c.off, c.ws)}
    run = calls[which]
    want = run()[:c.P].clone() if which not in ("down_wgrad",) else None
    L = moe.lib()
    try:
        L.moe_set_wait_limit_ns(50_000_000)
        L.moe_debug_withhold_first_load(1)
        run()
        with pytest.raises(moe.MoeError, match="MOE_ERR_TIMEOUT"):
            moe.check_status(c.ws)
    finally:
        L.moe_debug_withhold_first_load(0)
        L.moe_set_wait_limit_ns(0)
    again = run()
    moe.check_status(c.ws)
    if want is not None:
        assert torch.equal(again[:c.P], want)


def test_short_workspace_is_refused():
    c = Case(16, 64, 2, 1, 64)
    with pytest.raises(moe.MoeError, match="MOE_ERR_WORKSPACE"):
        moe.grouped_down_wgrad(c.cfg, c.rows(64), c.rows(64), c.off, c.ws[: c.ws.numel() - 256])


@pytest.mark.parametrize("score_fn,gate_mode,shared", [(0, 0, False), (1, 1, True), (0, 2, True)])
def test_training_step_of_the_block(score_fn, gate_mode, shared):
    """Forward and backward of norm -> router -> experts -> combine -> norm, gate, residual -> next norm through
    the library, against float64 autograd of the whole block on the library's routing.  Both directions round to
    bf16 ten times at most on the way to any gradient (n0, h13, act, y_perm, y/h, dy, dy_perm, dh13, dx_perm, dx);
    each moves a gradient by at most 2^-8 of its own magnitudes, so the whole gradient, in the Frobenius norm, by
    at most 10 * 2^-8; twice that is allowed for what the later products make of the earlier roundings."""
    T, H, E, K, I = 320, 256, 8, 2, 192
    g = gen(50)
    cfg = moe.config(T, H, E, K, I, score_fn=score_fn)
    nc = moe.norm_config(T, H, eps=1e-5, res_scale=0.8, gate_mode=gate_mode)
    pre = moe.norm_config(T, H, eps=1e-5)
    r = lambda *s, std=1.0: randn(*s, g=g, dtype=BF, std=std)
    x, w_r = r(T, H), r(E, H, std=H ** -0.5)
    w13, w2 = r(E, 2 * I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5)
    w_pre, w_post, w_next = (1 + 0.1 * r(H)).to(BF), (1 + 0.1 * r(H)).to(BF), (1 + 0.1 * r(H)).to(BF)
    gate = None if gate_mode == 0 else r(*((H,) if gate_mode == 1 else (T, H)), std=0.5)
    sh = r(T, H) if shared else None
    dh, dn = r(T, H), r(T, H)
    ws = moe.alloc_workspace(moe.gemm_workspace_size())
    nws = moe.alloc_workspace(max(moe.block_norm_grad_workspace_size(nc), moe.block_norm_grad_workspace_size(pre)))
    # forward
    _, n0 = moe.block_norm(pre, residual=x, w_next=w_pre)
    logits = moe.router_gemm(cfg, n0, w_r, ws)
    ids, w = moe.route(cfg, logits)
    al = moe.align_pad(cfg, ids)
    xp = moe.permute(cfg, n0, al["sorted_ids"], al["scalars"])
    h13, act = moe.grouped_gate_up_train(cfg, xp, w13, al["offsets"], ws)
    yp = moe.grouped_down(cfg, act, w2, al["offsets"], ws, torch.empty_like(xp))
    h, n, y = moe.combine_norm(cfg, nc, yp, al["pos"], w, sh, x, w_post, gate, w_next, save_y=True)
    # backward
    b = moe.block_norm_grad(nc, nws, h=h, dh=dh, dn=dn, y=y, w_post=w_post, gate=gate, w_next=w_next)
    dyp, dw = moe.combine_grad(cfg, b["dy"], yp, al["pos"], w, al["sorted_ids"], al["scalars"])
    dh13 = moe.grouped_down_grad(cfg, dyp, w2, h13, al["offsets"], ws)
    dw2 = moe.grouped_down_wgrad(cfg, dyp, act, al["offsets"], ws)
    dxp = moe.grouped_gate_up_grad(cfg, dh13, w13, al["offsets"], ws)
    dw13 = moe.grouped_gate_up_wgrad(cfg, dh13, xp, al["offsets"], ws)
    dl = moe.route_grad(cfg, logits, ids, dw)
    dn0 = moe.permute_grad(cfg, dxp, al["pos"], dx_add=(dl @ w_r.float()).to(BF))
    dw_r = dl.t() @ n0.float()
    a = moe.block_norm_grad(pre, nws, h=x, dh=b["dresidual"], dn=dn0, w_next=w_pre)
    moe.check_status(ws)
    got = dict(x=a["dresidual"], w_pre=a["dw_next"], w_r=dw_r, w13=dw13, w2=dw2, w_post=b["dw_post"],
               w_next=b["dw_next"], sh=b["dy"], gate=b["dgate"])

    # float64 autograd of the block on the same routing
    leaf = {k: v.double().requires_grad_() for k, v in dict(x=x, w_pre=w_pre, w_r=w_r, w13=w13, w2=w2, w_post=w_post,
                                                             w_next=w_next).items()}
    if shared:
        leaf["sh"] = sh.double().requires_grad_()
    if gate is not None:
        leaf["gate"] = gate.double().requires_grad_()
    f = leaf
    m0 = f["x"] * R.rho(f["x"], 1e-5) * f["w_pre"]
    wt = R.gate(m0 @ f["w_r"].t(), ids, score_fn, 1)
    out = torch.zeros_like(m0)
    for e in range(E):
        for k in range(K):
            t = torch.nonzero(ids[:, k] == e)[:, 0]
            hh = m0[t] @ f["w13"][e].t()
            o = (R.silu(hh[:, :I]) * hh[:, I:]) @ f["w2"][e].t()
            out = out.index_add(0, t, wt[t, k, None] * o)
    if shared:
        out = out + f["sh"]
    ref = R.block_norm(out, f["x"], f["w_post"], f.get("gate"), f["w_next"], 1e-5, 0.8)
    for name, lib, r64 in (("h", h, ref[0]), ("n", n, ref[1])):
        assert (lib.double() - r64).norm() <= 20 * 2.0 ** -8 * r64.norm(), name
    loss = (ref[0] * dh.double()).sum() + (ref[1] * dn.double()).sum()
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    for k, v in want.items():
        err = (got[k].double() - v).norm() / v.norm()
        assert err <= 20 * 2.0 ** -8, (k, err.item())


def check_products(c):
    """The five products of one case against 64-bit products of the same inputs."""
    H, I, E = c.cfg.H, c.cfg.I, c.cfg.E
    t = product_tensors(c)
    dh = c.rows(2 * I, 0.1)
    h13, act = moe.grouped_gate_up_train(c.cfg, t["x"], t["w13"], c.off, c.ws, h13=t["h13"], act=t["act"])
    dx = moe.grouped_gate_up_grad(c.cfg, dh, t["w13"], c.off, c.ws, dx_perm=t["dx"])
    dh2 = moe.grouped_down_grad(c.cfg, t["dy"], t["w2"], h13, c.off, c.ws, dh13=t["dh"])
    c.done(h13, act, dx, dh2)
    for out, a, w in ((h13, t["x"], t["w13"].transpose(1, 2)), (dx, dh, t["w13"])):
        v, m = c.each(lambda e, s: dot(a[s], w[e]), out.shape[1])
        acc = R.product_bound(w.shape[1], m)
        R.close(out[:c.P], v, HALF * (v.abs() + acc) + acc)
    v, m = c.each(lambda e, s: dot(t["dy"][s], t["w2"][e]), I)
    acc = R.product_bound(H, m)
    g, u = R.f64(h13[:c.P, :I]), R.f64(h13[:c.P, I:])
    ref = v * R.silu(g)
    e = R.silu(g).abs() * (acc + (v.abs() + acc) * 2.0 ** -20 * (1 + g.abs()))
    R.close(dh2[:c.P, I:], ref, HALF * (ref.abs() + e) + e, "du")
    for out, d, r in ((moe.grouped_down_wgrad(c.cfg, t["dy"], act, c.off, c.ws), t["dy"], act),
                      (moe.grouped_gate_up_wgrad(c.cfg, dh, t["x"], c.off, c.ws), dh, t["x"])):
        for e in range(E):
            a, b = c.seg[e], c.seg[e + 1]
            v, m = dot(d[a:b].t(), r[a:b])
            acc = R.product_bound(b - a, m.cpu())
            R.close(out[e], v.cpu(), HALF * (v.cpu().abs() + acc) + acc, f"expert {e}")
    moe.check_status(c.ws)


def uneven(T, E, K, seed):
    """Ids whose experts differ a hundredfold in tokens; some have none."""
    g = gen(seed)
    pref = -2.5 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    pref = pref[torch.randperm(E, generator=g, device="cuda")]
    return torch.topk(torch.randn((T, E), generator=g, device="cuda") + pref, K, dim=1).indices.int()


@pytest.mark.parametrize("T,H,E,K,I", [(1500, 1024, 40, 2, 264), (900, 520, 64, 4, 192), (2500, 640, 9, 3, 384)])
def test_uneven_experts(T, H, E, K, I):
    """Many and few rows side by side: streaming and resident weight-gradient units, mixed tile order."""
    check_products(Case(T, H, E, K, I, ids=uneven(T, E, K, T)))


def test_the_most_experts():
    check_products(Case(100, 64, 1024, 8, 72, seed=3))


@pytest.mark.parametrize("setting", ["contiguous split tail", "plain stream order"])
def test_schedules(setting):
    L = moe.lib()
    try:
        if setting == "contiguous split tail":
            assert L.moe_set_split_tail(0) == 0
        else:
            L.moe_set_programmatic_launch(0)
        check_products(Case(500, 1024, 6, 2, 520, seed=4))
    finally:
        L.moe_set_split_tail(1)
        L.moe_set_programmatic_launch(1)

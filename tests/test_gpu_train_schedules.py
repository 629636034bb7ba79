"""Every output of the experts' products of a training step where their order
of work is unusual (experts of very different sizes, the most experts, the
contiguous split of the last tiles, plain stream order), and after a wait that
ran out."""
import pytest
import torch

import mixture_experts_layer_61_b200 as moe
import train_ref as R
from test_gpu_train_products import BF, HALF, Case, dot, product_tensors, uneven

pytestmark = pytest.mark.gpu


def check(c):
    """gate_up_train's activations and both halves of the down gradient against 64-bit products, with the bounds of
    test_gate_up_train and test_down_grad (where their terms are explained)."""
    H, I = c.cfg.H, c.cfg.I
    t = product_tensors(c)
    h13, act = moe.grouped_gate_up_train(c.cfg, t["x"], t["w13"], c.off, c.ws, h13=t["h13"], act=t["act"])
    keep = h13.clone()
    dh = moe.grouped_down_grad(c.cfg, t["dy"], t["w2"], h13, c.off, c.ws, dh13=t["dh"])
    c.done(h13, act, dh)
    same = moe.grouped_down_grad(c.cfg, t["dy"], t["w2"], h13, c.off, c.ws, dh13=h13)  # in place
    c.done(same)
    assert torch.equal(same[:c.P], dh[:c.P])

    v, m = c.each(lambda e, s: dot(t["x"][s], t["w13"][e].t()), 2 * I)
    acc = R.product_bound(H, m)
    R.close(keep[:c.P], v, HALF * (v.abs() + acc) + acc, "h13")
    g, u = v[:, :I], v[:, I:]
    ref = R.silu(g) * u
    e = 1.1 * u.abs() * acc[:, :I] + R.silu(g).abs() * acc[:, I:] + 1.1 * acc[:, :I] * acc[:, I:]
    e = e + ref.abs() * 2.0 ** -20 * (1 + g.abs())
    R.close(act[:c.P], ref, HALF * (ref.abs() + e) + e, "act")

    da, m = c.each(lambda e, s: dot(t["dy"][s], t["w2"][e]), I)
    acc = R.product_bound(H, m)
    g, u = R.f64(keep[:c.P, :I]), R.f64(keep[:c.P, I:])
    s = torch.sigmoid(g)
    ds = 2.0 ** -20 * (1 + g.abs())
    ref = da * u * R.silu_grad(g)
    e = u.abs() * R.silu_grad(g).abs() * acc + (da.abs() + acc) * u.abs() * s * ds * (2 + 2 * g.abs())
    R.close(dh[:c.P, :I], ref, HALF * (ref.abs() + e) + e, "dg")
    ref = da * R.silu(g)
    e = R.silu(g).abs() * (acc + (da.abs() + acc) * ds)
    R.close(dh[:c.P, I:], ref, HALF * (ref.abs() + e) + e, "du")


@pytest.mark.parametrize("T,H,E,K,I", [(1500, 1024, 40, 2, 264), (900, 520, 64, 4, 192), (2500, 640, 9, 3, 384)])
def test_uneven_experts(T, H, E, K, I):
    check(Case(T, H, E, K, I, ids=uneven(T, E, K, T)))


def test_the_most_experts():
    check(Case(100, 64, 1024, 8, 72, seed=3))


@pytest.mark.parametrize("setting", ["contiguous split tail", "plain stream order"])
def test_schedules(setting):
    L = moe.lib()
    try:
        if setting == "contiguous split tail":
            assert L.moe_set_split_tail(0) == 0
        else:
            L.moe_set_programmatic_launch(0)
        check(Case(500, 1024, 6, 2, 520, seed=4))
    finally:
        L.moe_set_split_tail(1)
        L.moe_set_programmatic_launch(1)


@pytest.mark.parametrize("which", ["gate_up_train", "down_grad", "gate_up_grad", "down_wgrad", "gate_up_wgrad"])
def test_after_a_wait_that_ran_out_the_next_call_is_whole(which):
    """Every output of the call after the one that reported MOE_ERR_TIMEOUT, bit for bit that of the call before."""
    c = Case(300, 256, 4, 2, 256)
    t = product_tensors(c)
    h, a = c.rows(512), c.rows(256)
    run = {
        "gate_up_train": lambda: moe.grouped_gate_up_train(c.cfg, t["x"], t["w13"], c.off, c.ws),
        "down_grad": lambda: (moe.grouped_down_grad(c.cfg, t["dy"], t["w2"], h, c.off, c.ws),),
        "gate_up_grad": lambda: (moe.grouped_gate_up_grad(c.cfg, h, t["w13"], c.off, c.ws),),
        "down_wgrad": lambda: (moe.grouped_down_wgrad(c.cfg, t["dy"], a, c.off, c.ws),),
        "gate_up_wgrad": lambda: (moe.grouped_gate_up_wgrad(c.cfg, h, t["x"], c.off, c.ws),)}[which]
    whole = (lambda o: o) if which.endswith("wgrad") else (lambda o: o[:c.P])  # rows past P are not written
    want = [whole(o).clone() for o in run()]
    moe.check_status(c.ws)
    assert all(o.any() for o in want)
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
    for o, w in zip(again, want):
        assert torch.equal(whole(o), w)

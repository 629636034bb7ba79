"""The closed-form gradients of train_ref.py against central differences of
their forwards (float64, CPU): the step 1e-5 leaves a truncation error of the
order 1e-10 of the third derivatives and a rounding error of 1e-16 / 1e-5."""
import itertools

import pytest
import torch

import train_ref as R


def _diff(f, x, d, eps=1e-5):
    """d/dx of <f(x), d> by central differences."""
    g = torch.zeros_like(x)
    flat, gf = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + eps
        a = (f() * d).sum()
        flat[i] = keep - eps
        b = (f() * d).sum()
        flat[i] = keep
        gf[i] = (a - b) / (2 * eps)
    return g


def _rand(*shape, seed=0):
    return torch.randn(shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("post,gate_mode,nxt", list(itertools.product([False, True], [0, 1, 2], [False, True])))
def test_block_norm_gradient(post, gate_mode, nxt):
    T, H, eps, scale = 3, 5, 1e-3, 0.7
    y, r = _rand(T, H, seed=1), _rand(T, H, seed=2)
    wp = 1 + 0.3 * _rand(H, seed=3) if post else None
    g = None if gate_mode == 0 else _rand(*((H,) if gate_mode == 1 else (T, H)), seed=4)
    wn = 1 + 0.3 * _rand(H, seed=5) if nxt else None
    dh, dn = _rand(T, H, seed=6), _rand(T, H, seed=7) if nxt else None

    def f():
        h, n, _ = R.block_norm(y, r, wp, g, wn, eps, scale)
        return torch.stack([h, n]) if nxt else h

    h, _, _ = R.block_norm(y, r, wp, g, wn, eps, scale)
    got = R.block_norm_grad(h, dh, dn, y, wp, g, wn, eps, scale)
    d = torch.stack([dh, dn]) if nxt else dh
    for name, x in (("dy", y), ("dresidual", r), ("dw_post", wp), ("dgate", g), ("dw_next", wn)):
        if x is not None:
            ref = _diff(f, x, d)
            assert (got[name] - ref).abs().max() < 1e-7, name
            assert (got[name].abs() <= got[name + "|"] * (1 + 1e-12)).all(), name


@pytest.mark.parametrize("score_fn,renorm", list(itertools.product([0, 1], [0, 1])))
def test_gate_gradient(score_fn, renorm):
    l = _rand(4, 6, seed=8)
    ids = torch.tensor([[0, 3], [5, -1], [-1, -1], [2, 1]], dtype=torch.int32)
    dw = _rand(4, 2, seed=9)
    got, mag = R.gate_grad(l, ids, dw, score_fn, renorm)
    ref = _diff(lambda: R.gate(l, ids, score_fn, renorm), l, dw)
    assert (got - ref).abs().max() < 1e-8
    assert (got.abs() <= mag * (1 + 1e-12)).all()


def test_combine_gradient():
    T, K, H, P = 3, 2, 4, 8
    y, w, sh = _rand(P, H, seed=1), _rand(T, K, seed=2), _rand(T, H, seed=3)
    pos = torch.tensor([4, 0, -1, 7, 2, -1], dtype=torch.int32)
    d = _rand(T, H, seed=4)
    f = lambda: R.combine(y, pos, w, sh)[0]
    rows, dw, _ = R.combine_grad(d, y, pos, w)
    dy = torch.zeros_like(y)
    for a in range(T * K):
        if pos[a] >= 0:
            dy[pos[a]] = rows.view(T * K, H)[a]
    assert (dy - _diff(f, y, d)).abs().max() < 1e-8
    assert (dw - _diff(f, w, d)).abs().max() < 1e-8


def test_swiglu_gradient():
    g = torch.linspace(-30, 30, 301, dtype=torch.float64)
    ref = _diff(lambda: R.silu(g), g, torch.ones_like(g))
    # each of the two sums runs over 301 values of total magnitude S < 4600 in
    # a tree of at most 9 levels, so it is off by at most 9 * 2^-53 S = 4.6e-12;
    # two of them over the step 2e-5: 4.6e-7 (and 1e-10 of truncation)
    assert R.silu(g).abs().sum() < 4600
    assert (R.silu_grad(g) - ref).abs().max() < 4.7e-7

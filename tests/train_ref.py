"""64-bit forms of the training operators for the tests: the forwards and their
gradients in closed form (torch, float64, CPU).  The closed forms are checked
against central differences of the forwards in test_train_ref.py.

Error bounds.  An output of type t is rounded once: at most half a step,
HALF[t] relative to its value.  What precedes is fp32 arithmetic on sums whose
longest serial chain in the row kernels is 32 terms, then at most 10 levels of
a tree (and, for the column sums, the tokens of one block and 148 blocks): an
error below 2^-17 of the sum of the terms' magnitudes, which also covers the
few single operations and approximate reciprocal roots around it
(64 * 2^-24 = 2^-18, plus as much again).  FP32 below is that 2^-17."""
from __future__ import annotations

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FP32 = 2.0 ** -17


def f64(t):
    return None if t is None else t.detach().double().cpu()


def rounded(ref, dtype, mag):
    """Bound on |out - ref|: one rounding, fp32 arithmetic on terms of total magnitude mag."""
    return HALF[dtype] * (ref.abs() + FP32 * mag) + FP32 * mag


def close(out, ref, bound, what=""):
    out, bad = out.detach().double().cpu(), None
    assert out.shape == ref.shape, (what, out.shape, ref.shape)
    err = (out - ref).abs()
    ok = (err <= bound) | ((out == ref))
    if not bool(ok.all()):
        i = int(torch.argmax(torch.where(ok, torch.zeros_like(err), err - bound).nan_to_num(nan=float("inf"))))
        bad = (out.flatten()[i].item(), ref.flatten()[i].item(), bound.expand_as(ref).flatten()[i].item())
    assert bad is None, f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds; worst (out, ref, bound) {bad}"


# ---------------------------------------------------------------- block norm
def rho(x, eps):
    return (x.pow(2).mean(1, keepdim=True) + eps).rsqrt()


def block_norm(y, residual, w_post, gate, w_next, eps, scale):
    """(h, n, |terms of h|)"""
    z = y
    if y is not None and w_post is not None:
        z = y * rho(y, eps) * w_post
    if gate is not None:
        z = gate * z
    h = torch.zeros_like(z if z is not None else residual)
    mag = torch.zeros_like(h)
    if residual is not None:
        h, mag = h + scale * residual, mag + (scale * residual).abs()
    if z is not None:
        h, mag = h + z, mag + z.abs()
    n = None if w_next is None else h * rho(h, eps) * w_next
    return h, n, mag


def block_norm_grad(h, dh, dn, y, w_post, gate, w_next, eps, scale):
    """Gradients and, under the same names with "|", the magnitudes their sums run over."""
    out = {}
    some = dh if dh is not None else dn
    d = torch.zeros_like(some) if dh is None else dh.clone()
    m = d.abs()
    if dn is not None:
        r, g = rho(h, eps), w_next * dn
        coef, acoef = (g * h).mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
        d = d + r * (g - h * r * r * coef)
        m = m + r * (g.abs() + h.abs() * r * r * acoef)
        out["dw_next"], out["dw_next|"] = (dn * h * r).sum(0), (dn * h * r).abs().sum(0)
    out["dresidual"], out["dresidual|"] = scale * d, abs(scale) * m
    if y is None:
        return out
    r = rho(y, eps) if w_post is not None else torch.ones_like(y[:, :1])
    wp = w_post if w_post is not None else torch.ones_like(y[0])
    g = gate if gate is not None else torch.ones_like(y[0])
    z = y * r * wp
    if gate is not None:
        dg, ag = d * z, m * z.abs()
        out["dgate"], out["dgate|"] = (dg, ag) if gate.dim() == 2 else (dg.sum(0), ag.sum(0))
    dz, az = g * d, g.abs() * m
    if w_post is not None:
        out["dw_post"], out["dw_post|"] = (dz * y * r).sum(0), (az * (y * r).abs()).sum(0)
        k, ak = (wp * dz * y).mean(1, keepdim=True), ((wp * y).abs() * az).mean(1, keepdim=True)
        out["dy"] = r * (wp * dz - y * r * r * k)
        out["dy|"] = r * (wp.abs() * az + y.abs() * r * r * ak)
    else:
        out["dy"], out["dy|"] = dz, az
    return out


# ------------------------------------------------------- dispatch and combine
def combine(y_perm, pos, w, shared=None):
    """(out, |terms|)"""
    T, K = w.shape
    p = pos.view(T, K).long()
    rows = y_perm[p.clamp(min=0)] * (p >= 0)[..., None]
    t = w[..., None] * rows
    out, mag = t.sum(1), t.abs().sum(1)
    return (out, mag) if shared is None else (out + shared, mag + shared.abs())


def combine_grad(dout, y_perm, pos, w):
    """(dy rows by slot [T, K, H], dw, |terms of dw|)"""
    T, K = w.shape
    p = pos.view(T, K).long()
    have = (p >= 0)[..., None]
    rows = torch.where(have, y_perm[p.clamp(min=0)], torch.zeros((), dtype=y_perm.dtype))
    t = dout[:, None, :] * rows
    return w[..., None] * dout[:, None, :] * have, t.sum(2), t.abs().sum(2)


# ----------------------------------------------------------------------- gate
def gate(l, ids, score_fn, renorm):
    have = ids >= 0
    sel = l.gather(1, ids.clamp(min=0).long())
    if score_fn == 1:
        w = torch.where(have, torch.sigmoid(sel), torch.zeros_like(sel))
    elif renorm:
        w = torch.where(have, torch.exp(sel - l.amax(1, keepdim=True)), torch.zeros_like(sel))
    else:
        return torch.where(have, torch.softmax(l, 1).gather(1, ids.clamp(min=0).long()), torch.zeros_like(sel))
    if renorm:
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s > 0, s, torch.ones_like(s))
    return w


def gate_grad(l, ids, dw, score_fn, renorm):
    """(dlogits, |terms|)"""
    have = ids >= 0
    i = ids.clamp(min=0).long()
    dw = torch.where(have, dw, torch.zeros_like(dw))
    w = gate(l, ids, score_fn, renorm)
    mean, amean = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    if score_fn == 0 and not renorm:
        p = torch.softmax(l, 1)
        full = torch.zeros_like(l).scatter_add_(1, i, dw)
        afull = torch.zeros_like(l).scatter_add_(1, i, dw.abs())
        return p * (full - mean), p * (afull + amean)
    c = torch.ones_like(w) if score_fn == 0 else torch.sigmoid(-l.gather(1, i))
    d = w * c * ((dw - mean) if renorm else dw)
    a = w * c * ((dw.abs() + amean) if renorm else dw.abs())
    z = torch.zeros_like(l)
    return z.scatter_add(1, i, torch.where(have, d, torch.zeros_like(d))), \
        z.scatter_add(1, i, torch.where(have, a, torch.zeros_like(a)))


# ------------------------------------------------------------------- products
def silu(g):
    return g * torch.sigmoid(g)


def silu_grad(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


def product_bound(k, mag):
    """fp32 accumulation of products of total magnitude mag over k terms on the
    tensor cores: 16 products an instruction, k / 16 instructions in sequence
    and at most 16 additions inside one (and 4 partial sums of a split tile),
    each losing at most 2^-23 (truncation) of a partial sum below mag."""
    return (k / 16 + 24) * 2.0 ** -23 * mag

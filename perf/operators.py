"""The training half of the MoE block as measured cases: the gradients of the
token dispatch and combine, the norms around the block (with its gate and
residual scale) and their gradient, and the gradients of the experts' products.

`run` computes a case in plain torch operations (fp32, rounded once) or, with
`own` set, through the library's entry points.  `exact` gives the same outputs
in 64 bits from the definitions.
"""
import math

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------- cases

def _case(name, op, T, H, E=8, K=2, I=512, B=16, dtype="bf16", score=0, renorm=1, dyn=False, skew=1.0, post=True,
          gate=1, nxt=True, shared=False, res=1.0, add=False):
    """op: which entry point; T tokens, H hidden, E experts, K per token, I
    expert width, B padding tile; score/renorm: the gate's function; dyn:
    per-token expert counts (empty slots); skew: how uneven the experts' loads
    are; post/gate/nxt/shared/res: the norm's parts; add: a further gradient
    summed into the permute's."""
    c = dict(op=op, T=T, H=H, E=E, K=K, I=I, B=B, dtype=dtype, score=score, renorm=renorm, dyn=dyn, skew=skew,
             post=post, gate=gate, nxt=nxt, shared=shared, res=res, add=add)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of the Mixtral-shaped layer: combine, residual and the next block's norm
        _case("combine_norm_mixtral_T1", "combine_norm", 1, 4096, E=8, K=2, post=False, gate=0),
        # prefill of the Qwen2-MoE-shaped layer: shared experts, a norm after the block, channel gate
        _case("combine_norm_qwen2moe_T2048", "combine_norm", 2048, 3584, E=64, K=8, shared=True, res=0.5),
        # training step of the widest hidden size, every part of the norm
        _case("block_norm_grad_T4096_H7168", "block_norm_grad", 4096, 7168, gate=1, res=0.7),
        # odd row count and width, fp32, a gate per token and channel
        _case("block_norm_grad_fp32_T333_H1000", "block_norm_grad", 333, 1000, dtype="fp32", gate=2),
        # the tiny fp32 layer's combine gradient: latency
        _case("combine_grad_fp32_tiny", "combine_grad", 64, 256, E=8, K=2, dtype="fp32"),
        # training batch of the DeepSeek-V3-shaped layer: eight rows of 7168 per token
        _case("combine_grad_deepseekv3_T4096", "combine_grad", 4096, 7168, E=256, K=8),
        # the same layer's dispatch gradient with the shared branch's gradient added
        _case("permute_grad_deepseekv3_T4096", "permute_grad", 4096, 7168, E=256, K=8, add=True),
        # sigmoid gate over 256 experts, ragged per-token counts
        _case("route_grad_sigmoid_T2048_E256", "route_grad", 2048, 7168, E=256, K=8, score=1, dyn=True),
        # Mixtral-shaped training batch: gradient through the down projection and SwiGLU
        _case("down_grad_mixtral_T2048", "down_grad", 2048, 4096, E=8, K=2, I=14336),
        # Qwen2-MoE-shaped training batch: gradient of the permuted tokens
        _case("gate_up_grad_qwen2moe_T2048", "gate_up_grad", 2048, 3584, E=64, K=8, I=2560),
        # the same batch's gate/up weight gradients
        _case("gate_up_wgrad_qwen2moe_T2048", "gate_up_wgrad", 2048, 3584, E=64, K=8, I=2560),
        # odd sizes, per-token counts, very uneven experts (some without a token)
        _case("down_wgrad_odd_T777", "down_wgrad", 777, 1000, E=13, K=3, I=1544, dyn=True, skew=3.0),
    ]


_OPS = ("combine_norm", "block_norm", "block_norm_grad", "combine_grad", "permute_grad", "route_grad", "gate_up_train",
        "down_grad", "gate_up_grad", "down_wgrad", "gate_up_wgrad")


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(_OPS)
    E = rng.choice((4, 5, 8, 16, 33, 64, 128, 256))
    K = min(E, rng.choice((1, 2, 3, 4, 8)))
    product = op in ("gate_up_train", "down_grad", "gate_up_grad", "down_wgrad", "gate_up_wgrad")
    c = _case(None, op, T=_logint(rng, 1, 4096), H=8 * _logint(rng, 8, 896), E=E, K=K, I=8 * _logint(rng, 8, 640),
              B=rng.choice((16, 32, 64, 128)), dtype="bf16" if product else rng.choice(("bf16", "bf16", "fp32")),
              score=rng.randrange(2), renorm=rng.randrange(2), dyn=rng.random() < 0.3, skew=rng.uniform(0.0, 3.0),
              post=rng.random() < 0.6, gate=rng.randrange(3), nxt=rng.random() < 0.8, shared=rng.random() < 0.5,
              res=rng.choice((1.0, 0.5, 0.1)), add=rng.random() < 0.5)
    if product:  # weights and products at most the largest listed ones
        while c["E"] > 64 or c["E"] * c["H"] * c["I"] > 64 * 3584 * 2560:
            c["E"] //= 2
        c["K"] = min(c["K"], c["E"])
        while c["T"] * c["K"] * c["H"] * c["I"] > 16384 * 3584 * 2560:
            c["T"] //= 2
    return c


# -------------------------------------------------------------------- inputs

def _pmax(c):
    A = c["T"] * c["K"]
    return max(A + min(c["E"], A) * (c["B"] - 1), 1)


def _align(ids, E, B, P_max):
    """Block-wise padded segments of the assignments, experts ascending."""
    A = ids.numel()
    flat = ids.reshape(-1).long()
    valid = flat >= 0
    counts = torch.bincount(flat[valid], minlength=E)
    padded = (counts + B - 1) // B * B
    offs = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offs[1:] = padded.cumsum(0)
    order = torch.argsort(torch.where(valid, flat, torch.full_like(flat, E)), stable=True)[: int(valid.sum())]
    first = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    first[1:] = counts.cumsum(0)
    e = flat[order]
    p = offs[e] + torch.arange(order.numel(), device=ids.device) - first[e]
    pos = torch.full((A,), -1, dtype=torch.long, device=ids.device)
    pos[order] = p
    sorted_ids = torch.full((P_max,), -1, dtype=torch.long, device=ids.device)
    sorted_ids[p] = order
    scalars = torch.zeros(4, dtype=torch.int32, device=ids.device)
    scalars[0] = offs[E]
    scalars[1] = (counts > 0).sum()
    return dict(pos=pos.int(), sorted_ids=sorted_ids.int(), offsets=offs.int(), scalars=scalars,
                rows=int(offs[E]), seg=[int(v) for v in offs.tolist()])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, H, E, K, I, B, op = c["T"], c["H"], c["E"], c["K"], c["I"], c["B"], c["op"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def randn(*shape, std=1.0, dtype=dt):
        t = torch.randn(shape, generator=g, device="cuda")
        return t.mul_(std).to(dtype)

    s = dict(c, out={})
    P_max = _pmax(c)
    routed = op not in ("block_norm", "block_norm_grad")
    if routed:
        # a trained router's logits: a preference for some experts plus the token's own
        pref = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        pref = pref[torch.randperm(E, generator=g, device="cuda")]
        logits = torch.randn((T, E), generator=g, device="cuda") + pref
        val, ids = torch.sort(logits, dim=1, descending=True, stable=True)
        val, ids = val[:, :K].contiguous(), ids[:, :K].int().contiguous()
        if c["dyn"]:
            kt = torch.randint(0, K + 1, (T, 1), generator=g, device="cuda")
            empty = torch.arange(K, device="cuda")[None, :] >= kt
            ids = torch.where(empty, torch.full_like(ids, -1), ids)
        al = _align(ids, E, B, P_max)
        w = torch.softmax(val, 1)
        w = torch.where(ids >= 0, w, torch.zeros_like(w)).contiguous()
        s.update(al, ids=ids, w=w, logits=logits)
        del s["seg"]
        s["seg"] = al["seg"]
        real = (al["sorted_ids"] >= 0)[:, None]

    def rows(width, std=1.0):
        """Permuted rows: zero in the padding slots, as the permute and the gradients leave them."""
        return torch.where(real, randn(P_max, width, std=std), torch.zeros((), dtype=dt, device="cuda"))

    if op in ("combine_norm", "block_norm", "block_norm_grad"):
        s["residual"] = randn(T, H)
        s["w_post"] = (1 + 0.1 * randn(H, dtype=torch.float32)).to(dt) if c["post"] else None
        s["gate"] = None if c["gate"] == 0 else randn(*((H,) if c["gate"] == 1 else (T, H)), std=0.5)
        s["w_next"] = (1 + 0.1 * randn(H, dtype=torch.float32)).to(dt) if c["nxt"] else None
    if op == "combine_norm":
        s["y_perm"] = rows(H)
        s["shared"] = randn(T, H) if c["shared"] else None
    if op == "block_norm":
        s["y"] = randn(T, H)
    if op == "block_norm_grad":
        s["y"], s["h"] = randn(T, H), randn(T, H, std=2.0)
        s["dh"] = randn(T, H, std=0.1)
        s["dn"] = randn(T, H, std=0.1) if c["nxt"] else None
    if op == "combine_grad":
        s["dout"], s["y_perm"] = randn(T, H, std=0.1), rows(H)
        s["out"]["dy_perm"] = torch.zeros((P_max, H), dtype=dt, device="cuda")
    if op == "permute_grad":
        s["dx_perm"] = rows(H, std=0.1)
        s["dx_add"] = randn(T, H, std=0.1) if c["add"] else None
    if op == "route_grad":
        s["dw"] = randn(T, K, dtype=torch.float32)
    if op == "gate_up_train":
        s["x_perm"] = rows(H)
        s["out"]["h13"] = torch.zeros((P_max, 2 * I), dtype=dt, device="cuda")
        s["out"]["act"] = torch.zeros((P_max, I), dtype=dt, device="cuda")
    if op in ("gate_up_train", "gate_up_grad"):
        s["w13"] = randn(E, 2 * I, H, std=1 / math.sqrt(H))
    if op == "down_grad":
        s["dy_perm"], s["h13"] = rows(H, std=0.1), rows(2 * I)
        s["w2"] = randn(E, H, I, std=1 / math.sqrt(I))
        s["out"]["dh13"] = torch.zeros((P_max, 2 * I), dtype=dt, device="cuda")
    if op == "gate_up_grad":
        s["dh13"] = rows(2 * I, std=0.1)
        s["out"]["dx_perm"] = torch.zeros((P_max, H), dtype=dt, device="cuda")
    if op == "down_wgrad":
        s["dy_perm"], s["act"] = rows(H, std=0.1), rows(I)
    if op == "gate_up_wgrad":
        s["dh13"], s["x_perm"] = rows(2 * I, std=0.1), rows(H)

    if own:
        import mixture_experts_layer_61_b200 as moe

        if routed:
            s["cfg"] = moe.config(T, H, E, K, I, tile_B=B, score_fn=c["score"], renorm=c["renorm"], dtype=dt)
            s["ws"] = moe.alloc_workspace(moe.gemm_workspace_size())
        if op in ("combine_norm", "block_norm", "block_norm_grad"):
            s["nc"] = moe.norm_config(T, H, eps=EPS, res_scale=c["res"], gate_mode=c["gate"], dtype=dt)
        if op == "block_norm_grad":
            s["ws"] = moe.alloc_workspace(moe.block_norm_grad_workspace_size(s["nc"]))
    return s


# ----------------------------------------------------------------- the passes

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    import mixture_experts_layer_61_b200 as moe

    op, out = s["op"], s["out"]
    if op == "combine_norm":
        h, n, y = moe.combine_norm(s["cfg"], s["nc"], s["y_perm"], s["pos"], s["w"], shared_out=s["shared"],
                                   residual=s["residual"], w_post=s["w_post"], gate=s["gate"], w_next=s["w_next"],
                                   save_y=True)
        return {"h": h, "n": n, "y": y} if n is not None else {"h": h, "y": y}
    if op == "block_norm":
        h, n = moe.block_norm(s["nc"], residual=s["residual"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                              w_next=s["w_next"])
        return {"h": h, "n": n} if n is not None else {"h": h}
    if op == "block_norm_grad":
        r = moe.block_norm_grad(s["nc"], s["ws"], h=s["h"], dh=s["dh"], dn=s["dn"], y=s["y"], w_post=s["w_post"],
                                gate=s["gate"], w_next=s["w_next"])
        return {k: v for k, v in r.items() if v is not None}
    if op == "combine_grad":
        dy, dw = moe.combine_grad(s["cfg"], s["dout"], s["y_perm"], s["pos"], s["w"], s["sorted_ids"], s["scalars"],
                                  dy_perm=out["dy_perm"])
        return {"dy_perm": dy, "dw": dw}
    if op == "permute_grad":
        return moe.permute_grad(s["cfg"], s["dx_perm"], s["pos"], dx_add=s["dx_add"])
    if op == "route_grad":
        return moe.route_grad(s["cfg"], s["logits"], s["ids"], s["dw"])
    if op == "gate_up_train":
        h13, act = moe.grouped_gate_up_train(s["cfg"], s["x_perm"], s["w13"], s["offsets"], s["ws"], h13=out["h13"],
                                             act=out["act"])
        return {"h13": h13, "act": act}
    if op == "down_grad":
        return moe.grouped_down_grad(s["cfg"], s["dy_perm"], s["w2"], s["h13"], s["offsets"], s["ws"],
                                     dh13=out["dh13"])
    if op == "gate_up_grad":
        return moe.grouped_gate_up_grad(s["cfg"], s["dh13"], s["w13"], s["offsets"], s["ws"], dx_perm=out["dx_perm"])
    if op == "down_wgrad":
        return moe.grouped_down_wgrad(s["cfg"], s["dy_perm"], s["act"], s["offsets"], s["ws"])
    if op == "gate_up_wgrad":
        return moe.grouped_gate_up_wgrad(s["cfg"], s["dh13"], s["x_perm"], s["offsets"], s["ws"])
    raise ValueError(op)


def _gathered(rows, pos, T, K):
    """[T, K, H] fp32 rows of the assignments, zero for empty slots."""
    p = pos.long().view(T, K)
    r = rows.float()[p.clamp(min=0)]
    return r * (p >= 0)[..., None]


def _rms(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _plain_norm(s, y):
    dt = s["residual"].dtype
    z = y if s["w_post"] is None else y * _rms(y) * s["w_post"].float()
    if s["gate"] is not None:
        z = s["gate"].float() * z
    h = s["res"] * s["residual"].float() + z
    out = {"h": h.to(dt)}
    if s["w_next"] is not None:
        out["n"] = (h * _rms(h) * s["w_next"].float()).to(dt)
    return out


def _plain_block_norm(s):
    return _plain_norm(s, s["y"].float())


def _plain_combine_norm(s):
    T, K = s["T"], s["K"]
    y = (_gathered(s["y_perm"], s["pos"], T, K) * s["w"][..., None]).sum(1)
    if s["shared"] is not None:
        y = y + s["shared"].float()
    out = _plain_norm(s, y)
    out["y"] = y.to(s["y_perm"].dtype)
    return out


def _plain_block_norm_grad(s):
    dt = s["y"].dtype
    d = s["dh"].float()
    out = {}
    if s["w_next"] is not None:
        h, dn, w = s["h"].float(), s["dn"].float(), s["w_next"].float()
        r = _rms(h)
        out["dw_next"] = (dn * h * r).sum(0)
        wd = w * dn
        d = d + r * (wd - h * r * r * (wd * h).mean(1, keepdim=True))
    out["dresidual"] = (s["res"] * d).to(dt)
    y = s["y"].float()
    if s["w_post"] is not None:
        ry, wp = _rms(y), s["w_post"].float()
        z = y * ry * wp
    else:
        z = y
    dz = d
    if s["gate"] is not None:
        dgate = d * z
        out["dgate"] = dgate.sum(0) if s["gate"].dim() == 1 else dgate.to(dt)
        dz = d * s["gate"].float()
    if s["w_post"] is not None:
        out["dw_post"] = (dz * y * ry).sum(0)
        wd = wp * dz
        dz = ry * (wd - y * ry * ry * (wd * y).mean(1, keepdim=True))
    out["dy"] = dz.to(dt)
    return out


def _plain_combine_grad(s):
    T, K = s["T"], s["K"]
    do = s["dout"].float()
    dw = (_gathered(s["y_perm"], s["pos"], T, K) * do[:, None, :]).sum(2)
    rows = (s["w"][..., None] * do[:, None, :]).to(s["dout"].dtype).view(T * K, -1)
    dy = torch.zeros_like(s["y_perm"])
    have = s["pos"] >= 0
    dy[s["pos"][have].long()] = rows[have]
    return {"dy_perm": dy, "dw": dw}


def _plain_permute_grad(s):
    dx = _gathered(s["dx_perm"], s["pos"], s["T"], s["K"]).sum(1)
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    return dx.to(s["dx_perm"].dtype)


def _plain_route_grad(s):
    have = s["ids"] >= 0
    idx = s["ids"].clamp(min=0).long()
    l, dw = s["logits"], torch.where(have, s["dw"], torch.zeros_like(s["dw"]))
    sel = torch.gather(l, 1, idx)
    if s["score"] == 0:
        if s["renorm"]:
            sel = torch.where(have, sel, torch.full_like(sel, -math.inf))
            m = torch.where(have.any(1, keepdim=True), sel.amax(1, keepdim=True), torch.zeros_like(sel[:, :1]))
            e = torch.exp(sel - m)
            w = e / e.sum(1, keepdim=True).clamp(min=1e-30)
            d = w * (dw - (w * dw).sum(1, keepdim=True))
        else:
            e = torch.exp(l - l.amax(1, keepdim=True))
            p = e / e.sum(1, keepdim=True)
            full = torch.zeros_like(l).scatter_add_(1, idx, dw)
            return p * (full - (p * full).sum(1, keepdim=True))
    else:
        sg = torch.where(have, 1 / (1 + torch.exp(-sel)), torch.zeros_like(sel))
        co = 1 / (1 + torch.exp(sel))
        if s["renorm"]:
            w = sg / sg.sum(1, keepdim=True).clamp(min=1e-30)
            d = w * co * (dw - (w * dw).sum(1, keepdim=True))
        else:
            d = sg * co * dw
    d = torch.where(have, d, torch.zeros_like(d))
    return torch.zeros_like(l).scatter_add_(1, idx, d)


def _segments(s):
    seg = s["seg"]
    return [(e, seg[e], seg[e + 1]) for e in range(s["E"]) if seg[e + 1] > seg[e]]


def _plain_gate_up_train(s):
    I = s["I"]
    h13, act = torch.zeros_like(s["out"]["h13"]), torch.zeros_like(s["out"]["act"])
    for e, a, b in _segments(s):
        h = s["x_perm"][a:b].float() @ s["w13"][e].float().t()
        g, u = h[:, :I], h[:, I:]
        h13[a:b] = h.to(h13.dtype)
        act[a:b] = (g / (1 + torch.exp(-g)) * u).to(act.dtype)
    return {"h13": h13, "act": act}


def _plain_down_grad(s):
    I = s["I"]
    out = torch.zeros_like(s["out"]["dh13"])
    for e, a, b in _segments(s):
        da = s["dy_perm"][a:b].float() @ s["w2"][e].float()
        g, u = s["h13"][a:b, :I].float(), s["h13"][a:b, I:].float()
        sg = 1 / (1 + torch.exp(-g))
        out[a:b, :I] = (da * u * sg * (1 + g * (1 - sg))).to(out.dtype)
        out[a:b, I:] = (da * g * sg).to(out.dtype)
    return out


def _plain_gate_up_grad(s):
    out = torch.zeros_like(s["out"]["dx_perm"])
    for e, a, b in _segments(s):
        out[a:b] = (s["dh13"][a:b].float() @ s["w13"][e].float()).to(out.dtype)
    return out


def _plain_wgrad(s, d, x):
    out = torch.zeros((s["E"], d.shape[1], x.shape[1]), dtype=d.dtype, device=d.device)
    for e, a, b in _segments(s):
        out[e] = (d[a:b].float().t() @ x[a:b].float()).to(out.dtype)
    return out


_PLAIN = {
    "combine_norm": _plain_combine_norm,
    "block_norm": _plain_block_norm,
    "block_norm_grad": _plain_block_norm_grad,
    "combine_grad": _plain_combine_grad,
    "permute_grad": _plain_permute_grad,
    "route_grad": _plain_route_grad,
    "gate_up_train": _plain_gate_up_train,
    "down_grad": _plain_down_grad,
    "gate_up_grad": _plain_gate_up_grad,
    "down_wgrad": lambda s: _plain_wgrad(s, s["dy_perm"], s["act"]),
    "gate_up_wgrad": lambda s: _plain_wgrad(s, s["dh13"], s["x_perm"]),
}


# ----------------------------------------------------------- 64-bit definitions

def _x_norm(x, w):
    ms = x.pow(2).sum(-1, keepdim=True) / x.shape[-1]
    return x / torch.sqrt(ms + EPS) * w


def _x_block(s, y, residual, w_post, gate, w_next):
    z = _x_norm(y, w_post) if w_post is not None else y
    h = residual * s["res"] + (z * gate if gate is not None else z)
    return h, (_x_norm(h, w_next) if w_next is not None else None)


def _d(t):
    return None if t is None else t.double()


def _x_combine(s):
    out = torch.zeros((s["T"], s["H"]), dtype=torch.float64, device="cuda")
    pos = s["pos"].long().view(s["T"], s["K"])
    for k in range(s["K"]):
        rows = torch.nonzero(pos[:, k] >= 0)[:, 0]
        out[rows] += s["w"][rows, k, None].double() * s["y_perm"][pos[rows, k]].double()
    return out if s["shared"] is None else out + s["shared"].double()


def _x_gate(s, l):
    """The gate weights of the selected logits; empty slots weigh nothing."""
    have = s["ids"] >= 0
    sel = l.gather(1, s["ids"].long().clamp(min=0))
    if s["score"] == 1:
        w = torch.sigmoid(sel) * have
        return w / w.sum(1, keepdim=True).where(have.any(1, keepdim=True), torch.ones_like(w[:, :1])) if s["renorm"] \
            else w
    if s["renorm"]:
        w = torch.exp(sel - l.detach().amax(1, keepdim=True)) * have
        return w / w.sum(1, keepdim=True).where(have.any(1, keepdim=True), torch.ones_like(w[:, :1]))
    return torch.softmax(l, 1).gather(1, s["ids"].long().clamp(min=0)) * have


def exact(case, seed):
    s = prepare(case, seed)
    op, T, H, I = s["op"], s["T"], s["H"], s["I"]
    if op in ("combine_norm", "block_norm"):
        y = _x_combine(s) if op == "combine_norm" else s["y"].double()
        h, n = _x_block(s, y, _d(s["residual"]), _d(s["w_post"]), _d(s["gate"]), _d(s["w_next"]))
        out = {"h": h}
        if n is not None:
            out["n"] = n
        if op == "combine_norm":
            out["y"] = y
        return out
    if op == "block_norm_grad":
        # through h as stored: n's part first, then the block's part with h's whole gradient
        out = {}
        d = s["dh"].double()
        if s["w_next"] is not None:
            h, w = s["h"].double().requires_grad_(), s["w_next"].double().requires_grad_()
            gh, out["dw_next"] = torch.autograd.grad(_x_norm(h, w), (h, w), s["dn"].double())
            d = d + gh
        leaves = {"dresidual": torch.zeros_like(d).requires_grad_(), "dy": s["y"].double().requires_grad_()}
        if s["gate"] is not None:
            leaves["dgate"] = s["gate"].double().requires_grad_()
        if s["w_post"] is not None:
            leaves["dw_post"] = s["w_post"].double().requires_grad_()
        h, _ = _x_block(s, leaves["dy"], leaves["dresidual"], leaves.get("dw_post"), leaves.get("dgate"), None)
        out.update(zip(leaves, torch.autograd.grad(h, list(leaves.values()), d)))
        order = ("dw_next", "dresidual", "dgate", "dw_post", "dy")
        return {k: out[k] for k in order if k in out}
    if op == "combine_grad":
        dy = torch.zeros((s["y_perm"].shape[0], H), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, s["K"]), dtype=torch.float64, device="cuda")
        slot = s["sorted_ids"].long()
        p = torch.nonzero(slot >= 0)[:, 0]
        for q in p.split(8192):
            a = slot[q]
            do = s["dout"][a // s["K"]].double()
            dy[q] = do * s["w"].view(-1)[a, None].double()
            dw.view(-1)[a] = torch.einsum("ph,ph->p", do, s["y_perm"][q].double())
        return {"dy_perm": dy, "dw": dw}
    if op == "permute_grad":
        slot = s["sorted_ids"].long()
        p = torch.nonzero(slot >= 0)[:, 0]
        dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        dx.index_add_(0, slot[p] // s["K"], s["dx_perm"][p].double())
        return dx if s["dx_add"] is None else dx + s["dx_add"].double()
    if op == "route_grad":
        l = s["logits"].double().requires_grad_()
        return torch.autograd.grad(_x_gate(s, l), l, s["dw"].double())[0]

    def each(rows, width, f):
        out = torch.zeros((rows, width), dtype=torch.float64, device="cuda")
        for e, a, b in _segments(s):
            out[a:b] = f(e, a, b)
        return out

    P = s["sorted_ids"].numel()
    if op == "gate_up_train":
        h = each(P, 2 * I, lambda e, a, b: torch.einsum("ph,jh->pj", s["x_perm"][a:b].double(), s["w13"][e].double()))
        return {"h13": h, "act": torch.nn.functional.silu(h[:, :I]) * h[:, I:]}
    if op == "down_grad":
        def f(e, a, b):
            h = s["h13"][a:b].double().requires_grad_()
            act = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            da = torch.einsum("ph,hi->pi", s["dy_perm"][a:b].double(), s["w2"][e].double())
            return torch.autograd.grad(act, h, da)[0]
        return each(P, 2 * I, f)
    if op == "gate_up_grad":
        return each(P, H, lambda e, a, b: torch.einsum("pj,jh->ph", s["dh13"][a:b].double(), s["w13"][e].double()))
    d, x = (s["dy_perm"], s["act"]) if op == "down_wgrad" else (s["dh13"], s["x_perm"])
    out = torch.zeros((s["E"], d.shape[1], x.shape[1]), dtype=torch.float64, device="cuda")
    for e, a, b in _segments(s):
        out[e] = torch.einsum("pm,pn->mn", d[a:b].double(), x[a:b].double())
    return out


# ---------------------------------------------------------------------- floors

def work(case):
    """Each input read once, each output written once.  A: assigned rows (half
    the slots with per-token counts); padding rows are not counted."""
    c = case
    T, H, E, K, I, op = c["T"], c["H"], c["E"], c["K"], c["I"], c["op"]
    b = 2 if c["dtype"] == "bf16" else 4
    A = T * K * (0.5 if c["dyn"] else 1.0)
    Ea = min(E, A)  # experts with a token, at most
    norm_par = H * b * (bool(c["post"]) + bool(c["nxt"])) + (0, H * b, T * H * b)[c["gate"]]
    if op in ("combine_norm", "block_norm"):
        nb = T * H * b * (2 + bool(c["nxt"])) + norm_par  # residual, h, n
        if op == "combine_norm":
            nb += A * H * b + T * H * b * (1 + bool(c["shared"])) + 8 * T * K
            return {"bytes": nb, "flops": 2 * A * H + 10 * T * H}
        return {"bytes": nb + T * H * b, "flops": 10 * T * H}
    if op == "block_norm_grad":
        nb = T * H * b * (2 + 2 * bool(c["nxt"]) + 2) + norm_par  # y, dh, h, dn, dy, dresidual
        nb += 4 * H * (bool(c["post"]) + bool(c["nxt"])) + (0, 4 * H, T * H * b)[c["gate"]]
        return {"bytes": nb, "flops": 25 * T * H}
    if op == "combine_grad":
        return {"bytes": T * H * b + 2 * A * H * b + 16 * T * K, "flops": 3 * A * H}
    if op == "permute_grad":
        return {"bytes": A * H * b + T * H * b * (1 + bool(c["add"])) + 4 * T * K, "flops": A * H}
    if op == "route_grad":
        full = c["score"] == 0 and not c["renorm"]
        return {"bytes": 4 * T * E + 8 * T * K + 4 * (T * E if full else A), "flops": 8 * T * K}
    if op == "gate_up_train":
        return {"bytes": A * H * b + Ea * 2 * I * H * b + 3 * A * I * b, "flops": 4 * A * H * I}
    if op == "down_grad":
        return {"bytes": A * H * b + Ea * H * I * b + 4 * A * I * b, "flops": 2 * A * H * I}
    if op == "gate_up_grad":
        return {"bytes": 2 * A * I * b + Ea * 2 * I * H * b + A * H * b, "flops": 4 * A * H * I}
    if op == "down_wgrad":
        return {"bytes": A * (H + I) * b + E * H * I * b, "flops": 2 * A * H * I}
    return {"bytes": A * (H + 2 * I) * b + E * 2 * H * I * b, "flops": 4 * A * H * I}

"""The routed-expert sub-layer's operators: what is measured, in plain form and by the library.

Four operators, each with its cases:
  norm      sparsesam_norm_residual and its backward: the norms after one block and before the
            next, fused with the block's gate, residual scale and residual add
  route     sparsesam_expert_route, sparsesam_expert_sort and the router's gradient: a token's
            top-k experts and weights, and the tokens' stable order by expert
  dispatch  sparsesam_expert_gather, sparsesam_expert_combine and their gradients: rows to the
            sorted order and back, weights applied
  mlp       sparsesam_expert_mlp: the experts' fc1-GELU-fc2 products over the sorted rows
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # One token of the serving path (a single query's residual stream): latency.
        dict(name="norm_token", op="norm", rows=1, C=1280, dtype="bf16", norm="rms", per_gate=1,
             post=True, gate=False, scale=True, pre=True, grad=False),
        # The ViT-H batch (4 images of 64 x 64 tokens) with everything on: bandwidth.
        dict(name="norm_vith", op="norm", rows=16384, C=1280, dtype="bf16", norm="layer",
             per_gate=4096, post=True, gate=True, scale=True, pre=True, grad=False),
        # The gradients over the ViT-L batch (8 images): the largest.
        dict(name="norm_vitl_grad", op="norm", rows=32768, C=1024, dtype="bf16", norm="layer",
             per_gate=4096, post=True, gate=True, scale=True, pre=True, grad=True),
        # Gradients of class token + 24 x 24 patches, 7 images, an odd width, fp32.
        dict(name="norm_odd_grad", op="norm", rows=4039, C=1160, dtype="f32", norm="rms",
             per_gate=577, post=True, gate=True, scale=False, pre=True, grad=True),
        # One 14 x 14 window's tokens: latency of the router and the sort.
        dict(name="route_window", op="route", tokens=196, experts=8, topk=2, renorm=True,
             dropped=0.0, skew=0.5, grad=False),
        # Eight images in windows padded to 70 x 70 (16% pads, routed nowhere), with the gradient.
        dict(name="route_images_grad", op="route", tokens=39200, experts=64, topk=4, renorm=False,
             dropped=0.16, skew=1.0, grad=True),
        # The ViT-H batch to 8 experts and back.
        dict(name="dispatch_vith", op="dispatch", tokens=16384, experts=8, topk=2, C=1280,
             dtype="bf16", dropped=0.0, skew=0.5, grad=False),
        # The gradients of the way there and back over the ViT-L batch.
        dict(name="dispatch_vitl_grad", op="dispatch", tokens=32768, experts=32, topk=2, C=1024,
             dtype="bf16", dropped=0.05, skew=1.0, grad=True),
        # A ragged small one in fp32: 3 x 577 tokens, three experts a token.
        dict(name="dispatch_odd_grad", op="dispatch", tokens=1731, experts=12, topk=3, C=200,
             dtype="f32", dropped=0.1, skew=1.0, grad=True),
        # One token at ViT-H widths: two experts' weights are read, nothing else matters.
        dict(name="mlp_token", op="mlp", tokens=1, experts=8, topk=2, C=1280, hidden=5120,
             dropped=0.0, skew=0.0),
        # Four windows' tokens over 16 experts at ViT-L widths: ragged, about 100 rows an expert.
        dict(name="mlp_windows", op="mlp", tokens=784, experts=16, topk=2, C=1024, hidden=4096,
             dropped=0.02, skew=0.7),
        # The ViT-H batch over 8 experts: the tensor cores.
        dict(name="mlp_vith", op="mlp", tokens=16384, experts=8, topk=2, C=1280, hidden=5120,
             dropped=0.0, skew=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(("norm", "route", "dispatch", "mlp"))
    if op == "norm":
        C, dtype = _width(rng, 64, 4096), rng.choice(("bf16", "bf16", "f16", "f32"))
        rows = _log(rng, 1, max(2, min(65536, 2 ** 26 // (C * SIZES[dtype]))))
        post, pre = rng.choice(((True, True), (True, False), (False, True)))
        return dict(op=op, rows=rows, C=C, dtype=dtype, norm=rng.choice(("layer", "rms")),
                    per_gate=_log(rng, 1, rows), post=post, gate=rng.random() < 0.5,
                    scale=rng.random() < 0.5, pre=pre, grad=rng.random() < 0.5)
    experts = _log(rng, 2, 64 if op == "mlp" else 256)
    topk = rng.randint(1, min(experts, 4))
    case = dict(op=op, experts=experts, topk=topk, dropped=rng.choice((0.0, 0.05, 0.2)),
                skew=rng.choice((0.0, 0.5, 1.0)))
    if op == "route":
        case.update(tokens=_log(rng, 1, 39200 * 64 // max(64, experts)),
                    renorm=rng.random() < 0.5, grad=rng.random() < 0.5)
    elif op == "dispatch":
        C, dtype = _width(rng, 64, 4096), rng.choice(("bf16", "bf16", "f16", "f32"))
        case.update(tokens=_log(rng, 1, max(2, min(32768, 2 ** 27 // (C * topk * SIZES[dtype])))),
                    C=C, dtype=dtype, grad=rng.random() < 0.5)
    else:
        C, hidden = _width(rng, 64, 1280), _width(rng, 64, 5120)
        case["experts"] = min(experts, max(topk, 2 ** 27 // (C * hidden)))
        case.update(tokens=_log(rng, 1, 16384 * 2 // topk), C=C, hidden=hidden)
    return case


# ---- inputs ---------------------------------------------------------------------------------

def _logits(case, g):
    """Router logits: normal, some experts more popular; dropped tokens have nothing but -inf, and
    one in fifty of the others' entries is -inf too (an expert closed to that token)."""
    T, E = case["tokens"], case["experts"]
    lg = torch.randn(T, E, generator=g, device="cuda")
    lg += case["skew"] * torch.randn(E, generator=g, device="cuda")
    closed = torch.rand(T, E, generator=g, device="cuda") < 0.02
    closed |= torch.rand(T, 1, generator=g, device="cuda") < case["dropped"]
    closed[0] = False
    return lg.masked_fill_(closed, -math.inf)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "norm":
        dt, R, C = DTYPES[case["dtype"]], case["rows"], case["C"]
        groups = -(-R // case["per_gate"])
        # A residual stream: some channels far larger than others, means off zero.
        wide = torch.exp(0.7 * f(C))
        s.update(y=(0.5 * f(R, C) + 0.2 * f(C)).to(dt), x=(f(R, C) * wide + 0.3 * f(C)).to(dt))
        s["gate"] = f(groups, C).to(dt) if case["gate"] else None
        s["scale"] = (0.5 + 0.2 * f(C)).to(dt) if case["scale"] else None
        bias = case["norm"] == "layer"
        for k in ("post", "pre"):
            s[k + "_w"] = (1 + 0.1 * f(C)).to(dt) if case[k] else None
            s[k + "_b"] = (0.1 * f(C)).to(dt) if case[k] and bias else None
        s["eps"] = 1e-6
        if case["grad"]:
            s.update(dx_out=f(R, C).to(dt), dn=f(R, C).to(dt) if case["pre"] else None)
            # What the forward left: x is now its stored result, with the norms' statistics.
            st = torch.zeros(R, 4, dtype=torch.float64, device="cuda")
            for i, k, v in ((0, "post", s["y"]), (2, "pre", s["x"])):
                if case[k]:
                    v = v.double()
                    if bias:
                        st[:, i] = v.mean(1)
                    st[:, i + 1] = (v - st[:, i:i + 1]).square().mean(1).add(s["eps"]).rsqrt()
            s["stats"] = st.float()
    else:
        s["logits"] = _logits(case, g)
        T, E, k = case["tokens"], case["experts"], case["topk"]
        if case["op"] == "route":
            s["dweight"] = f(T, k)
        else:
            s["ids"], s["weight"] = _route(s["logits"], k, True)
            del s["logits"]
        if case["op"] == "dispatch":
            dt, C = DTYPES[case["dtype"]], case["C"]
            _, s["slot"], s["offsets"] = _sort(s["ids"], E)
            s.update(ys=f(T * k, C).to(dt))
            if case["grad"]:
                s.update(dout=f(T, C).to(dt), dxs=f(T * k, C).to(dt))
            else:
                s.update(x=f(T, C).to(dt), residual=f(T, C).to(dt))
        elif case["op"] == "mlp":
            C, H = case["C"], case["hidden"]
            b = torch.bfloat16
            s.update(x=f(T, C).to(b), residual=f(T, C).to(b),
                     w1=(f(E, H, C) / math.sqrt(C)).to(b), b1=(0.1 * f(E, H)).to(b),
                     w2=(f(E, C, H) / math.sqrt(H)).to(b), b2=(0.1 * f(E, C)).to(b))
    if own:
        _buffers(s)
    return s


# ---- the plain form -------------------------------------------------------------------------

def _route(logits, k, renorm):
    value, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    open_ = value > -math.inf
    top = torch.where(open_[:, :1], value[:, :1], 0.0)
    e = torch.exp(value - top)
    total = (e if renorm else torch.exp(logits - top)).sum(-1, keepdim=True)
    weight = torch.where(open_, e / total, 0.0)
    return torch.where(open_, ids, -1).int(), weight


def _sort(ids, E):
    flat = ids.reshape(-1)
    n = flat.numel()
    key = torch.where(flat < 0, E, flat).long()
    order = torch.sort(key, stable=True)[1]
    count = torch.zeros(E + 1, dtype=torch.long, device=flat.device)
    count.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.long, device=flat.device)
    offsets[1:] = torch.cumsum(count[:E], 0)
    place = torch.arange(n, device=flat.device)
    slot = torch.empty_like(order)
    slot[order] = place
    slot = torch.where(flat < 0, -1, slot)
    order = torch.where(place < offsets[E], order, -1)
    return order.int(), slot.int().view_as(ids), offsets.int()


def _plain_norm(v, w, b, eps, center):
    mean = v.mean(1, keepdim=True) if center else 0.0
    rstd = 1.0 / torch.sqrt((v - mean).square().mean(1, keepdim=True) + eps)
    h = (v - mean) * rstd * w
    return h if b is None else h + b


def _f(t):
    return None if t is None else t.float()


def _gate_rows(s):
    if s["gate"] is None:
        return None
    at = torch.arange(s["rows"], device="cuda") // s["per_gate"]
    return s["gate"].float()[at]


def _plain_norm_forward(s):
    dt, center = s["x"].dtype, s["norm"] == "layer"
    p = s["y"].float()
    if s["post"]:
        p = _plain_norm(p, _f(s["post_w"]), _f(s["post_b"]), s["eps"], center)
    gate = _gate_rows(s)
    if gate is not None:
        p = p * gate
    if s["scale"] is not None:
        p = p * s["scale"].float()
    x = (s["x"].float() + p).to(dt)
    out = {"x": x}
    if s["pre"]:
        out["n"] = _plain_norm(x.float(), _f(s["pre_w"]), _f(s["pre_b"]), s["eps"], center).to(dt)
    return out


def _plain_norm_rows(d, h, w, rstd, center):
    """The gradient through h * w, h = (v - mean) * rstd, for the gradient d of the norm."""
    g = d * w
    g_h = (g * h).mean(1, keepdim=True)
    g = g - g.mean(1, keepdim=True) if center else g
    return rstd * (g - h * g_h)


def _plain_norm_backward(s):
    dt, center = s["x"].dtype, s["norm"] == "layer"
    st = s["stats"]
    out = {}
    D = s["dx_out"].float()
    if s["pre"]:
        h = (s["x"].float() - st[:, 2:3]) * st[:, 3:4]
        dn = s["dn"].float()
        out["pre_w"] = (dn * h).sum(0)
        if center:
            out["pre_b"] = dn.sum(0)
        D = D + _plain_norm_rows(dn, h, _f(s["pre_w"]), st[:, 3:4], center)
    out["dx"] = D.to(dt)
    h = p = s["y"].float()
    if s["post"]:
        h = (h - st[:, 0:1]) * st[:, 1:2]
        p = h * s["post_w"].float()
        p = p if s["post_b"] is None else p + s["post_b"].float()
    gate, scale = _gate_rows(s), _f(s["scale"])
    if gate is not None:
        groups = s["gate"].shape[0]
        at = torch.arange(s["rows"], device="cuda") // s["per_gate"]
        each = D * p if scale is None else D * p * scale
        out["gate"] = torch.zeros(groups, s["C"], device="cuda").index_add_(0, at, each)
        D = D * gate
    if scale is not None:
        out["scale"] = (D * p).sum(0)
        D = D * scale
    if s["post"]:
        out["post_w"] = (D * h).sum(0)
        if center:
            out["post_b"] = D.sum(0)
        D = _plain_norm_rows(D, h, _f(s["post_w"]), st[:, 1:2], center)
    out["dy"] = D.to(dt)
    return out


def _plain_route(s):
    ids, weight = _route(s["logits"], s["topk"], s["renorm"])
    order, slot, offsets = _sort(ids, s["experts"])
    out = {"ids": ids, "weight": weight, "order": order, "slot": slot, "offsets": offsets}
    if s["grad"]:
        dw = torch.where(ids >= 0, s["dweight"], 0.0)
        mean = (dw * weight).sum(1, keepdim=True)
        at = ids.clamp(min=0).long()
        if s["renorm"]:
            d = torch.zeros_like(s["logits"])
        else:
            top = s["logits"].amax(1, keepdim=True)
            top = torch.where(top > -math.inf, top, 0.0)
            e = torch.exp(s["logits"] - top)
            total = e.sum(1, keepdim=True)
            d = -mean * torch.where(total > 0, e / total, 0.0)
        each = weight * (dw - mean) if s["renorm"] else weight * dw
        out["dlogits"] = d.scatter_add_(1, at, each)
    return out


def _plain_combine(rows, slot, weight):
    each = rows.float()[slot.clamp(min=0).long()]
    w = (slot >= 0).float() if weight is None else torch.where(slot >= 0, weight, 0.0)
    return (each * w[..., None]).sum(1)


def _plain_gather(x, slot, n):
    """The rows of x at their sorted places; places without a row are zero here."""
    k = slot.shape[1]
    flat = slot.reshape(-1).long()
    at = torch.where(flat < 0, n, flat)
    out = torch.zeros(n + 1, x.shape[1], dtype=x.dtype, device=x.device)
    out[at] = x.repeat_interleave(k, 0)
    return out[:n]


def _plain_dispatch(s):
    n, slot = s["slot"].numel(), s["slot"]
    if not s["grad"]:
        out = s["residual"].float() + _plain_combine(s["ys"], slot, s["weight"])
        return {"xs": _plain_gather(s["x"], slot, n), "out": out.to(s["x"].dtype)}
    dt = s["ys"].dtype
    dout = s["dout"].float()
    each = (s["weight"][..., None] * dout[:, None, :]).to(dt)
    at = torch.where(slot < 0, n, slot).reshape(-1).long()
    dys = torch.zeros(n + 1, s["C"], dtype=dt, device=dout.device)
    dys[at] = each.reshape(n, -1)
    rows = s["ys"].float()[slot.clamp(min=0).long()]
    dweight = torch.where(slot >= 0, (rows * dout[:, None, :]).sum(-1), 0.0)
    return {"dys": dys[:n], "dweight": dweight, "dx": _plain_combine(s["dxs"], slot, None).to(dt)}


def _gelu(z):
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _plain_mlp(s):
    T, k, E = s["tokens"], s["topk"], s["experts"]
    flat = s["ids"].reshape(-1).long()
    n = T * k
    x = s["x"].float().repeat_interleave(k, 0)
    w1, b1, w2, b2 = s["w1"], s["b1"], s["w2"], s["b2"]
    if n <= E:  # fewer rows than experts: each row with its own expert's weights
        e = flat.clamp(min=0)
        h = _gelu(torch.bmm(w1[e].float(), x[:, :, None])[..., 0] + b1[e].float())
        y = torch.bmm(w2[e].float(), h[:, :, None])[..., 0] + b2[e].float()
    else:  # the experts' rows side by side, each as long as the longest
        order, slot, offsets = _sort(s["ids"], E)
        cap = int((offsets[1:] - offsets[:-1]).max())
        place = slot.reshape(-1).long() - offsets.long()[flat.clamp(min=0)]
        place = torch.where(flat < 0, E * cap, flat * cap + place)
        packed = torch.zeros(E * cap + 1, s["C"], device=x.device)
        packed[place] = x
        h = _gelu(torch.baddbmm(b1.float()[:, None], packed[:-1].view(E, cap, -1),
                                w1.float().transpose(1, 2)))
        y = torch.baddbmm(b2.float()[:, None], h, w2.float().transpose(1, 2))
        y = y.reshape(E * cap, -1)[place.clamp(max=E * cap - 1)]
    w = torch.where(s["ids"] >= 0, s["weight"], 0.0)
    out = s["residual"].float() + (y.view(T, k, -1) * w[..., None]).sum(1)
    return {"out": out.to(torch.bfloat16)}


# ---- the library's calls --------------------------------------------------------------------

def _buffers(s):
    """What a program that uses the library keeps: the plan, outputs and workspace."""
    import structured_activation_sparsity_b200 as ss
    new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    zero = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    if s["op"] == "norm":
        dt, R, C = DTYPES[s["dtype"]], s["rows"], s["C"]
        s["cfg"] = ss.make_norm_cfg(R, C, dtype=s["dtype"], norm=s["norm"], eps=s["eps"],
                                    rows_per_gate=s["per_gate"] if s["gate"] is not None else 0)
        if s["grad"]:
            like = lambda t: None if t is None else new(*t.shape, dtype=f32)  # noqa: E731
            s.update(dx=new(R, C, dtype=dt), dy=new(R, C, dtype=dt))
            s["dparams"] = {k: like(s[k]) for k in ("gate", "scale", "post_w", "post_b", "pre_w",
                                                    "pre_b")}
            s["ws_bytes"] = ss.sparsesam_norm_residual_backward_workspace(s["cfg"])
        else:
            s.update(x_out=new(R, C, dtype=dt), n=new(R, C, dtype=dt) if s["pre"] else None)
            s["ws_bytes"] = 0
    else:
        T, k, E = s["tokens"], s["topk"], s["experts"]
        s["cfg"] = ss.make_expert_cfg(T, E, k, C=s.get("C", 8), hidden=s.get("hidden", 8),
                                      dtype=s.get("dtype", "bf16"))
        s["ws_bytes"] = 0
        if s["op"] == "route":
            s.update(ids=new(T, k, dtype=i32), weight=new(T, k, dtype=f32),
                     order=new(T * k, dtype=i32), slot=new(T, k, dtype=i32),
                     offsets=new(E + 1, dtype=i32), dlogits=new(T, E, dtype=f32))
            s["ws_bytes"] = ss.sparsesam_expert_sort_workspace(s["cfg"])
        elif s["op"] == "dispatch":
            dt, C = DTYPES[s["dtype"]], s["C"]
            if s["grad"]:
                s.update(dys=zero(T * k, C, dtype=dt), dx=new(T, C, dtype=dt),
                         dweight=new(T, k, dtype=f32))
            else:
                s.update(xs=zero(T * k, C, dtype=dt), out=new(T, C, dtype=dt))
        else:
            s["out"] = new(T, s["C"], dtype=torch.bfloat16)
            s["ws_bytes"] = ss.sparsesam_expert_mlp_workspace(s["cfg"])
    s["ws"] = new(max(s["ws_bytes"], 1), dtype=torch.uint8)


def _own_run(s):
    import structured_activation_sparsity_b200 as ss
    st = torch.cuda.current_stream()
    cfg = s["cfg"]
    if s["op"] == "norm" and not s["grad"]:
        ss.sparsesam_norm_residual(cfg, s["y"], s["x"], s["gate"], s["scale"], s["post_w"],
                                   s["post_b"], s["pre_w"], s["pre_b"], s["x_out"], s["n"], None,
                                   stream=st)
        out = {"x": s["x_out"]}
        if s["pre"]:
            out["n"] = s["n"]
        return out
    if s["op"] == "norm":
        d = s["dparams"]
        ss.sparsesam_norm_residual_backward(
            cfg, s["y"], s["x"], s["gate"], s["scale"], s["post_w"], s["post_b"], s["pre_w"],
            s["stats"], s["dx_out"], s["dn"], s["dx"], s["dy"], d["gate"], d["scale"],
            d["post_w"], d["post_b"], d["pre_w"], d["pre_b"], s["ws"], s["ws_bytes"], stream=st)
        out = {k: v for k, v in d.items() if v is not None}
        out.update(dx=s["dx"], dy=s["dy"])
        return out
    if s["op"] == "route":
        ss.sparsesam_expert_route(cfg, s["logits"], s["renorm"], s["ids"], s["weight"], stream=st)
        ss.sparsesam_expert_sort(cfg, s["ids"], s["order"], s["slot"], s["offsets"], s["ws"],
                                 s["ws_bytes"], stream=st)
        out = {k: s[k] for k in ("ids", "weight", "order", "slot", "offsets")}
        if s["grad"]:
            ss.sparsesam_expert_route_backward(cfg, s["logits"], s["renorm"], s["ids"],
                                               s["weight"], s["dweight"], s["dlogits"], stream=st)
            out["dlogits"] = s["dlogits"]
        return out
    if s["op"] == "dispatch" and not s["grad"]:
        ss.sparsesam_expert_gather(cfg, s["x"], s["slot"], s["xs"], stream=st)
        ss.sparsesam_expert_combine(cfg, s["ys"], s["slot"], s["weight"], s["residual"], s["out"],
                                    stream=st)
        return {"xs": s["xs"], "out": s["out"]}
    if s["op"] == "dispatch":
        ss.sparsesam_expert_combine_backward(cfg, s["dout"], s["ys"], s["slot"], s["weight"],
                                             s["dys"], s["dweight"], stream=st)
        ss.sparsesam_expert_combine(cfg, s["dxs"], s["slot"], None, None, s["dx"], stream=st)
        return {"dys": s["dys"], "dweight": s["dweight"], "dx": s["dx"]}
    ss.sparsesam_expert_mlp(cfg, s["x"], s["ids"], s["weight"], s["residual"], s["w1"], s["b1"],
                            s["w2"], s["b2"], s["out"], s["ws"], s["ws_bytes"], stream=st)
    return {"out": s["out"]}


def run(s):
    if own:
        return _own_run(s)
    if s["op"] == "norm":
        return _plain_norm_backward(s) if s["grad"] else _plain_norm_forward(s)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "mlp": _plain_mlp}[s["op"]](s)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        R, C, es = case["rows"], case["C"], SIZES[case["dtype"]]
        groups = -(-R // case["per_gate"]) if case["gate"] else 0
        params = (groups + case["scale"] + (2 if case["norm"] == "layer" else 1) *
                  (case["post"] + case["pre"])) * C
        if not case["grad"]:
            return {"bytes": R * C * es * (3 + case["pre"]) + params * es, "flops": 12 * R * C}
        return {"bytes": R * C * es * (4 + 2 * case["pre"]) + R * 16 + params * (es + 4),
                "flops": 30 * R * C}
    T, E, k = case["tokens"], case["experts"], case["topk"]
    n = T * k
    live = round(n * (1 - case["dropped"]))
    if case["op"] == "route":
        b = T * E * 4 + n * 16 + E * 4
        if case["grad"]:
            b += T * E * 4 + n * 4
        return {"bytes": b, "flops": 4 * T * E}
    C = case["C"]
    if case["op"] == "dispatch":
        es = SIZES[case["dtype"]]
        if not case["grad"]:
            return {"bytes": (3 * T + 2 * live) * C * es + n * 8, "flops": 2 * n * C}
        return {"bytes": (2 * T + 3 * live) * C * es + n * 12, "flops": 4 * n * C}
    used = min(E, live) if live else 0
    return {"bytes": used * (2 * C * case["hidden"] + C + case["hidden"]) * 2 + T * C * 6 + n * 8,
            "flops": 4 * live * C * case["hidden"]}


# ---- in 64 bits, from the definitions -------------------------------------------------------

def _exact_norm(case, s):
    eps, center = s["eps"], case["norm"] == "layer"
    dd = lambda t: None if t is None else t.double()  # noqa: E731

    def norm(v, w, b):
        v = v - v.mean(1, keepdim=True) if center else v
        v = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * w
        return v if b is None else v + b

    P = {k: dd(s[k]) for k in ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b")}
    leaves = {k: v.requires_grad_() for k, v in P.items() if v is not None} if case["grad"] else {}
    y = dd(s["y"])
    if case["grad"]:
        y.requires_grad_()
    p = norm(y, P["post_w"], P["post_b"]) if case["post"] else y
    if P["gate"] is not None:
        p = p * P["gate"].repeat_interleave(case["per_gate"], 0)[:case["rows"]]
    if P["scale"] is not None:
        p = p * P["scale"]
    if not case["grad"]:
        x = (dd(s["x"]) + p)
        out = {"x": x}
        if case["pre"]:
            out["n"] = norm(x.to(s["x"].dtype).double(), P["pre_w"], P["pre_b"])
        return out
    # The forward's result x is given: the branch into the pre norm starts at it.
    x = dd(s["x"]).requires_grad_()
    total = (x * dd(s["dx_out"])).sum()
    if case["pre"]:
        total = total + (norm(x, P["pre_w"], P["pre_b"]) * dd(s["dn"])).sum()
    pre = [k for k in leaves if k.startswith("pre")]
    got = torch.autograd.grad(total, [x] + [leaves[k] for k in pre])
    out = {"dx": got[0], **dict(zip(pre, got[1:]))}
    rest = [k for k in leaves if not k.startswith("pre")]
    got = torch.autograd.grad((p * got[0].detach()).sum(), [y] + [leaves[k] for k in rest])
    out.update({"dy": got[0], **dict(zip(rest, got[1:]))})
    return out


def _exact_route(case, s):
    k = case["topk"]
    lg = s["logits"].double().requires_grad_(case["grad"])
    with torch.no_grad():
        ids, _ = _route(s["logits"], k, True)
    live = ids >= 0
    chosen = torch.gather(lg, 1, ids.clamp(min=0).long()).masked_fill(~live, -math.inf)
    base = chosen if case["renorm"] else lg
    total = torch.logsumexp(base.masked_fill(~live.any(1, keepdim=True), 0.0), 1, keepdim=True)
    weight = torch.exp(chosen.masked_fill(~live, 0.0) - total) * live
    out = {"ids": None, "weight": weight.detach(), "order": None, "slot": None, "offsets": None}
    if case["grad"]:
        d = torch.autograd.grad((weight * s["dweight"].double()).sum(), lg)[0]
        out["dlogits"] = torch.nan_to_num(d, nan=0.0)
    return out


def _exact_dispatch(case, s):
    T, k = s["slot"].shape
    n = T * k
    slot = s["slot"].reshape(-1).long()
    live = slot >= 0
    token = torch.arange(n, device="cuda") // k
    src, dst = token[live], slot[live]
    w = s["weight"].double().reshape(-1)[live][:, None]
    ys = s["ys"].double()
    if not case["grad"]:
        xs = torch.zeros(n, case["C"], dtype=torch.float64, device="cuda")
        xs[dst] = s["x"].double()[src]
        return {"xs": xs, "out": s["residual"].double().index_add(0, src, w * ys[dst])}
    dout = s["dout"].double()
    dys = torch.zeros(n, case["C"], dtype=torch.float64, device="cuda")
    dys[dst] = w * dout[src]
    dweight = torch.zeros(n, dtype=torch.float64, device="cuda")
    dweight[live] = (ys[dst] * dout[src]).sum(1)
    dx = torch.zeros(T, case["C"], dtype=torch.float64, device="cuda")
    dx.index_add_(0, src, s["dxs"].double()[dst])
    return {"dys": dys, "dweight": dweight.view(T, k), "dx": dx}


def _exact_mlp(case, s):
    out = s["residual"].double()
    ids = s["ids"].long()
    for e in range(case["experts"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        z = s["x"].double()[t] @ s["w1"][e].double().T + s["b1"][e].double()
        h = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        y = h @ s["w2"][e].double().T + s["b2"][e].double()
        out.index_add_(0, t, s["weight"].double()[t, j][:, None] * y)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    fn = {"norm": _exact_norm, "route": _exact_route, "dispatch": _exact_dispatch,
          "mlp": _exact_mlp}[case["op"]]
    return fn(case, s)

"""sparsesam_norm_residual and its backward on the GPU against the float64 oracle.

Tolerances, derived from the arithmetic (u = half a step of the rows' type, relative: bf16 2^-8, fp16
2^-11, fp32 2^-24). A row's sums are fp32 in a tree of at most 40 sequential terms a lane and
eight more joins: 48 * 2^-24 of the sum of magnitudes, taken as S = 2^-18. A normalised value
h = (v - mean) rstd is then off by at most E_h = S (2 |h| + rstd mean|v|) + 2^-22 |h|. Every output is
rounded once: u |out|. fp16 below its normal range rounds by half of 2^-24."""
import numpy as np
import pytest
import torch

from oracle import expert_oracle as X
from structured_activation_sparsity_b200 import _lib as L

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
S = 2.0 ** -18
EPS = 1e-6


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(rows, C, dtype, kind, per_gate, post, gate, scale, pre, seed=0, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = lambda v: v.to(TORCH[dtype]).cuda()  # noqa: E731
    groups = -(-rows // per_gate) if rows else 0
    b = kind == "layer"
    return dict(y=t(r(rows, C) + mean), x=t(2 * r(rows, C) + mean),
                gate=t(r(groups, C)) if gate else None, scale=t(0.5 + r(C)) if scale else None,
                post_w=t(1 + 0.2 * r(C)) if post else None,
                post_b=t(0.2 * r(C)) if post and b else None,
                pre_w=t(1 + 0.2 * r(C)) if pre else None,
                pre_b=t(0.2 * r(C)) if pre and b else None)


def _cfg(rows, C, dtype, kind, per_gate, gate, **kw):
    return L.make_norm_cfg(rows, C, dtype=dtype, norm=kind, eps=EPS,
                           rows_per_gate=per_gate if gate else 0, **kw)


def _forward(cfg, v, pre, x_out=None, n=None, stats=None, stream=None):
    rows, C = v["x"].shape
    x_out = torch.full_like(v["x"], 7.0) if x_out is None else x_out
    n = (torch.full_like(v["x"], 7.0) if n is None else n) if pre else None
    stats = torch.full((rows, 4), 7.0, device="cuda") if stats is None else stats
    L.sparsesam_norm_residual(cfg, v["y"], v["x"], v["gate"], v["scale"], v["post_w"],
                              v["post_b"], v["pre_w"], v["pre_b"], x_out, n, stats, stream=stream)
    return x_out, n, stats


def _h_off(v, kind):
    """(h, E_h) of the rows v."""
    mean, rstd = X.norm_stats(v, kind, EPS)
    h = (v - mean) * rstd
    return h, S * (2 * np.abs(h) + rstd * np.abs(v).mean(1, keepdims=True)) + 2.0 ** -22 * np.abs(h)


def _check_forward(v, per_gate, kind, dtype, x_out, n, stats):
    o = {k: f64(t) for k, t in v.items()}
    want = X.norm_residual(o["y"], o["x"], o["gate"], per_gate, o["scale"], o["post_w"],
                           o["post_b"], kind, EPS)
    k = np.abs(X.gate_rows(o["gate"], len(o["y"]), per_gate) * (1 if o["scale"] is None else o["scale"]))
    p, off = o["y"], 0.0
    if o["post_w"] is not None:
        h, eh = _h_off(o["y"], kind)
        b = 0.0 if o["post_b"] is None else o["post_b"]
        p, off = h * o["post_w"] + b, np.abs(o["post_w"]) * eh + 2.0 ** -22 * (np.abs(h * o["post_w"]) + np.abs(b))
    tol = U[dtype] * np.abs(want) + k * off + 2.0 ** -22 * (k * np.abs(p) + np.abs(o["x"])) + TINY[dtype]
    got = f64(x_out)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    st = f64(stats)
    for i, w, r in ((0, "post_w", o["y"]), (2, "pre_w", got)):
        if o[w] is None:
            assert (st[:, i:i + 2] == 0).all()
            continue
        mean, rstd = X.norm_stats(r, kind, EPS)
        assert (np.abs(st[:, i:i + 1] - mean) <= S * np.abs(r).mean(1, keepdims=True)).all()
        assert (np.abs(st[:, i + 1:i + 2] - rstd) <= 2 * S * rstd).all()
    if n is not None:
        want = X.norm(got, o["pre_w"], o["pre_b"], kind, EPS)
        h, eh = _h_off(got, kind)
        b = 0.0 if o["pre_b"] is None else np.abs(o["pre_b"])
        tol = (U[dtype] * np.abs(want) + np.abs(o["pre_w"]) * eh
               + 2.0 ** -22 * (np.abs(h * o["pre_w"]) + b) + TINY[dtype])
        assert (np.abs(f64(n) - want) <= tol).all(), float((np.abs(f64(n) - want) / tol).max())


CASES = [
    # rows, C, dtype, kind, per_gate, post, gate, scale, pre
    (1, 1280, "bf16", "rms", 1, True, False, True, True),
    (1, 8, "bf16", "layer", 1, True, True, True, True),
    (37, 72, "f32", "layer", 5, True, True, True, True),
    (300, 256, "bf16", "layer", 100, True, True, True, True),
    (577, 264, "f16", "rms", 577, False, True, False, True),
    (64, 768, "bf16", "layer", 16, True, False, False, False),
    (130, 1160, "f32", "rms", 1, True, True, True, True),
    (1200, 1024, "bf16", "layer", 400, True, True, True, True),
    (41, 2056, "f16", "layer", 7, True, True, True, True),
    (23, 4096, "f32", "layer", 8, True, True, True, True),
    (50, 4096, "bf16", "rms", 50, False, False, True, True),
    (19, 1288, "bf16", "layer", 4, False, False, False, False),
    (4000, 64, "bf16", "layer", 3, True, True, False, True),
    (9001, 40, "f16", "rms", 9001, True, True, True, True),
    # one warp a row, more, ragged: the spans of the many-row kernel
    (3500, 1280, "bf16", "layer", 100, True, True, True, True),
    (1300, 2048, "bf16", "rms", 650, True, True, False, True),
    (1100, 1800, "f16", "layer", 100, True, False, True, True),
    (700, 4096, "bf16", "layer", 350, True, True, True, True),
    (900, 1160, "f32", "layer", 300, True, True, True, True),
    (400, 3880, "f32", "rms", 400, True, True, True, True),
    (300, 4096, "f32", "layer", 7, True, True, True, True),
    (1400, 1536, "f16", "layer", 200, False, True, True, True),
    (2500, 512, "f32", "layer", 500, True, True, False, False),
]
IDS = ["-".join(map(str, c[:5])) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    rows, C, dtype, kind, per_gate, post, gate, scale, pre = case
    v = _inputs(*case)
    x_out, n, stats = _forward(_cfg(rows, C, dtype, kind, per_gate, gate), v, pre)
    torch.cuda.synchronize()
    _check_forward(v, per_gate, kind, dtype, x_out, n, stats)


def _backward(cfg, v, x_out, stats, dx_out, dn, dx=None, dy=None, stream=None, skip=(), grads=None, ws=None):
    like = lambda k: None if v[k] is None or k in skip else torch.full(v[k].shape, 7.0, device="cuda")  # noqa: E731
    g = grads or {"d" + k: like(k) for k in ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b")}
    dx = torch.full_like(x_out, 7.0) if dx is None else dx
    dy = torch.full_like(v["y"], 7.0) if dy is None else dy
    nb = L.sparsesam_norm_residual_backward_workspace(cfg)
    if ws is None:
        ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda")
    L.sparsesam_norm_residual_backward(
        cfg, v["y"], x_out, v["gate"], v["scale"], v["post_w"], v["post_b"], v["pre_w"], stats,
        dx_out, dn, dx, dy, g["dgate"], g["dscale"], g["dpost_w"], g["dpost_b"], g["dpre_w"],
        g["dpre_b"], ws, nb, stream=stream)
    return dx, dy, g


def _check_backward(v, per_gate, kind, dtype, x_out, dx_out, dn, dx, dy, g):
    """Row gradients: with m = S (|g| + mean|g| + |h| mean|g h|) rstd for each norm's own sums and
    E_h through its terms, all taken as 8 of that; then u of the output. Column sums over R rows: the
    terms' errors (D's own and E_h) plus R 2^-24 (at most R joins) of the sum of magnitudes."""
    o = {k: f64(t) for k, t in v.items()}
    xo, dxo, dnn = f64(x_out), f64(dx_out), f64(dn)
    want = X.norm_residual_backward(o["y"], xo, o["gate"], per_gate, o["scale"], o["post_w"],
                                    o["post_b"], o["pre_w"], kind, EPS, dxo, dnn)
    R = len(xo)

    def through(gr, h, eh, rstd):
        """Magnitude of the error of a norm's input gradient for g = gr."""
        a = np.abs(gr)
        return rstd * (8 * S * (a + a.mean(1, keepdims=True) + np.abs(h) * (a * np.abs(h)).mean(1, keepdims=True))
                       + eh * (a * np.abs(h)).mean(1, keepdims=True)
                       + np.abs(h) * (a * eh).mean(1, keepdims=True))

    D, d_off = want["dx"], 2.0 ** -22 * np.abs(dxo)
    if o["pre_w"] is not None:
        h, eh = _h_off(xo, kind)
        rstd = X.norm_stats(xo, kind, EPS)[1]
        d_off = d_off + through(dnn * o["pre_w"], h, eh, rstd)
    tol = U[dtype] * np.abs(D) + d_off + TINY[dtype]
    got = f64(dx)
    assert (np.abs(got - D) <= tol).all(), float((np.abs(got - D) / tol).max())
    G = X.gate_rows(o["gate"], R, per_gate) * np.ones((R, 1))
    Sc = 1.0 if o["scale"] is None else o["scale"]
    h, eh, w, b = o["y"], 0.0 * o["y"], 1.0, 0.0
    q, q_off = D * G * Sc, np.abs(G * Sc) * (d_off + 2.0 ** -22 * np.abs(D))
    dy_off = q_off
    if o["post_w"] is not None:
        h, eh = _h_off(o["y"], kind)
        w, b = o["post_w"], (0.0 if o["post_b"] is None else o["post_b"])
        rstd = X.norm_stats(o["y"], kind, EPS)[1]
        qo = q_off * np.abs(w)
        dy_off = through(q * w, h, eh, rstd) + rstd * (
            qo + qo.mean(1, keepdims=True) + np.abs(h) * (qo * np.abs(h)).mean(1, keepdims=True))
    tol = U[dtype] * np.abs(want["dy"]) + dy_off + TINY[dtype]
    assert (np.abs(f64(dy) - want["dy"]) <= tol).all(), float((np.abs(f64(dy) - want["dy"]) / tol).max())
    add = (R + 16) * 2.0 ** -24 + 2.0 ** -21
    a = np.abs
    aw, ab = a(w), a(b)
    # sum D h and sum D, each with its terms' errors and the additions'
    t1 = a(D) * a(h) * add + d_off * a(h) + a(D) * eh
    t0 = a(D) * add + d_off
    bounds = {"dscale": (a(G) * (aw * t1 + ab * t0)).sum(0), "dpost_w": a(Sc) * (a(G) * t1).sum(0),
              "dpost_b": a(Sc) * (a(G) * t0).sum(0)}
    if o["gate"] is not None:
        bounds["dgate"] = np.zeros_like(o["gate"])
        np.add.at(bounds["dgate"], np.arange(R) // per_gate, a(Sc) * (aw * t1 + ab * t0))
    if o["pre_w"] is not None:
        hp, ehp = _h_off(xo, kind)
        bounds["dpre_w"] = (a(dnn) * (a(hp) * add + ehp)).sum(0)
        bounds["dpre_b"] = (a(dnn) * add).sum(0)
    for k, t in g.items():
        if t is None:
            continue
        err = a(f64(t) - want[k])
        assert (err <= bounds[k] + 1e-30).all(), (k, float((err / (bounds[k] + 1e-30)).max()))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    rows, C, dtype, kind, per_gate, post, gate, scale, pre = case
    v = _inputs(*case, seed=1)
    cfg = _cfg(rows, C, dtype, kind, per_gate, gate)
    x_out, n, stats = _forward(cfg, v, pre)
    g = torch.Generator().manual_seed(9)
    dx_out = torch.randn(rows, C, generator=g).to(x_out)
    dn = torch.randn(rows, C, generator=g).to(x_out) if pre else None
    dx, dy, grads = _backward(cfg, v, x_out, stats, dx_out, dn)
    assert L.sparsesam_device_status() == L.SS_OK
    _check_backward(v, per_gate, kind, dtype, x_out, dx_out, dn, dx, dy, grads)
    # the same bits again; in place; only one gradient wanted
    dx2, dy2, grads2 = _backward(cfg, v, x_out, stats, dx_out, dn)
    y, d = v["y"].clone(), dx_out.clone()
    _backward(cfg, {**v, "y": y}, x_out, stats, d, dn, dx=d, dy=y, skip=("post_w", "pre_b", "gate"))
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dy, dy2) and torch.equal(dx, d) and torch.equal(dy, y)
    for k, t in grads.items():
        assert t is None or torch.equal(t, grads2[k]), k


def test_in_place_and_strides():
    """x_out over x, n over y; rows of a wider buffer, whose other columns stay as they were."""
    rows, C, ld = 45, 200, 264
    v = _inputs(rows, C, "bf16", "layer", 9, True, True, True, True)
    cfg = _cfg(rows, C, "bf16", "layer", 9, True)
    x_out, n, stats = _forward(cfg, v, True)
    x, y = v["x"].clone(), v["y"].clone()
    _forward(cfg, {**v, "x": x, "y": y}, True, x_out=x, n=y)
    wide = torch.full((3, rows, ld), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[0, :, :C], wide[1, :, :C] = v["y"], v["x"]
    cfg2 = _cfg(rows, C, "bf16", "layer", 9, True, ld_y=ld, ld_x=ld, ld_n=ld)
    st2 = torch.empty(rows, 4, device="cuda")
    L.sparsesam_norm_residual(cfg2, wide[0], wide[1], v["gate"], v["scale"], v["post_w"],
                              v["post_b"], v["pre_w"], v["pre_b"], wide[1], wide[2], st2)
    torch.cuda.synchronize()
    assert torch.equal(x, x_out) and torch.equal(y, n)
    assert torch.equal(wide[1, :, :C], x_out) and torch.equal(wide[2, :, :C], n)
    assert torch.equal(st2, stats) and (wide[:, :, C:] == 5.0).all()
    dx_out, dn = torch.randn_like(x_out), torch.randn_like(x_out)
    dx, dy, g = _backward(cfg, v, x_out, stats, dx_out, dn)
    w2 = torch.full((6, rows, ld), 5.0, dtype=torch.bfloat16, device="cuda")
    for i, t in enumerate((v["y"], x_out, dx_out, dn)):
        w2[i, :, :C] = t
    dx2, dy2, g2 = _backward(cfg2, {**v, "y": w2[0]}, w2[1], stats, w2[2], w2[3], dx=w2[4],
                             dy=w2[5])
    torch.cuda.synchronize()
    assert torch.equal(dx, w2[4, :, :C]) and torch.equal(dy, w2[5, :, :C])
    assert (w2[:, :, C:] == 5.0).all()
    for k in g:
        assert torch.equal(g[k], g2[k]), k


def test_constant_rows_and_infinities():
    """A constant row has variance 0 (rstd = 1/sqrt(eps), finite); a row with an infinity or a NaN
    spoils itself only."""
    rows, C = 6, 256
    v = _inputs(rows, C, "bf16", "layer", 6, True, False, False, True)
    v["y"][1] = 3.0
    v["y"][3, 5] = float("inf")
    v["x"][4, 7] = float("nan")
    cfg = _cfg(rows, C, "bf16", "layer", 6, False)
    x_out, n, stats = _forward(cfg, v, True)
    torch.cuda.synchronize()
    fine = [0, 1, 2, 5]
    assert torch.isfinite(x_out[fine]).all() and torch.isfinite(n[fine]).all()
    assert torch.isnan(n[[3, 4]]).all() and torch.isnan(x_out[4, 7])
    sub = {k: t if k not in ("x", "y") else t[fine] for k, t in v.items()}
    _check_forward(sub, 6, "layer", "bf16", x_out[fine], n[fine], stats[fine])
    assert abs(stats[1, 1].item() - 1e3) <= 1e3 * 2 * S


def test_a_spoiled_call_leaves_nothing_behind():
    """A call on NaN rows, then one whose workers have an odd row left over: shared memory still holds
    the NaN where that row's partner would be."""
    C = 1024
    for rows in (1777, 3):
        v = _inputs(rows, C, "bf16", "layer", rows, True, True, True, True, seed=4)
        cfg = _cfg(rows, C, "bf16", "layer", rows, True)
        x_out, n, stats = _forward(cfg, v, True)
        dx_out, dn = torch.randn_like(x_out), torch.randn_like(x_out)
        want = _backward(cfg, v, x_out, stats, dx_out, dn)
        big = _inputs(4000, C, "bf16", "layer", 4000, True, True, True, True)
        nan = torch.full_like(big["x"], float("nan"))
        bcfg = _cfg(4000, C, "bf16", "layer", 4000, True)
        _backward(bcfg, {**big, "y": nan}, nan, torch.full((4000, 4), float("nan"), device="cuda"), nan, nan)
        got = _backward(cfg, v, x_out, stats, dx_out, dn)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        for k in want[2]:
            assert torch.equal(want[2][k], got[2][k]), k
        _check_backward(v, rows, "layer", "bf16", x_out, dx_out, dn, *got)


def test_no_rows():
    v = _inputs(0, 64, "bf16", "layer", 4, True, True, True, True)
    cfg = _cfg(0, 64, "bf16", "layer", 4, True)
    _forward(cfg, v, True)
    _, _, g = _backward(cfg, v, v["x"], torch.empty(0, 4, device="cuda"), v["x"], v["x"])
    torch.cuda.synchronize()
    for k in ("dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b"):
        assert (g[k] == 0).all(), k


def test_captured_and_on_another_stream():
    rows, C = 700, 384
    v = _inputs(rows, C, "bf16", "layer", 100, True, True, True, True)
    cfg = _cfg(rows, C, "bf16", "layer", 100, True)
    dx_out, dn = torch.randn_like(v["x"]), torch.randn_like(v["x"])
    x_out, n, stats = _forward(cfg, v, True)
    want = _backward(cfg, v, x_out, stats, dx_out, dn)
    out = [torch.empty_like(t) for t in (x_out, n, stats, *want[:2])]
    grads = {k: None if t is None else torch.empty_like(t) for k, t in want[2].items()}
    ws = torch.empty(L.sparsesam_norm_residual_backward_workspace(cfg), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st = torch.cuda.current_stream()
        _forward(cfg, v, True, out[0], out[1], out[2], stream=st)
        _backward(cfg, v, out[0], out[2], dx_out, dn, out[3], out[4], stream=st, grads=grads, ws=ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, (x_out, n, stats, *want[:2])):
            assert torch.equal(a, b)
        for k in grads:
            assert grads[k] is None or torch.equal(grads[k], want[2][k])


def test_rows_past_32_bits():
    """More than 2^31 channels: the last rows, and the sums over all of them where the rows repeat."""
    C, part = 2048, 512
    rows = (1 << 20) + 3 * part
    assert rows * C > 1 << 31
    small = _inputs(part, C, "bf16", "layer", part, True, True, True, True)
    many = rows // part
    tile = lambda t: t.repeat(many, 1)  # noqa: E731
    v = {**small, "x": tile(small["x"]), "y": tile(small["y"])}
    cfg = _cfg(rows, C, "bf16", "layer", rows, True)
    x_out, n, stats = _forward(cfg, v, True, x_out=v["x"], n=torch.full_like(v["x"], 7.0))
    torch.cuda.synchronize()
    for at in (0, (1 << 20) - part, rows - part):
        s = slice(at, at + part)
        _check_forward(small, part, "layer", "bf16", x_out[s], n[s], stats[s])
    for s in range(part, rows, part):
        assert torch.equal(x_out[s:s + part], x_out[:part]) and torch.equal(n[s:s + part], n[:part])
    del n
    dx_out, dn = torch.randn_like(small["x"]), torch.randn_like(small["x"])
    big = tile(dx_out)
    dx, dy, g = _backward(cfg, v, x_out, stats, big, tile(dn), dx=big, dy=v["y"])
    torch.cuda.synchronize()
    one = _backward(_cfg(part, C, "bf16", "layer", part, True), small, x_out[:part].clone(),
                    stats[:part].clone(), dx_out, dn)
    _check_backward(small, part, "layer", "bf16", x_out[:part], dx_out, dn, *one)
    for s in range(0, rows, part):
        assert torch.equal(dx[s:s + part], dx[:part]) and torch.equal(dy[s:s + part], dy[:part])
    assert torch.equal(dx[-part:], one[0]) and torch.equal(dy[-part:], one[1])

"""The norms around a block at the row counts where their many-row kernels run: constant rows, every
width class, strides, in-place calls, captured calls and sums over many rows. Tolerances are those of
test_gpu_norm.py unless a test says otherwise."""
import numpy as np
import pytest
import torch

import test_gpu_norm as N
from oracle import expert_oracle as X
from structured_activation_sparsity_b200 import _lib as L

pytestmark = pytest.mark.gpu

# rows, C, dtype: few rows (the direct kernel), then many: one warp a row or several, whole and ragged spans
CONSTANT = [(6, 256, "bf16"), (40, 1160, "f32"), (5, 4096, "f16"), (10400, 40, "f16"), (5200, 128, "bf16"),
            (2000, 1280, "bf16"), (2000, 1160, "f32"), (1200, 2056, "bf16"), (800, 4096, "bf16"),
            (700, 3880, "f32"), (800, 4096, "f32")]


@pytest.mark.parametrize("rows,C,dtype", CONSTANT, ids=lambda v: str(v))
def test_constant_rows_cancel(rows, C, dtype):
    """A row of C equal values of at most 8 significant bits has sums that fp32 holds exactly, so its mean
    is the value, its deviations are 0 and its LayerNorm is the bias, bit for bit, however large the
    value is against the norm's eps; h is 0 in the gradients, too."""
    dt = N.TORCH[dtype]
    values = torch.tensor([0.0, 1.0, -3.0, 1000.0, 30720.0, 0.109375, -251.0])
    col = values[torch.arange(rows) % 7].to(dt).cuda()[:, None]
    v = N._inputs(rows, C, dtype, "layer", rows, True, True, True, True, seed=3)
    v["y"] = col.expand(rows, C).contiguous()
    cfg = N._cfg(rows, C, dtype, "layer", rows, False)
    zero = torch.zeros_like(v["y"])
    # the post norm: 0 + bias
    post = {**v, "x": zero, "gate": None, "scale": None, "pre_w": None, "pre_b": None}
    x_out, _, stats = N._forward(cfg, post, False)
    assert torch.equal(x_out, v["post_b"].expand(rows, C))
    assert torch.equal(stats[:, 0], col[:, 0].float())
    assert ((stats[:, 1].double() - 1e3).abs() <= 1e3 * 2 * N.S).all()
    # the pre norm of 0 + the constant
    pre = {**post, "x": v["y"], "y": zero, "post_w": None, "post_b": None, "pre_w": v["pre_w"],
           "pre_b": v["pre_b"]}
    x_out, n, stats = N._forward(cfg, pre, True)
    assert torch.equal(x_out, v["y"]) and torch.equal(n, v["pre_b"].expand(rows, C))
    assert torch.equal(stats[:, 2], col[:, 0].float())
    # gradients: h = 0 in both norms, so the weights' gradients are 0
    both = {**v, "gate": None, "x": zero}
    stats[:, :2] = stats[:, 2:]
    d = torch.randn(2, rows, C, device="cuda").to(dt)
    _, _, g = N._backward(cfg, both, v["y"], stats, d[0], d[1])
    assert (g["dpost_w"] == 0).all() and (g["dpre_w"] == 0).all()
    assert L.sparsesam_device_status() == L.SS_OK


# rows of several rounds of the many-row kernels (16, 8 or 4 rows a CTA at a time), with each norm alone and both
ROUNDS = [(800, 4096, "f32"), (1500, 2560, "f32"), (3000, 4096, "bf16"), (3000, 2056, "f16"),
          (5000, 1280, "bf16"), (9000, 256, "f32"), (30000, 64, "bf16")]


@pytest.mark.parametrize("norms", ["post", "pre", "both", "none"])
@pytest.mark.parametrize("rows,C,dtype", ROUNDS, ids=lambda v: str(v))
def test_no_row_meets_the_next_one(rows, C, dtype, norms):
    """Copies of later rows go into the shared memory that a row is read from. With constant rows of very
    different values, exact sums and exact outputs, a single channel of another row shows. (fp32 gradients'
    column sums of constant rows and of gradients that are small whole numbers are exact as well.)"""
    dt = N.TORCH[dtype]
    col = torch.tensor([0.0, 1.0, -3.0, 1000.0, 30720.0, 0.109375, -251.0])[torch.arange(rows) % 7]
    col = col.to(dt).cuda()[:, None]
    flat, zero = col.expand(rows, C).contiguous(), torch.zeros(rows, C, dtype=dt, device="cuda")
    post, pre = norms in ("post", "both"), norms in ("pre", "both")
    v = N._inputs(rows, C, dtype, "layer", rows, post, False, False, pre, seed=3)
    v["y"], v["x"] = flat, zero
    cfg = N._cfg(rows, C, dtype, "layer", rows, False)
    want = v["post_b"].expand(rows, C) if post else flat
    for _ in range(20):
        x_out, n, stats = N._forward(cfg, v, pre)
        assert torch.equal(x_out, want)
        if post:
            assert torch.equal(stats[:, 0], col[:, 0].float())
        elif pre:
            assert torch.equal(stats[:, 2], col[:, 0].float()) and torch.equal(n, v["pre_b"].expand(rows, C))
    # gradients: dx_out and dn whole numbers -1, 0, 1 along the rows
    d = ((torch.arange(rows) % 3) - 1).to(dt).cuda()[:, None].expand(rows, C).contiguous()
    scaled = {**v, "scale": torch.ones(C, dtype=dt, device="cuda")}
    for key in ("post_w", "pre_w"):
        if v[key] is not None:
            scaled[key] = torch.ones(C, dtype=dt, device="cuda")
    for key in ("post_b", "pre_b"):
        scaled[key] = None
    st = torch.zeros(rows, 4, device="cuda")
    st[:, 0], st[:, 2], st[:, 1], st[:, 3] = col[:, 0].float(), col[:, 0].float(), 1.0, 1.0
    total = d.double().sum(0).float()
    for _ in range(20):
        dx, dy, g = N._backward(cfg, scaled, flat, st, d, d if pre else None)
        # a constant gradient of a norm: g - mean(g) = 0 (LayerNorm), so D = d with or without the pre norm
        assert torch.equal(dx, d)
        if post:
            assert (dy == 0).all() and (g["dpost_w"] == 0).all() and (g["dscale"] == 0).all()
        else:
            assert torch.equal(dy, d)
            big = (d.double() * flat.double()).sum(0)
            assert ((g["dscale"].double() - big).abs() <= rows * 2.0 ** -24 * (d * flat).double().abs().sum(0)).all()
        if pre:
            assert (g["dpre_w"] == 0).all()
    assert L.sparsesam_device_status() == L.SS_OK

@pytest.mark.parametrize("rows,C", [(20, 1280), (3000, 1280), (5200, 128), (900, 4096)])
def test_parameters_written_by_the_call_before(rows, C):
    """Gates are activations: gate, scale and weights that the library call just before writes, with no
    wait in between, count as written, in the forward and in the gradient."""
    groups, eps = 4, 1e-6
    v = N._inputs(rows, C, "bf16", "layer", -(-rows // groups), True, True, True, True, seed=6)
    cfg = N._cfg(rows, C, "bf16", "layer", -(-rows // groups), True)
    big = 40000
    src = torch.randn(big, C, device="cuda").bfloat16()
    made = torch.empty_like(src)
    bcfg = L.make_norm_cfg(big, C, eps=eps)
    d = torch.randn(2, rows, C, device="cuda").bfloat16()
    # rows of `made`: the gate rows, then scale and the norms' parameters, first and last of them
    at = dict(scale=groups, post_w=groups + 1, post_b=big - 1, pre_w=big - 2, pre_b=big - 3)
    v.update(gate=made[:groups], **{k: made[i] for k, i in at.items()})

    def make():
        L.sparsesam_norm_residual(bcfg, src, src, None, None, None, None, None, None, made, None, None)
    make()
    torch.cuda.synchronize()
    x_out, n, stats = N._forward(cfg, v, True)
    want = N._backward(cfg, v, x_out, stats, d[0], d[1])
    N._check_forward(v, -(-rows // groups), "layer", "bf16", x_out, n, stats)
    torch.cuda.synchronize()
    for _ in range(20):
        made.fill_(float("nan"))
        out, n2 = torch.empty_like(x_out), torch.empty_like(n)
        make()
        N._forward(cfg, v, True, x_out=out, n=n2)
        assert torch.equal(out, x_out) and torch.equal(n2, n)
        made.fill_(float("nan"))
        ws = torch.empty(L.sparsesam_norm_residual_backward_workspace(cfg), dtype=torch.uint8, device="cuda")
        dx, dy = torch.empty_like(x_out), torch.empty_like(x_out)
        grads = {k: None if t is None else torch.empty_like(t) for k, t in want[2].items()}
        make()
        N._backward(cfg, v, x_out, stats, d[0], d[1], dx=dx, dy=dy, grads=grads, ws=ws)
        assert torch.equal(dx, want[0]) and torch.equal(dy, want[1])
        for k, t in grads.items():
            assert torch.equal(t, want[2][k]), k


# the many-row forward's width classes, whole and ragged: rows, C, dtype, kind, per_gate, post, gate, scale, pre
WIDTHS = [
    (6000, 8, "bf16", "layer", 7, True, True, True, True), (5200, 56, "f32", "rms", 100, True, True, False, True),
    (4000, 128, "bf16", "layer", 1000, True, True, True, True), (4000, 104, "f16", "layer", 9, True, True, True, True),
    (4000, 72, "f32", "rms", 50, False, True, True, True), (3000, 256, "bf16", "layer", 64, True, True, True, True),
    (3000, 200, "f32", "layer", 1, True, True, True, True), (3000, 136, "f16", "rms", 11, True, False, True, True),
    (1500, 768, "bf16", "layer", 300, True, True, True, True), (1500, 520, "f32", "layer", 4, True, True, True, True),
    (900, 1736, "bf16", "layer", 100, True, True, True, True), (900, 1792, "f16", "rms", 90, True, True, True, True),
    (700, 2048, "f32", "layer", 70, True, True, True, True), (700, 1288, "f32", "rms", 70, True, True, True, True),
    (700, 2560, "f32", "layer", 100, True, True, True, True), (700, 2304, "bf16", "layer", 100, True, True, True, True),
    (700, 3584, "f16", "layer", 77, True, True, True, True), (700, 3400, "bf16", "rms", 8, True, True, True, True),
    # several warps a row with one norm alone
    (700, 4096, "bf16", "layer", 100, True, True, True, False), (700, 4096, "bf16", "rms", 100, False, True, True, True),
    (600, 3880, "f32", "layer", 60, True, True, False, False), (600, 3880, "f32", "rms", 60, False, False, True, True),
    (1200, 2056, "f16", "layer", 60, True, False, False, False), (800, 2816, "bf16", "layer", 60, False, True, False, True),
]


@pytest.mark.parametrize("case", WIDTHS, ids=["-".join(map(str, c)) for c in WIDTHS])
def test_widths(case):
    rows, C, dtype, kind, per_gate, post, gate, scale, pre = case
    v = N._inputs(*case, seed=2)
    cfg = N._cfg(rows, C, dtype, kind, per_gate, gate)
    x_out, n, stats = N._forward(cfg, v, pre)
    assert L.sparsesam_device_status() == L.SS_OK
    N._check_forward(v, per_gate, kind, dtype, x_out, n, stats)
    d = torch.randn(2, rows, C, device="cuda").to(x_out)
    dx, dy, grads = N._backward(cfg, v, x_out, stats, d[0], d[1] if pre else None)
    N._check_backward(v, per_gate, kind, dtype, x_out, d[0], d[1] if pre else None, dx, dy, grads)
    # rows of wider buffers, x_out over x and n over y: the same bits, and nothing beside the rows
    ld = C + 24
    wide = torch.full((2, rows, ld), 5.0, dtype=x_out.dtype, device="cuda")
    wide[0, :, :C], wide[1, :, :C] = v["y"], v["x"]
    cfg2 = N._cfg(rows, C, dtype, kind, per_gate, gate, ld_y=ld, ld_x=ld, ld_n=ld)
    st2 = torch.empty_like(stats)
    L.sparsesam_norm_residual(cfg2, wide[0], wide[1], v["gate"], v["scale"], v["post_w"], v["post_b"],
                              v["pre_w"], v["pre_b"], wide[1], wide[0] if pre else None, st2)
    torch.cuda.synchronize()
    assert torch.equal(wide[1, :, :C], x_out) and torch.equal(st2, stats)
    assert torch.equal(wide[0, :, :C], n if pre else v["y"]) and (wide[:, :, C:] == 5.0).all()
    if pre and dtype != "f16":
        # n is what a call with nothing but the norm makes of x_out
        alone, zero = torch.empty_like(x_out), torch.zeros_like(x_out)
        L.sparsesam_norm_residual(N._cfg(rows, C, dtype, kind, 1, False), x_out, zero, None, None, v["pre_w"],
                                  v["pre_b"], None, None, alone, None, None)
        torch.cuda.synchronize()
        assert torch.equal(alone, n)


@pytest.mark.parametrize("rows,C", [(3000, 200), (2000, 1280), (900, 4096)])
def test_spoiled_rows_stay_alone(rows, C):
    """A row with an infinity or a NaN spoils itself only, wherever it is in a block's rounds."""
    v = N._inputs(rows, C, "bf16", "layer", rows, True, True, True, True, seed=5)
    cfg = N._cfg(rows, C, "bf16", "layer", rows, True)
    want = N._forward(cfg, v, True)
    bad = torch.tensor([0, 17, rows // 2, rows - 1], device="cuda")
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[bad] = False
    w = {**v, "y": v["y"].clone(), "x": v["x"].clone()}
    w["y"][bad[:2], 5] = float("inf")
    w["x"][bad[2:], C - 1] = float("nan")
    got = N._forward(cfg, w, True)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[fine], b[fine])
    assert torch.isnan(got[1][bad]).all()


@pytest.mark.parametrize("rows,C,dtype", [(5000, 1280, "bf16"), (800, 4096, "f32")])
def test_many_rows_captured(rows, C, dtype):
    """A captured call on another stream, replayed with other rows in the same buffers."""
    a, b = (N._inputs(rows, C, dtype, "layer", 100, True, True, True, True, seed=s) for s in (7, 8))
    cfg = N._cfg(rows, C, dtype, "layer", 100, True)
    want = [N._forward(cfg, {**a, "y": t["y"], "x": t["x"]}, True) for t in (a, b)]
    live = {**a, "y": a["y"].clone(), "x": a["x"].clone()}
    out = [torch.empty_like(t) for t in want[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        N._forward(cfg, live, True, *out, stream=torch.cuda.current_stream())
    for i, t in ((1, b), (0, a), (1, b)):
        live["y"].copy_(t["y"])
        live["x"].copy_(t["x"])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want[i]):
            assert torch.equal(x, y)


def test_parameter_gradients_past_32_bits():
    """More than 2^31 channels whose rows repeat: every parameter's gradient is that many times the one of the
    rows that repeat. Each of the 296 workers adds 3548 rows one after another, 148 CTAs' sums follow:
    (3548 + 148 + 16) 2^-24 of the sum of magnitudes, besides the terms' own errors."""
    C, part = 2048, 512
    rows = (1 << 20) + 3 * part
    many = rows // part
    assert rows * C > 1 << 31 and rows % part == 0
    v = N._inputs(part, C, "bf16", "layer", part, True, True, True, True)
    x_out, _, stats = N._forward(N._cfg(part, C, "bf16", "layer", part, True), v, True)
    g = torch.Generator().manual_seed(4)
    d = [torch.randn(part, C, generator=g).bfloat16().cuda() for _ in range(2)]
    tile = lambda t: t.repeat(many, 1)  # noqa: E731
    big = {**v, "y": tile(v["y"])}
    ws = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    dx = tile(d[0])
    _, _, got = N._backward(N._cfg(rows, C, "bf16", "layer", rows, True), big, tile(x_out), tile(stats), dx,
                            tile(d[1]), dx=dx, dy=big["y"], ws=ws)
    o = {k: N.f64(t) for k, t in v.items()}
    xo, dxo, dnn = N.f64(x_out), N.f64(d[0]), N.f64(d[1])
    want = X.norm_residual_backward(o["y"], xo, o["gate"], part, o["scale"], o["post_w"], o["post_b"],
                                    o["pre_w"], "layer", N.EPS, dxo, dnn)
    a, S = np.abs, N.S
    add = (3548 + 148 + 16) * 2.0 ** -24 + 2.0 ** -21
    h, eh = N._h_off(o["y"], "layer")
    hp, ehp = N._h_off(xo, "layer")
    rstd = X.norm_stats(xo, "layer", N.EPS)[1]
    gr = a(dnn * o["pre_w"])
    d_off = 2.0 ** -22 * a(dxo) + rstd * (
        8 * S * (gr + gr.mean(1, keepdims=True) + a(hp) * (gr * a(hp)).mean(1, keepdims=True))
        + ehp * (gr * a(hp)).mean(1, keepdims=True) + a(hp) * (gr * ehp).mean(1, keepdims=True))
    D, G = a(want["dx"]), a(o["gate"])
    t1, t0 = D * a(h) * add + d_off * a(h) + D * eh, D * add + d_off
    pair = a(o["post_w"]) * t1 + a(o["post_b"]) * t0
    bounds = {"dgate": (a(o["scale"]) * pair).sum(0, keepdims=True), "dscale": (G * pair).sum(0),
              "dpost_w": (a(o["scale"]) * G * t1).sum(0), "dpost_b": (a(o["scale"]) * G * t0).sum(0),
              "dpre_w": (a(dnn) * (a(hp) * add + ehp)).sum(0), "dpre_b": (a(dnn) * add).sum(0)}
    for k, bound in bounds.items():
        err = a(N.f64(got[k]) - many * want[k])
        assert (err <= many * bound).all(), (k, float((err / (many * bound)).max()))
    assert L.sparsesam_device_status() == L.SS_OK

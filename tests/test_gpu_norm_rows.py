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

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

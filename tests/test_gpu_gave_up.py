"""Calls whose device waits give up at once: the limit is set so low that a wait for a copy that has only
just been asked for runs out. Whatever was recorded, each kernel must have waited for its own copies before
it ended, and the calls that follow, on the same shared memory, are right."""
import pytest
import torch

import test_gpu_experts as G
import test_gpu_norm as N
from structured_activation_sparsity_b200 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture
def hasty():
    """A limit of one nanosecond while the test holds it."""
    def on(limit):
        torch.cuda.synchronize()
        L.sparsesam_set_wait_limit_ns(limit)
    yield on
    on(0)


@pytest.mark.parametrize("rows,C,dtype", [(5000, 1280, "bf16"), (800, 4096, "f32"), (30000, 64, "bf16"),
                                          (3000, 2056, "f16")])
@pytest.mark.parametrize("norms", [(True, True), (True, False), (False, True)])
def test_norms(hasty, rows, C, dtype, norms):
    post, pre = norms
    v = N._inputs(rows, C, dtype, "layer", 100, post, True, True, pre)
    cfg = N._cfg(rows, C, dtype, "layer", 100, True)
    x_out, n, stats = N._forward(cfg, v, pre)
    d = torch.randn(2, rows, C, device="cuda").to(x_out)
    dn = d[1] if pre else None
    want = N._backward(cfg, v, x_out, stats, d[0], dn)
    assert L.sparsesam_device_status() == L.SS_OK
    for _ in range(3):
        hasty(1)
        for _ in range(5):
            N._forward(cfg, v, pre)
            N._backward(cfg, v, x_out, stats, d[0], dn)
        assert L.sparsesam_device_status() in (L.SS_OK, L.SS_ETIMEOUT)
        hasty(0)
        again = N._forward(cfg, v, pre)
        got = N._backward(cfg, v, x_out, stats, d[0], dn)
        assert torch.equal(again[0], x_out) and torch.equal(again[2], stats)
        assert not pre or torch.equal(again[1], n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for k in want[2]:
            assert want[2][k] is None or torch.equal(got[2][k], want[2][k]), k
        assert L.sparsesam_device_status() == L.SS_OK


@pytest.mark.parametrize("T,E,k,C,H", [(12, 4, 2, 64, 1024), (100, 4, 1, 256, 512), (900, 64, 2, 64, 1096),
                                       (1100, 40, 2, 64, 2056), (1200, 4, 2, 256, 1024), (2000, 4, 2, 64, 4800)])
def test_expert_mlp(hasty, T, E, k, C, H):
    """Products by one CTA a tile (64 and 128 rows, with and without k-splits) and by pairs."""
    v = G._mlp_inputs(T, E, k, C, H, 1)
    ids = G._ids(T, E, k, 2)
    cfg = L.make_expert_cfg(T, E, k, C=C, hidden=H)
    want = G._mlp(cfg, v, ids)
    assert L.sparsesam_device_status() == L.SS_OK
    for _ in range(3):
        hasty(1)
        for _ in range(5):
            G._mlp(cfg, v, ids)
        assert L.sparsesam_device_status() in (L.SS_OK, L.SS_ETIMEOUT)
        hasty(0)
        assert torch.equal(G._mlp(cfg, v, ids), want)
        assert L.sparsesam_device_status() == L.SS_OK

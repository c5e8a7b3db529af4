"""The routed-expert calls away from ordinary inputs and at sizes where every CTA has several tiles.
Tolerances are those of test_gpu_experts.py unless a test says otherwise."""
import numpy as np
import pytest
import torch

import test_gpu_experts as G
from oracle import expert_oracle as X
from structured_activation_sparsity_b200 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(4, 4), (64, 8), (512, 16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_far_logits(E, k, renorm):
    """Distances up to 103 from the largest logit, where weights get subnormal. A weight is exp(d) / sum with
    d the logits' difference to within 2^-47 of it: the exponential 2 ulp, a sum of positive terms
    (their errors and at most 16 joins), a division: (2 * 2 + 2 * 16 + 4) 2^-24 relative, under the 64 2^-24 of
    the near logits; a subnormal result is off by a few steps of 2^-149 instead."""
    T = 500
    rng = np.random.default_rng(E)
    lg = -rng.uniform(0, 103, (T, E))
    lg[np.arange(T), rng.integers(0, E, T)] = 0
    lg = (lg + rng.uniform(-40, 40, (T, 1))).astype(np.float32)
    lg = torch.from_numpy(lg).cuda()
    ids, w = G._route(lg, k, renorm)
    want_ids, want = X.route(G.f64(lg), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    err = np.abs(G.f64(w) - want)
    tol = 64 * G.F * want + 4 * 2.0 ** -149
    assert (err <= tol).all(), float((err / tol).max())
    dw = torch.randn(T, k, device="cuda")
    dlg = torch.full((T, E), 7.0, device="cuda")
    L.sparsesam_expert_route_backward(L.make_expert_cfg(T, E, k), lg, renorm, ids, w, dw, dlg)
    want = X.route_backward(G.f64(lg), k, renorm, G.f64(dw))
    # p (dw - mean) as in the near test; subnormal p's steps times |dw - mean|
    z = G.f64(lg)
    prob = np.exp(z - z.max(1, keepdims=True))
    if renorm:
        chosen = np.zeros((T, E), bool)
        np.put_along_axis(chosen, want_ids, True, 1)
        prob *= chosen
    prob /= prob.sum(1, keepdims=True)
    size = 1 + np.abs(G.f64(dw)).max(1, keepdims=True)
    assert (np.abs(G.f64(dlg) - want) <= size * (2 * (64 + 32 + 64) * G.F * prob + 16 * 2.0 ** -149)).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_route_huge_logits(renorm):
    """Logits whose steps are larger than any distance that counts, with closed ones among them. (The last
    row's third weight is e^-128 = 2.6e-56, less than half of fp32's least step: 0, off by itself.)"""
    inf, big = float("inf"), 3.4028234663852886e38
    lg = torch.tensor([[-big, -inf, -big, -inf], [1e30, 1e30, -1e30, 0.0], [big, -big, 0.0, -inf],
                       [-1e30, -inf, -1.0000001e30, -big], [1e9, 1e9 - 64, 1e9 - 128, 0.0]], device="cuda")
    ids, w = G._route(lg, 3, renorm)
    want_ids, want = X.route(G.f64(lg), 3, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(G.f64(w) - want) <= 64 * G.F * want + 2.0 ** -150).all()
    dw = torch.tensor([[1.0, -2.0, 0.5]] * 5, device="cuda")
    dlg = torch.full_like(lg, 7.0)
    L.sparsesam_expert_route_backward(L.make_expert_cfg(5, 4, 3), lg, renorm, ids, w, dw, dlg)
    want = X.route_backward(G.f64(lg), 3, renorm, G.f64(dw))
    assert (np.abs(G.f64(dlg) - want) <= 4 * 160 * G.F * (np.abs(want) + (want != 0))).all()


def test_route_backward_of_an_infinite_logit():
    """A logit of +inf makes the softmax NaN, and so the gradient of every open expert, while closed
    experts (-inf, NaN) have 0 and other tokens their own."""
    inf, nan = float("inf"), float("nan")
    lg = torch.tensor([[0.0, 1.0, 2.0, 3.0, -1.0], [inf, 1.0, -inf, 0.0, nan], [1.0, -inf, nan, 0.5, 2.0]],
                      device="cuda")
    ids, w = G._route(lg, 2, False)
    dw = torch.tensor([[1.0, -2.0]] * 3, device="cuda")
    dlg = torch.full((3, 5), 7.0, device="cuda")
    L.sparsesam_expert_route_backward(L.make_expert_cfg(3, 5, 2), lg, False, ids, w, dw, dlg)
    assert torch.isnan(w[1]).all()
    assert torch.isnan(dlg[1, [0, 1, 3]]).all() and (dlg[1, [2, 4]] == 0).all()
    assert torch.isfinite(dlg[[0, 2]]).all() and (dlg[2, [1, 2]] == 0).all()


MANY_TILES = [
    # tokens, experts, topk, C, hidden. Pairs of CTAs (256 rows a tile): fc1 with over 4 x 74 units, then fc2
    (2000, 4, 2, 64, 4800), (2000, 4, 2, 4800, 64), (2300, 5, 2, 136, 4360),
    # 64 and 128 rows a tile, one CTA each: over 3 x 148 units
    (900, 64, 2, 64, 1096), (900, 64, 2, 1096, 64), (1100, 40, 2, 64, 2056), (1100, 40, 2, 2056, 72),
]


@pytest.mark.parametrize("T,E,k,C,H", MANY_TILES)
def test_expert_mlp_several_tiles_a_cta(T, E, k, C, H):
    """Ragged experts, some without a row, with several units a CTA or pair: its ring, its two
    accumulators and their barriers go round more than once."""
    v = G._mlp_inputs(T, E, k, C, H, T + C)
    ids = G._ids(T, E, k, T + H, gone=0.05, skew=0.5)
    ids[ids == E - 2] = E - 1
    cfg = L.make_expert_cfg(T, E, k, C=C, hidden=H)
    out = G._mlp(cfg, v, ids)
    assert L.sparsesam_device_status() == L.SS_OK
    again = G._mlp(cfg, v, ids)
    assert torch.equal(out, again)
    some = np.unique(np.concatenate([[0, 1, T - 1], np.random.default_rng(T).integers(0, T, 300)]))
    sub = {n: t[some] if n in ("x", "residual", "weight") else t for n, t in v.items()}
    G._check_mlp(sub, ids[torch.from_numpy(some).cuda()], out[torch.from_numpy(some).cuda()])

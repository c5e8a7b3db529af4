"""Pins of the norm and routed-expert oracle: gradients against central differences, the order against
a plain stable sort, closed forms."""
import numpy as np
import pytest

from oracle import expert_oracle as X


def _diff(f, v, d, h=1e-6):
    """Directional derivative of the scalar f at v along d."""
    return (f(v + h * d) - f(v - h * d)) / (2 * h)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_norm_residual_gradients_are_differences(kind, post, gate, pre):
    rng = np.random.default_rng(3)
    R, C, per, eps = 7, 16, 3, 1e-6
    v = dict(y=rng.standard_normal((R, C)), x=rng.standard_normal((R, C)),
             gate=rng.standard_normal((3, C)) if gate else None,
             scale=rng.standard_normal(C) if gate else None,
             post_w=rng.standard_normal(C) if post else None,
             post_b=rng.standard_normal(C) if post else None,
             pre_w=rng.standard_normal(C) if pre else None,
             pre_b=rng.standard_normal(C) if pre else None)
    dx_out, dn = rng.standard_normal((R, C)), rng.standard_normal((R, C)) if pre else None

    def loss(v):
        x_out = X.norm_residual(v["y"], v["x"], v["gate"], per, v["scale"], v["post_w"],
                                v["post_b"], kind, eps)
        s = (x_out * dx_out).sum()
        return s + (X.norm(x_out, v["pre_w"], v["pre_b"], kind, eps) * dn).sum() if pre else s

    x_out = X.norm_residual(v["y"], v["x"], v["gate"], per, v["scale"], v["post_w"], v["post_b"],
                            kind, eps)
    g = X.norm_residual_backward(v["y"], x_out, v["gate"], per, v["scale"], v["post_w"],
                                 v["post_b"], v["pre_w"], kind, eps, dx_out, dn)
    for name, value in v.items():
        if value is None:
            assert "d" + name not in g
            continue
        d = rng.standard_normal(value.shape)
        want = _diff(lambda t: loss({**v, name: t}), value, d)
        assert abs((g["d" + name] * d).sum() - want) <= 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_a_difference(renorm):
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((5, 6))
    logits[1, 2] = -np.inf
    logits[3] = -np.inf
    logits[4, 1:] = -np.inf
    dw = rng.standard_normal((5, 2))
    d = rng.standard_normal(logits.shape)
    f = lambda z: (X.route(z, 2, renorm)[1] * dw).sum()
    assert abs((X.route_backward(logits, 2, renorm, dw) * d).sum() - _diff(f, logits, d)) < 1e-8


def test_route_rows():
    inf = np.inf
    ids, w = X.route(np.array([[0., 1., 1., -inf], [-inf] * 4, [-inf, -inf, -inf, 2.]]), 2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [3, -1]]
    assert np.allclose(w, [[.5, .5], [0, 0], [1, 0]])


def test_sort_is_stable():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 5, (40, 3)).astype(np.int32)
    order, slot, offsets = X.expert_sort(ids, 5)
    flat = ids.reshape(-1)
    live = np.nonzero(flat >= 0)[0]
    want = live[np.argsort(flat[live], kind="stable")]
    assert (order[:len(want)] == want).all() and (order[len(want):] == -1).all()
    assert offsets[-1] == len(want)
    assert all(slot.reshape(-1)[a] == p for p, a in enumerate(want))
    assert (slot[ids < 0] == -1).all()


def test_combine_gradient_is_a_difference():
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, 4, (9, 2)).astype(np.int32)
    _, slot, offsets = X.expert_sort(ids, 4)
    ys, w, dout = rng.standard_normal((18, 8)), rng.standard_normal((9, 2)), rng.standard_normal((9, 8))
    dys, dw = X.combine_backward(dout, ys, slot, w)
    assert np.isnan(dys[offsets[-1]:]).all()
    d = rng.standard_normal(ys.shape)
    f = lambda v: (X.combine(v, slot, w, None) * dout).sum()
    assert abs((np.nan_to_num(dys) * d).sum() - _diff(f, ys, d)) < 1e-7
    d = rng.standard_normal(w.shape)
    f = lambda v: (X.combine(ys, slot, v, None) * dout).sum()
    assert abs((dw * d).sum() - _diff(f, w, d)) < 1e-7


def test_one_expert_is_the_dense_mlp():
    rng = np.random.default_rng(7)
    x, w1, w2 = rng.standard_normal((5, 8)), rng.standard_normal((1, 16, 8)), rng.standard_normal((1, 8, 16))
    out, bound = X.expert_mlp(x, np.zeros((5, 1), np.int32), None, x, w1, None, w2, None)
    assert np.allclose(out, x + X.gelu(x @ w1[0].T) @ w2[0].T) and (bound > 0).all()

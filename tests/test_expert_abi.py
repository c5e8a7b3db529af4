"""Refusals of the norm and routed-expert calls: every case fails on the host before any CUDA call."""
import ctypes

import pytest

from structured_activation_sparsity_b200 import _lib as L

FAKE = 1 << 20      # an aligned, never-dereferenced address
ODD = FAKE + 8
by = ctypes.byref
OK_NORM = dict(rows=10, C=64, dtype="bf16", norm="layer", eps=1e-6, rows_per_gate=5)
OK_X = dict(tokens=10, experts=4, topk=2, C=64, hidden=128)


def _norm(cfg=None, **kw):
    a = dict(y=FAKE, x=FAKE, gate=None, scale=None, post_w=FAKE, post_b=None, pre_w=FAKE,
             pre_b=None, x_out=FAKE, n=2 * FAKE, stats=None)
    a.update(kw)
    return L.lib.sparsesam_norm_residual(by(cfg or L.make_norm_cfg(**OK_NORM)), *a.values(), None)


def _norm_bwd(cfg=None, **kw):
    a = dict(y=FAKE, x_out=FAKE, gate=None, scale=None, post_w=FAKE, post_b=None, pre_w=FAKE,
             stats=FAKE, dx_out=FAKE, dn=FAKE, dx=FAKE, dy=2 * FAKE, dgate=None, dscale=None,
             dpost_w=FAKE, dpost_b=None, dpre_w=FAKE, dpre_b=None, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return L.lib.sparsesam_norm_residual_backward(by(cfg or L.make_norm_cfg(**OK_NORM)),
                                                  *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), L.SS_EINVAL), (dict(C=0), L.SS_EINVAL), (dict(C=60), L.SS_EUNSUPPORTED),
    (dict(C=4104), L.SS_EUNSUPPORTED), (dict(rows=1 << 31), L.SS_EUNSUPPORTED),
    (dict(dtype=3), L.SS_EINVAL), (dict(norm=2), L.SS_EINVAL), (dict(eps=0.0), L.SS_EINVAL),
    (dict(eps=float("nan")), L.SS_EINVAL), (dict(eps=float("inf")), L.SS_EINVAL),
    (dict(rows_per_gate=-1), L.SS_EINVAL), (dict(ld_x=63), L.SS_EINVAL),
    (dict(ld_y=68), L.SS_EINVAL), (dict(ld_n=56), L.SS_EINVAL),
])
def test_norm_cfg(kw, code):
    cfg = L.make_norm_cfg(**{**OK_NORM, **kw})
    assert _norm(cfg) == code
    assert _norm_bwd(cfg) == code
    assert L.sparsesam_norm_residual_backward_workspace(cfg) == 0


def test_norm_arguments():
    assert L.lib.sparsesam_norm_residual(None, *[FAKE] * 11, None) == L.SS_EINVAL
    for name in ("y", "x", "x_out", "n"):
        assert _norm(**{name: None}) == L.SS_EINVAL, name
        assert _norm(**{name: ODD}) == L.SS_EINVAL, name
    for name in ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b", "stats"):
        assert _norm(**{name: ODD}) == L.SS_EINVAL, name
    assert _norm(pre_w=None) == L.SS_EINVAL                    # n without a pre norm
    assert _norm(pre_w=None, n=None, pre_b=FAKE) == L.SS_EINVAL
    assert _norm(post_w=None, post_b=FAKE) == L.SS_EINVAL
    assert _norm(n=FAKE) == L.SS_EINVAL                        # n over x_out
    assert _norm(L.make_norm_cfg(**{**OK_NORM, "rows_per_gate": 0}), gate=FAKE) == L.SS_EINVAL
    # no rows: nothing to do, whatever the row pointers
    assert _norm(L.make_norm_cfg(**{**OK_NORM, "rows": 0}), y=None, x=None, x_out=None, n=None) == L.SS_OK


def test_norm_backward_arguments():
    cfg = L.make_norm_cfg(**OK_NORM)
    assert L.sparsesam_norm_residual_backward_workspace(cfg) > 0
    assert _norm_bwd() == L.SS_EWORKSPACE
    assert _norm_bwd(ws=None, ws_bytes=1 << 30) == L.SS_EWORKSPACE
    assert _norm_bwd(ws=FAKE + 16, ws_bytes=1 << 30) == L.SS_EWORKSPACE
    for name in ("y", "x_out", "stats", "dx_out", "dn", "dx", "dy"):
        assert _norm_bwd(**{name: None}) == L.SS_EINVAL, name
        assert _norm_bwd(**{name: ODD}) == L.SS_EINVAL, name
    assert _norm_bwd(dy=FAKE) == L.SS_EINVAL                   # dx and dy in one place
    for d, p in (("dgate", "gate"), ("dscale", "scale"), ("dpost_w", "post_w"),
                 ("dpost_b", "post_w"), ("dpre_w", "pre_w"), ("dpre_b", "pre_w")):
        assert _norm_bwd(**{p: None, d: FAKE}) == L.SS_EINVAL, d
        assert _norm_bwd(**{d: ODD}) == L.SS_EINVAL, d
    assert _norm_bwd(dn=None, pre_w=None, dpre_w=None) == L.SS_EWORKSPACE
    assert _norm_bwd(dn=FAKE, pre_w=None, dpre_w=None) == L.SS_EINVAL


def _calls(cfg, **kw):
    """The expert calls with arguments that pass, `kw` aside, except that no workspace is given."""
    lib, c = L.lib, by(cfg)
    a = lambda name, v=FAKE: kw.get(name, v)  # noqa: E731
    return {
        "route": lambda: lib.sparsesam_expert_route(c, a("logits"), 1, a("ids"), a("weight"), None),
        "route_backward": lambda: lib.sparsesam_expert_route_backward(
            c, a("logits"), a("renorm", 0), a("ids"), a("weight"), a("dweight"), a("dlogits"), None),
        "sort": lambda: lib.sparsesam_expert_sort(c, a("ids"), a("order"), a("slot"), a("offsets"),
                                                  None, 0, None),
        "gather": lambda: lib.sparsesam_expert_gather(c, a("x"), a("slot"), a("xs", 2 * FAKE), None),
        "combine": lambda: lib.sparsesam_expert_combine(c, a("ys"), a("slot"), a("weight"),
                                                        a("residual"), a("out", 2 * FAKE), None),
        "combine_backward": lambda: lib.sparsesam_expert_combine_backward(
            c, a("dout"), a("ys"), a("slot"), a("weight"), a("dys", 2 * FAKE), a("dweight"), None),
        "mlp": lambda: lib.sparsesam_expert_mlp(c, a("x"), a("ids"), a("weight"), a("residual"),
                                                a("w1"), a("b1"), a("w2"), a("b2"), a("out"), None,
                                                0, None),
    }


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), L.SS_EINVAL), (dict(experts=0), L.SS_EINVAL), (dict(topk=0), L.SS_EINVAL),
    (dict(topk=5), L.SS_EINVAL), (dict(experts=513), L.SS_EUNSUPPORTED),
    (dict(experts=32, topk=17), L.SS_EUNSUPPORTED),
    (dict(tokens=1 << 29), L.SS_EUNSUPPORTED),
])
def test_expert_cfg(kw, code):
    cfg = L.make_expert_cfg(**{**OK_X, **kw})
    for name, call in _calls(cfg).items():
        assert call() == code, name
    assert L.sparsesam_expert_sort_workspace(cfg) == 0
    assert L.sparsesam_expert_mlp_workspace(cfg) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(C=0), L.SS_EINVAL), (dict(C=60), L.SS_EUNSUPPORTED), (dict(dtype=7), L.SS_EINVAL),
    (dict(ld=56), L.SS_EINVAL), (dict(ld=70), L.SS_EINVAL),
])
def test_expert_row_cfg(kw, code):
    calls = _calls(L.make_expert_cfg(**{**OK_X, **kw}))
    for name in ("gather", "combine", "combine_backward", "mlp"):
        assert calls[name]() == code, name


def test_expert_arguments():
    cfg = L.make_expert_cfg(**OK_X)
    needed = {"route": ("logits", "ids", "weight"),
              "route_backward": ("logits", "ids", "weight", "dweight", "dlogits"),
              "sort": ("ids",), "gather": ("x", "slot", "xs"), "combine": ("ys", "slot", "out"),
              "combine_backward": ("dout", "ys", "slot", "weight", "dys", "dweight"),
              "mlp": ("x", "ids", "w1", "w2", "out")}
    for name, args in needed.items():
        for arg in args:
            assert _calls(cfg, **{arg: None})[name]() == L.SS_EINVAL, (name, arg)
    for name, args in {"gather": ("x", "xs"), "combine": ("ys", "residual", "out"),
                       "combine_backward": ("dout", "ys", "dys"),
                       "mlp": ("x", "residual", "w1", "w2", "out")}.items():
        for arg in args:
            assert _calls(cfg, **{arg: ODD})[name]() == L.SS_EINVAL, (name, arg)
    assert _calls(cfg, order=None, slot=None, offsets=None)["sort"]() == L.SS_EINVAL
    assert _calls(cfg, xs=FAKE)["gather"]() == L.SS_EINVAL
    assert _calls(cfg, out=FAKE)["combine"]() == L.SS_EINVAL
    assert _calls(cfg, dys=2 * FAKE, dout=2 * FAKE)["combine_backward"]() == L.SS_EINVAL
    assert _calls(cfg)["mlp"]() == L.SS_EWORKSPACE
    assert L.sparsesam_expert_mlp_workspace(cfg) > 0
    big = L.make_expert_cfg(1 << 20, 8, 2)
    assert L.sparsesam_expert_sort_workspace(big) > 0
    assert _calls(big)["sort"]() == L.SS_EWORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(hidden=0), L.SS_EINVAL), (dict(hidden=100), L.SS_EUNSUPPORTED),
    (dict(dtype="f16"), L.SS_EUNSUPPORTED), (dict(dtype="f32"), L.SS_EUNSUPPORTED),
])
def test_expert_mlp_cfg(kw, code):
    cfg = L.make_expert_cfg(**{**OK_X, **kw})
    assert _calls(cfg)["mlp"]() == code
    assert L.sparsesam_expert_mlp_workspace(cfg) == 0


def test_no_tokens_need_nothing():
    cfg = L.make_expert_cfg(**{**OK_X, "tokens": 0})
    none = dict.fromkeys(("logits", "ids", "weight", "dweight", "dlogits", "x", "slot", "xs", "ys",
                          "residual", "out", "dout", "dys", "w1", "b1", "w2", "b2"))
    calls = _calls(cfg, **none)
    for name in ("route", "route_backward", "gather", "combine", "combine_backward", "mlp"):
        assert calls[name]() == L.SS_OK, name


def test_cfg_makers():
    with pytest.raises(ValueError):
        L.make_norm_cfg(1, 64, dtype="int8")
    with pytest.raises(KeyError):
        L.make_norm_cfg(1, 64, norm="batch")
    with pytest.raises(L.SparseSAMError):
        L.sparsesam_expert_route(L.make_expert_cfg(1, 2, 3), FAKE, 1, FAKE, FAKE)

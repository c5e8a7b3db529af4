"""The routed-expert calls on the GPU against the float64 oracle: router, sort, gather, combine, their
gradients and the whole expert MLP; alone and as they are used together.

Tolerances: ids, order, slot and offsets are equal. Weights are fp32 exponentials (2 ulp) over a sum of
at most 512 of them: 64 * 2^-24 relative covers argument, exponential, tree sum and division. Row
moves copy bits. A combine of k terms is off by (k + 1) 2^-24 of its magnitudes plus one rounding (u);
a dot product of C terms by at most (C / 32 + 8) 2^-24 of its magnitudes. The MLP's bound comes with the
oracle's result."""
import numpy as np
import pytest
import torch

from oracle import expert_oracle as X
from structured_activation_sparsity_b200 import _lib as L

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
F = 2.0 ** -24


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def _logits(T, E, seed, closed=0.1, gone=0.1):
    rng = np.random.default_rng(seed)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    lg[rng.random((T, E)) < closed] = -np.inf
    lg[rng.random(T) < gone] = -np.inf
    # exact ties, zeros of both signs
    lg[::3] = np.round(lg[::3])
    return torch.from_numpy(lg).cuda()


def _route(lg, k, renorm, stream=None):
    T, E = lg.shape
    cfg = L.make_expert_cfg(T, E, k)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    L.sparsesam_expert_route(cfg, lg, renorm, ids, w, stream=stream)
    return ids, w


ROUTES = [(1, 1, 1), (1, 8, 2), (5, 2, 2), (196, 8, 2), (33, 33, 5), (300, 64, 4), (77, 100, 8),
          (50, 256, 6), (40, 512, 16), (9, 16, 16)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, renorm):
    lg = _logits(T, E, T + E)
    ids, w = _route(lg, k, renorm)
    want_ids, want_w = X.route(f64(lg), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(f64(w) - want_w) <= 64 * F * want_w).all()
    dw = torch.randn(T, k, device="cuda")
    dlg = torch.full((T, E), 7.0, device="cuda")
    L.sparsesam_expert_route_backward(L.make_expert_cfg(T, E, k), lg, renorm, ids, w, dw, dlg)
    dw64 = f64(dw)
    want = X.route_backward(f64(lg), k, renorm, dw64)
    # each entry is p (dw - mean): p to 64 ulp, and the mean of at most 16 terms
    p = np.where(np.isfinite(f64(lg)), 1.0, 0.0)
    size = np.abs(dw64).max(1, keepdims=True)
    prob = np.zeros((T, E))
    for t in range(T):
        if renorm:
            for j in range(k):
                if want_ids[t, j] >= 0:
                    prob[t, want_ids[t, j]] = want_w[t, j]
        elif p[t].any():
            z = f64(lg[t])
            e = np.exp(z - z.max())
            prob[t] = e / e.sum()
    assert (np.abs(f64(dlg) - want) <= 2 * (64 + 32 + 64) * F * prob * size + 1e-38).all()
    # a dropped slot's dweight is not read
    dw2 = torch.where(ids < 0, float("nan"), dw)
    dlg2 = torch.empty_like(dlg)
    L.sparsesam_expert_route_backward(L.make_expert_cfg(T, E, k), lg, renorm, ids, w, dw2, dlg2)
    assert torch.equal(dlg, dlg2)


def test_route_special_logits():
    inf, nan = float("inf"), float("nan")
    lg = torch.tensor([[nan, 1.0, nan, 0.0], [-inf, nan, -inf, nan], [-0.0, 0.0, -0.0, -1.0],
                       [-3.4e38, -inf, -3.4e38, -inf], [1e30, 1e30, -1e30, 0.0]], device="cuda")
    ids, w = _route(lg, 3, True)
    assert ids.tolist() == [[1, 3, -1], [-1, -1, -1], [0, 1, 2], [0, 2, -1], [0, 1, 3]]
    assert torch.isfinite(w).all() and (w[1] == 0).all()
    assert np.allclose(f64(w.sum(1)), [1, 0, 1, 1, 1], atol=1e-6)
    ids, w = _route(torch.tensor([[inf, 0.0, 1.0]], device="cuda"), 2, True)
    assert ids.tolist() == [[0, 2]] and torch.isnan(w[0, 0])


def _sort(ids, E, stream=None):
    T, k = ids.shape
    cfg = L.make_expert_cfg(T, E, k)
    order = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    slot = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    nb = L.sparsesam_expert_sort_workspace(cfg)
    ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda")
    L.sparsesam_expert_sort(cfg, ids, order, slot, offsets, ws, nb, stream=stream)
    return order, slot, offsets


def _ids(T, E, k, seed, gone=0.1, skew=1.0):
    rng = np.random.default_rng(seed)
    p = np.exp(skew * rng.standard_normal(E))
    ids = rng.choice(E, size=(T, k), p=p / p.sum()).astype(np.int32)
    ids[rng.random((T, k)) < gone] = -1
    return torch.from_numpy(ids).cuda()


def _check_sort(ids, E):
    got = [t.cpu().numpy() for t in _sort(ids, E)]
    flat = ids.cpu().numpy().reshape(-1)
    live = np.nonzero((flat >= 0) & (flat < E))[0]
    order = live[np.argsort(flat[live], kind="stable")]
    assert np.array_equal(got[0][:len(order)], order) and (got[0][len(order):] == -1).all()
    slot = np.full(flat.size, -1)
    slot[order] = np.arange(len(order))
    assert np.array_equal(got[1].reshape(-1), slot)
    assert np.array_equal(got[2], np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=E))]))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 3, 2), (196, 8, 2), (1365, 12, 3),
                                   (2048, 16, 2), (2049, 16, 2), (20000, 512, 1), (39200, 64, 4),
                                   (70001, 5, 3), (200000, 256, 8)])
def test_sort(T, E, k):
    _check_sort(_ids(T, E, k, T), E)


def test_sort_extremes():
    _check_sort(torch.full((5000, 2), -1, dtype=torch.int32, device="cuda"), 8)   # none routed
    _check_sort(torch.full((5000, 2), 7, dtype=torch.int32, device="cuda"), 8)    # all to one
    _check_sort(torch.arange(300, dtype=torch.int32, device="cuda")[:, None] % 512, 512)
    order, slot, offsets = _sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4)
    assert offsets.tolist() == [0] * 5
    assert L.sparsesam_device_status() == L.SS_OK


@pytest.mark.parametrize("T", [100, 9000])
def test_sort_bad_ids_are_recorded_and_dropped(T):
    ids = _ids(T, 6, 2, 3)
    ids[5, 1], ids[T - 1, 0] = 6, -2
    _check_sort(ids, 6)
    assert L.sparsesam_device_status() == L.SS_EINDEX
    assert L.sparsesam_device_status() == L.SS_OK


ROWS = [(1, 4, 2, 8, "bf16"), (1, 8, 1, 1280, "bf16"), (60, 12, 3, 200, "f32"),
        (257, 8, 2, 768, "bf16"), (100, 16, 6, 264, "f16"), (33, 4, 4, 2056, "f32"),
        (500, 32, 16, 64, "bf16"), (40, 2, 1, 4096, "f16"), (9, 3, 2, 5120, "bf16")]


@pytest.mark.parametrize("T,E,k,C,dtype", ROWS)
@pytest.mark.parametrize("ld", [0, 64])
def test_rows_there_and_back(T, E, k, C, dtype, ld):
    dt, n = TORCH[dtype], T * k
    # distinct experts are not needed: an id may repeat within a token
    ids = _ids(T, E, k, C, gone=0.2 if T > 1 else 0.0)
    _, slot, offsets = _sort(ids, E)
    total = int(offsets[-1])
    stride = C + ld
    cfg = L.make_expert_cfg(T, E, k, C=C, dtype=dtype, ld=stride if ld else 0)
    rows = lambda: torch.randn(T, stride, device="cuda").to(dt)  # noqa: E731
    x, res, dout = rows(), rows(), rows()
    xs = torch.full((n, C), 7.0, dtype=dt, device="cuda")
    L.sparsesam_expert_gather(cfg, x, slot, xs)
    sl = slot.cpu().numpy()
    want = torch.full((n, C), 7.0, dtype=dt)
    for t in range(T):
        for j in range(k):
            if sl[t, j] >= 0:
                want[sl[t, j]] = x[t, :C].cpu()
    assert torch.equal(xs.cpu(), want) and (xs[total:] == 7.0).all()
    w = torch.randn(T, k, device="cuda")
    w[ids < 0] = float("nan")                       # not read
    wz = np.nan_to_num(f64(w))
    for weight, residual in ((w, res), (None, None)):
        out = torch.full((T, stride), 7.0, dtype=dt, device="cuda")
        L.sparsesam_expert_combine(cfg, xs, slot, weight, residual, out)
        r = None if residual is None else f64(residual[:, :C])
        ww = None if weight is None else wz
        ref = X.combine(f64(xs), sl, ww, r)
        mag = X.combine(np.abs(f64(xs)), sl, None if ww is None else np.abs(ww), None if r is None else np.abs(r))
        tol = U[dtype] * np.abs(ref) + (k + 2) * F * mag + TINY[dtype]
        assert (np.abs(f64(out[:, :C]) - ref) <= tol).all()
        assert (out[:, C:] == 7.0).all()
    # in place over the residual
    out2 = res.clone()
    L.sparsesam_expert_combine(cfg, xs, slot, w, out2, out2)
    out3 = torch.empty_like(res)
    L.sparsesam_expert_combine(cfg, xs, slot, w, res, out3)
    assert torch.equal(out2[:, :C], out3[:, :C])
    # gradients
    ys = torch.randn(n, C, device="cuda").to(dt)
    dys = torch.full((n, C), 7.0, dtype=dt, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    L.sparsesam_expert_combine_backward(cfg, dout, ys, slot, w, dys, dw)
    rd, rw = X.combine_backward(f64(dout[:, :C]), f64(ys), sl, wz)
    live = ~np.isnan(rd[:, 0])
    assert live.sum() == total and (dys[total:] == 7.0).all()
    assert (np.abs(f64(dys)[live] - rd[live]) <= (U[dtype] + 2 * F) * np.abs(rd[live]) + TINY[dtype]).all()
    _, mag = X.combine_backward(np.abs(f64(dout[:, :C])), np.abs(f64(ys)), sl, wz)
    assert (np.abs(f64(dw) - rw) <= (C / 32 + 8) * F * mag).all()
    inplace, dw2 = ys.clone(), torch.empty_like(dw)
    L.sparsesam_expert_combine_backward(cfg, dout, inplace, slot, w, inplace, dw2)
    assert torch.equal(inplace[:total], dys[:total]) and torch.equal(dw, dw2)
    assert torch.equal(inplace[total:], ys[total:])


def test_rows_bad_slots_are_recorded_and_skipped():
    T, k, C = 20, 2, 64
    ids = _ids(T, 4, k, 1, gone=0.0)
    _, slot, _ = _sort(ids, 4)
    lost = slot[3, 1].item()
    slot[3, 1] = T * k
    cfg = L.make_expert_cfg(T, 4, k, C=C)
    x = torch.randn(T, C, device="cuda").bfloat16()
    xs = torch.full((T * k, C), 7.0, device="cuda").bfloat16()
    L.sparsesam_expert_gather(cfg, x, slot, xs)
    assert L.sparsesam_device_status() == L.SS_EINDEX
    assert (xs[lost] == 7.0).all() and torch.equal(xs[slot[3, 0].item()], x[3])
    out = torch.empty_like(x)
    L.sparsesam_expert_combine(cfg, xs, slot, None, None, out)
    assert L.sparsesam_device_status() == L.SS_EINDEX
    assert torch.equal(out[3], x[3])
    dys, dw = torch.full_like(xs, 7.0), torch.empty(T, k, device="cuda")
    L.sparsesam_expert_combine_backward(cfg, x, xs, slot, torch.ones(T, k, device="cuda"), dys, dw)
    assert L.sparsesam_device_status() == L.SS_EINDEX
    assert (dys[lost] == 7.0).all() and dw[3, 1] == 0


def _mlp_inputs(T, E, k, C, H, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    b = lambda v: v.bfloat16().cuda()  # noqa: E731
    return dict(x=b(r(T, C)), w1=b(r(E, H, C) / C ** 0.5), b1=b(0.2 * r(E, H)) if bias else None,
                w2=b(r(E, C, H) / H ** 0.5), b2=b(0.2 * r(E, C)) if bias else None,
                residual=b(r(T, C)) if bias else None, weight=r(T, k).abs().cuda())


def _mlp(cfg, v, ids, out=None, ws=None, stream=None):
    out = torch.full((cfg.tokens, cfg.ld or cfg.C), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    nb = L.sparsesam_expert_mlp_workspace(cfg)
    ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    L.sparsesam_expert_mlp(cfg, v["x"], ids, v["weight"], v["residual"], v["w1"], v["b1"], v["w2"],
                           v["b2"], out, ws, nb, stream=stream)
    return out


def _check_mlp(v, ids, out):
    o = {k: f64(t) for k, t in v.items()}
    want, bound = X.expert_mlp(o["x"], ids.cpu().numpy(), o["weight"], o["residual"], o["w1"],
                               o["b1"], o["w2"], o["b2"])
    err = np.abs(f64(out) - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-30)).max())


MLPS = [
    # tokens, experts, topk, C, hidden, bias, skew
    (1, 1, 1, 64, 64, True, 0.0), (1, 8, 2, 256, 1024, True, 0.0), (2, 4, 1, 72, 200, False, 0.0),
    (3, 64, 4, 128, 136, True, 0.0), (40, 8, 2, 128, 256, True, 1.0), (100, 4, 3, 64, 520, True, 1.0),
    (150, 3, 2, 192, 128, False, 1.0), (300, 2, 1, 64, 320, True, 0.0), (513, 2, 2, 64, 64, True, 0.5),
    (700, 1, 1, 136, 72, True, 0.0), (260, 512, 1, 64, 64, True, 1.0), (30, 4, 2, 16, 24, True, 1.0),
    (1500, 4, 2, 64, 128, True, 2.0), (50, 3, 3, 96, 264, True, 0.5), (2, 6, 3, 1288, 2056, True, 0.0),
    (8, 2, 1, 64, 72, False, 0.0), (1, 2, 2, 64, 10240, True, 0.0), (1, 3, 1, 10248, 64, True, 0.0),
    (30, 4, 2, 8, 8, True, 1.0), (12, 4, 2, 64, 1024, True, 0.0), (3, 5, 2, 8, 16, False, 0.0),
    (130, 1, 1, 72, 136, True, 0.0), (257, 1, 1, 64, 264, True, 0.0),
]


@pytest.mark.parametrize("T,E,k,C,H,bias,skew", MLPS)
def test_expert_mlp(T, E, k, C, H, bias, skew):
    v = _mlp_inputs(T, E, k, C, H, T + C, bias)
    ids = _ids(T, E, k, T + H, gone=0.1 if T > 2 else 0.0, skew=skew)
    cfg = L.make_expert_cfg(T, E, k, C=C, hidden=H)
    out = _mlp(cfg, v, ids)
    assert L.sparsesam_device_status() == L.SS_OK
    _check_mlp(v, ids, out)
    assert torch.equal(out, _mlp(cfg, v, ids))          # the same bits again
    for name in ("x",) + (("residual",) if bias else ()):    # in place
        w = {**v, name: v[name].clone()}
        _mlp(cfg, w, ids, out=w[name])
        assert torch.equal(w[name], out), name


def test_expert_mlp_strided_rows_and_no_weights():
    T, E, k, C, H = 90, 5, 2, 96, 160
    v = _mlp_inputs(T, E, k, C, H, 0)
    ids = _ids(T, E, k, 1)
    ones = {**v, "weight": torch.ones_like(v["weight"])}
    want = _mlp(L.make_expert_cfg(T, E, k, C=C, hidden=H), ones, ids)
    wide = torch.full((3, T, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[0, :, :C], wide[1, :, :C] = v["x"], v["residual"]
    cfg = L.make_expert_cfg(T, E, k, C=C, hidden=H, ld=128)
    _mlp(cfg, {**v, "x": wide[0], "residual": wide[1], "weight": None}, ids, out=wide[2])
    torch.cuda.synchronize()
    assert torch.equal(wide[2, :, :C], want) and (wide[:, :, C:] == 5.0).all()


@pytest.mark.parametrize("T", [3, 30, 70, 700])
def test_expert_mlp_nothing_routed(T):
    E, k, C, H = 4, 2, 64, 128
    v = _mlp_inputs(T, E, k, C, H, 2)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    v["weight"][:] = float("nan")
    assert torch.equal(_mlp(L.make_expert_cfg(T, E, k, C=C, hidden=H), v, ids), v["residual"])


@pytest.mark.parametrize("T", [4, 50])
def test_expert_mlp_bad_ids_count_as_none(T):
    E, k, C, H = 4, 2, 64, 128
    v = _mlp_inputs(T, E, k, C, H, 3)
    ids = _ids(T, E, k, 4)
    ids[T - 2, 0], ids[1, 1] = 99, -5
    out = _mlp(L.make_expert_cfg(T, E, k, C=C, hidden=H), v, ids)
    assert L.sparsesam_device_status() == L.SS_EINDEX
    _check_mlp(v, ids, out)


def test_expert_mlp_a_poisoned_token_stays_alone():
    """A token of infinities and NaN reaches no other token, not even in its own tile."""
    E, k, C, H = 2, 1, 64, 128
    for T in (8, 64, 100, 300):
        v = _mlp_inputs(T, E, k, C, H, 5)
        ids = _ids(T, E, k, 6, gone=0.0)
        cfg = L.make_expert_cfg(T, E, k, C=C, hidden=H)
        want = _mlp(cfg, v, ids)
        v["x"][5, 3], v["x"][5, 4] = float("inf"), float("nan")
        out = _mlp(cfg, v, ids)
        keep = [t for t in range(T) if t != 5]
        assert torch.equal(out[keep], want[keep]) and torch.isnan(out[5]).all()


def test_expert_mlp_the_same_expert_twice():
    """A token that names one expert twice gets it twice; more assignments than an expert has rows."""
    for T in (2, 90):
        E, k, C, H = 3, 3, 64, 128
        v = _mlp_inputs(T, E, k, C, H, 15)
        ids = torch.tensor([[1, 1, 1], [2, 0, 2]] * (T // 2), dtype=torch.int32, device="cuda")
        _check_mlp(v, ids, _mlp(L.make_expert_cfg(T, E, k, C=C, hidden=H), v, ids))


@pytest.mark.parametrize("T", [3, 200, 900])
def test_two_streams_and_a_captured_graph(T):
    """Two calls at once with a workspace each, and a captured one replayed with new inputs."""
    E, k, C, H = 8, 2, 128, 256
    cfg = L.make_expert_cfg(T, E, k, C=C, hidden=H)
    a, b = _mlp_inputs(T, E, k, C, H, 7), _mlp_inputs(T, E, k, C, H, 8)
    ia, ib = _ids(T, E, k, 9), _ids(T, E, k, 10)
    wa, wb = _mlp(cfg, a, ia), _mlp(cfg, b, ib)
    nb = L.sparsesam_expert_mlp_workspace(cfg)
    ws = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        _mlp(cfg, a, ia, out=oa, ws=ws[0], stream=s1)
        _mlp(cfg, b, ib, out=ob, ws=ws[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    graph = torch.cuda.CUDAGraph()
    x, ids = a["x"].clone(), ia.clone()
    with torch.cuda.graph(graph):
        _mlp(cfg, {**a, "x": x}, ids, out=oa, ws=ws[0], stream=torch.cuda.current_stream())
    for v, i in ((a, ia), (b, ib), (a, ia)):
        x.copy_(v["x"])
        ids.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, _mlp(cfg, {**a, "x": v["x"]}, i))


def test_a_block_of_routed_experts():
    """The calls as an encoder block uses them: the norm before, the router, the experts, and the norm
    after with gate, residual scale and residual, which also makes the next block's input."""
    B, T, E, k, C, H, eps = 2, 49, 6, 2, 128, 256, 1e-6
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    R = B * T
    y0, x0, gate, scale = r(R, C), r(R, C), r(B, C), r(C)
    pw, pb, qw, qb, wr = r(C), r(C), r(C), r(C), r(E, C)
    v = _mlp_inputs(R, E, k, C, H, 12)
    ncfg = L.make_norm_cfg(R, C, norm="layer", eps=eps, rows_per_gate=T)
    x1, n1, x2, n2 = (torch.empty_like(x0) for _ in range(4))
    L.sparsesam_norm_residual(L.make_norm_cfg(R, C, norm="layer", eps=eps), y0, x0, None, None,
                              None, None, qw, qb, x1, n1, None)
    logits = (n1.float() @ wr.float().T).contiguous()
    ids, weight = _route(logits, k, True)
    cfg = L.make_expert_cfg(R, E, k, C=C, hidden=H)
    moe = _mlp(cfg, {**v, "x": n1, "weight": weight, "residual": None}, ids)
    L.sparsesam_norm_residual(ncfg, moe, x1, gate, scale, pw, pb, qw, qb, x2, n2, None)
    torch.cuda.synchronize()
    # step by step from the library's own stored values, so that each tolerance is one call's
    w_ids, w_w = X.route(f64(logits), k, True)
    assert np.array_equal(ids.cpu().numpy(), w_ids)
    _check_mlp({**v, "x": n1, "weight": weight, "residual": None}, ids, moe)
    want = X.norm_residual(f64(moe), f64(x1), f64(gate), T, f64(scale), f64(pw), f64(pb), "layer", eps)
    assert (np.abs(f64(x2) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * (1 + np.abs(want - f64(x1)))).all()
    want = X.norm(f64(x2), f64(qw), f64(qb), "layer", eps)
    assert (np.abs(f64(n2) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * (1 + np.abs(want))).all()


def test_training_through_the_routed_rows():
    """Gradients of a linear expert layer through route, sort, gather and combine, fp32, against
    central differences in 64 bits: loss = sum(dout * combine(W_e x, weight(logits)))."""
    T, E, k, C = 24, 4, 2, 16
    rng = np.random.default_rng(13)
    lg, x = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal((T, C)).astype(np.float32)
    lg[5] = -np.inf
    W = rng.standard_normal((E, C, C)).astype(np.float32) / 4
    dout = rng.standard_normal((T, C)).astype(np.float32)
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    cfg = L.make_expert_cfg(T, E, k, C=C, dtype="f32")
    ids, w = _route(d(lg), k, False)
    order, slot, offsets = _sort(ids, E)
    xs = torch.zeros(T * k, C, device="cuda")
    L.sparsesam_expert_gather(cfg, d(x), slot, xs)
    seg = offsets.tolist()
    ys, dxs = torch.zeros_like(xs), torch.zeros_like(xs)
    for e in range(E):
        ys[seg[e]:seg[e + 1]] = (xs[seg[e]:seg[e + 1]].double() @ d(W[e]).double().T).float()
    dys, dw, dlg = torch.zeros_like(xs), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    L.sparsesam_expert_combine_backward(cfg, d(dout), ys, slot, w, dys, dw)
    for e in range(E):
        dxs[seg[e]:seg[e + 1]] = (dys[seg[e]:seg[e + 1]].double() @ d(W[e]).double()).float()
    dx = torch.empty(T, C, device="cuda")
    L.sparsesam_expert_combine(cfg, dxs, slot, None, None, dx)
    L.sparsesam_expert_route_backward(cfg, d(lg), False, ids, w, dw, dlg)

    def loss(lg64, x64):
        i, ww = X.route(lg64, k, False)
        out = np.zeros((T, C))
        for t in range(T):
            for j in range(k):
                if i[t, j] >= 0:
                    out[t] += ww[t, j] * (W[i[t, j]].astype(float) @ x64[t])
        return (out * dout).sum()

    lg64, x64, h = lg.astype(float), x.astype(float), 1e-6
    for got, which in ((dx, 1), (dlg, 0)):
        v = rng.standard_normal(got.shape)
        a = [lg64, x64]
        hi, lo = list(a), list(a)
        hi[which], lo[which] = a[which] + h * v, a[which] - h * v
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        mine = (f64(got) * v).sum()
        # fp32 throughout: a few hundred roundings of 2^-24 in sums of |terms| near 1e3; the
        # difference's own error is near 1e-7
        assert abs(mine - want) <= 1e-4 * max(1.0, np.abs(f64(got) * v).sum()), (mine, want)


def test_rows_past_32_bits():
    """More than 2^31 channels of sorted rows, and of logits."""
    T, k, C = 70000, 4, 8192
    n = T * k
    assert n * C > 1 << 31
    cfg = L.make_expert_cfg(T, 8, k, C=C)
    slot = torch.randperm(n, device="cuda", dtype=torch.int32).view(T, k)
    x = torch.randn(T, C, device="cuda", dtype=torch.bfloat16)
    xs = torch.full((n, C), 7.0, device="cuda", dtype=torch.bfloat16)
    L.sparsesam_expert_gather(cfg, x, slot, xs)
    for t0 in range(0, T, 10000):
        want = x[t0:t0 + 10000]
        for j in range(k):
            assert torch.equal(xs[slot[t0:t0 + 10000, j].long()], want)
    # k equal rows weighted 2^-2, 2^-1, 2^-3, 2^-3: their sum is the row, exactly
    w = torch.tensor([0.25, 0.5, 0.125, 0.125], device="cuda").expand(T, k).contiguous()
    out = torch.full_like(x, 7.0)
    L.sparsesam_expert_combine(cfg, xs, slot, w, None, out)
    assert torch.equal(out, x)
    dw = torch.full((T, k), 7.0, device="cuda")
    L.sparsesam_expert_combine_backward(cfg, x, xs, slot, w, xs, dw)
    for t0 in range(0, T, 10000):
        want = x[t0:t0 + 10000]
        for j in range(k):
            assert torch.equal(xs[slot[t0:t0 + 10000, j].long()], want * w[0, j].item())
        sq = (want.double() ** 2).sum(1, keepdim=True)      # all terms of the dot product are positive
        assert ((dw[t0:t0 + 10000] - sq).abs() <= (C / 32 + 8) * F * sq).all()
    del xs, x, out
    T, E = (1 << 22) + 300, 512
    assert T * E > 1 << 31
    lg = torch.zeros(T, E, device="cuda")
    hot = torch.randint(0, E, (T, 1), device="cuda")
    lg.scatter_(1, hot, 1.0)
    ids, weight = _route(lg, 1, 1)
    assert torch.equal(ids, hot.int()) and (weight == 1.0).all()
    dl = torch.full_like(lg, 7.0)
    L.sparsesam_expert_route_backward(L.make_expert_cfg(T, E, 1), lg, 1, ids, weight, weight, dl)
    assert not dl.any()
    assert L.sparsesam_device_status() == L.SS_OK


@pytest.mark.parametrize("T", [2, 30])
def test_expert_mlp_weights_past_32_bits(T):
    """Each weight tensor holds more than 2^31 values; the last experts work as in a call with them alone."""
    E, C, H = 512, 2048, 2056
    assert E * C * H > 1 << 31
    v = _mlp_inputs(T, 2, 1, C, H, 5)
    ids = torch.arange(T, device="cuda", dtype=torch.int32)[:, None] % 2
    big = dict(v)
    for name in ("w1", "w2"):
        big[name] = torch.zeros(E, *v[name].shape[1:], device="cuda", dtype=torch.bfloat16)
    for name in ("b1", "b2"):
        big[name] = torch.zeros(E, v[name].shape[1], device="cuda", dtype=torch.bfloat16)
    for name in ("w1", "w2", "b1", "b2"):
        big[name][-2:] = v[name]
    out = _mlp(L.make_expert_cfg(T, E, 1, C=C, hidden=H), big, ids + E - 2)
    assert L.sparsesam_device_status() == L.SS_OK
    _check_mlp(v, ids, out)

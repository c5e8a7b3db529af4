"""Float64 definitions of the norm and routed-expert calls (test infrastructure only; shares no code
with the library). Rows are numpy float64 arrays holding the values of the library's inputs."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erf

LAYER, RMS = "layer", "rms"


def norm_stats(v, kind, eps):
    """(mean, 1/sqrt) of each row, as columns."""
    mean = v.mean(1, keepdims=True) if kind == LAYER else np.zeros((v.shape[0], 1))
    var = ((v - mean) ** 2).mean(1, keepdims=True)
    return mean, 1.0 / np.sqrt(var + eps)


def norm(v, w, b, kind, eps):
    mean, rstd = norm_stats(v, kind, eps)
    out = (v - mean) * rstd * w
    return out if b is None else out + b


def gate_rows(gate, rows, per_gate):
    return 1.0 if gate is None else gate[np.arange(rows) // per_gate]


def norm_residual(y, x, gate, per_gate, scale, post_w, post_b, kind, eps):
    """x_out, unrounded."""
    p = y if post_w is None else norm(y, post_w, post_b, kind, eps)
    return x + gate_rows(gate, len(y), per_gate) * (1.0 if scale is None else scale) * p


def _norm_grad(g, h, rstd, kind):
    """Input gradient of h = (v - mean) rstd for the gradient g of h."""
    out = g - h * (g * h).mean(1, keepdims=True)
    if kind == LAYER:
        out = out - g.mean(1, keepdims=True)
    return rstd * out


def norm_residual_backward(y, x_out, gate, per_gate, scale, post_w, post_b, pre_w, kind, eps,
                           dx_out, dn):
    """Gradients by name (dx, dy, dgate, dscale, dpost_w, dpost_b, dpre_w, dpre_b; those of absent
    parameters left out), with x_out the forward's stored result."""
    out = {}
    D = dx_out
    if pre_w is not None:
        mean, rstd = norm_stats(x_out, kind, eps)
        h = (x_out - mean) * rstd
        out["dpre_w"], out["dpre_b"] = (dn * h).sum(0), dn.sum(0)
        D = D + _norm_grad(dn * pre_w, h, rstd, kind)
    out["dx"] = D
    G = gate_rows(gate, len(y), per_gate)
    S = 1.0 if scale is None else scale
    h, p = y, y
    if post_w is not None:
        mean, rstd = norm_stats(y, kind, eps)
        h = (y - mean) * rstd
        p = h * post_w + (0.0 if post_b is None else post_b)
    if gate is not None:
        out["dgate"] = np.zeros_like(gate)
        np.add.at(out["dgate"], np.arange(len(y)) // per_gate, D * S * p)
    if scale is not None:
        out["dscale"] = (D * G * p).sum(0)
    q = D * G * S
    if post_w is not None:
        out["dpost_w"], out["dpost_b"] = (q * h).sum(0), q.sum(0)
        q = _norm_grad(q * post_w, h, rstd, kind)
    out["dy"] = q
    return out


def route(logits, topk, renorm):
    """ids (int32, -1: none) and weights of each token, one token at a time."""
    T, E = logits.shape
    ids = np.full((T, topk), -1, np.int32)
    weight = np.zeros((T, topk))
    for t in range(T):
        open_ = [e for e in range(E) if logits[t, e] > -np.inf]
        chosen = sorted(open_, key=lambda e: (-logits[t, e], e))[:topk]
        if not chosen:
            continue
        top = logits[t, chosen[0]]
        total = sum(math.exp(logits[t, e] - top) for e in (chosen if renorm else open_))
        for j, e in enumerate(chosen):
            ids[t, j] = e
            weight[t, j] = math.exp(logits[t, e] - top) / total
    return ids, weight


def route_backward(logits, topk, renorm, dweight):
    """dlogits by the softmax's Jacobian, one token at a time."""
    T, E = logits.shape
    ids, weight = route(logits, topk, renorm)
    out = np.zeros((T, E))
    for t in range(T):
        live = [j for j in range(topk) if ids[t, j] >= 0]
        if not live:
            continue
        support = ([ids[t, j] for j in live] if renorm
                   else [e for e in range(E) if logits[t, e] > -np.inf])
        z = np.array([logits[t, e] for e in support])
        p = np.exp(z - z.max())
        p /= p.sum()
        jac = np.diag(p) - np.outer(p, p)
        at = {e: i for i, e in enumerate(support)}
        for j in live:
            out[t, support] += dweight[t, j] * jac[at[ids[t, j]]]
    return out


def expert_sort(ids, E):
    """order, slot, offsets; ids outside [0, E) are routed nowhere."""
    flat = ids.reshape(-1)
    order = [a for e in range(E) for a in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    slot = np.full(flat.size, -1, np.int32)
    slot[order] = np.arange(len(order))
    full = np.full(flat.size, -1, np.int32)
    full[:len(order)] = order
    return full, slot.reshape(ids.shape), offsets.astype(np.int32)


def combine(ys, slot, weight, residual):
    T, k = slot.shape
    out = np.zeros((T, ys.shape[1])) if residual is None else residual.copy()
    for j in range(k):
        live = slot[:, j] >= 0
        w = 1.0 if weight is None else weight[live, j][:, None]
        out[live] += w * ys[slot[live, j]]
    return out


def combine_backward(dout, ys, slot, weight):
    """dys (rows at no slot: NaN) and dweight."""
    dys = np.full_like(ys, np.nan)
    dweight = np.zeros(slot.shape)
    for j in range(slot.shape[1]):
        live = slot[:, j] >= 0
        dys[slot[live, j]] = weight[live, j][:, None] * dout[live]
        dweight[live, j] = (dout[live] * ys[slot[live, j]]).sum(1)
    return dys, dweight


def gelu(z):
    return 0.5 * z * (1.0 + erf(z / math.sqrt(2.0)))


def expert_mlp(x, ids, weight, residual, w1, b1, w2, b2):
    """(out, bound): the result, and for every element what the library's roundings can add up to:
    the hidden rows and the experts' rows rounded to bf16 (2^-8 of each value), products in fp32
    (K 2^-24 of the sum of magnitudes) and the GELU's 1.5e-7."""
    u, f = 2.0 ** -8, 2.0 ** -24
    E, H, C = w1.shape
    out = np.zeros_like(x) if residual is None else residual.copy()
    bound = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if e < 0 or e >= E:
                continue
            w = 1.0 if weight is None else weight[t, j]
            z = w1[e] @ x[t] + (0.0 if b1 is None else b1[e])
            h = gelu(z)
            y = w2[e] @ h + (0.0 if b2 is None else b2[e])
            z_off = (C + 2) * f * (np.abs(w1[e]) @ np.abs(x[t]) + (0 if b1 is None else np.abs(b1[e])))
            h_off = u * np.abs(h) + 1.2 * z_off + 3e-7 * np.abs(z)
            y_off = (np.abs(w2[e]) @ h_off + (H + 2) * f * (np.abs(w2[e]) @ np.abs(h))
                     + f * np.abs(y))
            out[t] += w * y
            bound[t] += abs(w) * (y_off * (1 + u) + u * np.abs(y))
    return out, bound * (1 + u) + u * np.abs(out)

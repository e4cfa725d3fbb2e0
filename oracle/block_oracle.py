"""What surrounds an MoE block's experts, in fp64: the norms, gate and residual
between two blocks, the training losses of a router and the gradients of both,
and the ends of the FP8 products."""
from __future__ import annotations

import math

import numpy as np

from .bq_oracle import softplus


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(x):
    x = _f64(x)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def _inverse_rms(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + float(eps))


def _gate(gate, use_sigmoid):
    if gate is None:
        return 1.0
    return sigmoid(gate) if use_sigmoid else _f64(gate)


def residual_norm(y, h, gain, post_gain=None, gate=None, use_sigmoid=False, scale=1.0, residual_scale=1.0, eps=1e-6):
    """``h' = residual_scale h + scale g b``, ``b = post_gain n(y)`` (or y), ``x = gain n(h')``.

    y, h: [T, H]; gate: anything that broadcasts to [T, H], or None.  Returns (h', x)."""
    y, h = _f64(y), _f64(h)
    b = y if post_gain is None else _f64(post_gain) * y * _inverse_rms(y, eps)
    out = residual_scale * h + scale * _gate(gate, use_sigmoid) * b
    x = None if gain is None else _f64(gain) * out * _inverse_rms(out, eps)
    return out, x


def _norm_gradient(v, gain, d, eps):
    """Gradients of gain * n(v) with respect to v and, summed over rows, gain."""
    r = _inverse_rms(v, eps)
    dg = d * gain
    return r * dg - v * r ** 3 * np.mean(dg * v, axis=-1, keepdims=True), np.sum(d * v * r, axis=0)


def residual_norm_backward(y, h_out, dh_out, dx, gain, post_gain=None, gate=None, use_sigmoid=False, scale=1.0,
                           residual_scale=1.0, eps=1e-6):
    """Gradients of residual_norm: dict of dy, dh, dgain, dpost_gain and dgate (in the gate's shape).
    dh_out or dx may be None (zero)."""
    y, h_out = _f64(y), _f64(h_out)
    g_out = np.zeros_like(y) if dh_out is None else _f64(dh_out).copy()
    found = {"dgain": None, "dpost_gain": None, "dgate": None}
    if dx is not None:
        dh, found["dgain"] = _norm_gradient(h_out, _f64(gain), _f64(dx), eps)
        g_out = g_out + dh
    found["dh"] = residual_scale * g_out
    d, g = scale * g_out, _gate(gate, use_sigmoid)
    b = y if post_gain is None else _f64(post_gain) * y * _inverse_rms(y, eps)
    if gate is not None:
        dgate = d * b * (g * (1 - g) if use_sigmoid else 1.0)
        shape = (1,) * (2 - np.ndim(gate)) + np.shape(gate)
        for axis in range(2):
            if shape[axis] == 1:
                dgate = dgate.sum(axis=axis, keepdims=True)
        found["dgate"] = dgate.reshape(np.shape(gate))
    db = d * g
    if post_gain is None:
        found["dy"] = db
    else:
        found["dy"], found["dpost_gain"] = _norm_gradient(y, _f64(post_gain), db, eps)
    return found


# --------------------------------------------------------------------------
# Router training
# --------------------------------------------------------------------------

def _ranges(t, offsets):
    o = [0, t] if offsets is None else [int(v) for v in offsets]
    return list(zip(o[:-1], o[1:]))


def router_logits(logits, bias=None):
    """``logits + bias`` in fp32, as the router adds them."""
    z = np.asarray(logits, dtype=np.float32)
    return _f64(z if bias is None else z + np.asarray(bias, dtype=np.float32)[None, :])


def router_softmax(z):
    """Softmax and log-sum-exp of each row; a row of -inf only: zeros."""
    with np.errstate(invalid="ignore"):
        top = z.max(axis=1, keepdims=True)
        dead = top == -np.inf
        e = np.exp(z - np.where(dead, 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        lse = np.where(dead, 0.0, top + np.log(np.where(dead, 1.0, total)))
    return e / np.where(dead, 1.0, total), lse


def router_scores(z):
    """``s = sqrt(softplus(z))`` and ``ds/dz = sigmoid(z) / (2 s)`` (exp(z/2) / 2 far below 0)."""
    far = z < -40
    near = np.where(far, 0.0, z)
    s = np.where(far, np.exp(0.5 * z), np.sqrt(softplus(near)))
    slope = np.where(far, 0.5 * np.exp(0.5 * z), 0.5 * sigmoid(near) / np.sqrt(softplus(near)))
    return s, slope


def router_shares(z):
    """``s / sum s`` and ``ds/dz / sum s`` of each row.  A row far below 0, where s is exp(z/2): without the factor
    exp(max z / 2), which cancels (and is 0 in fp64 below -1490)."""
    top = z.max(axis=1, keepdims=True)
    far = (top < -80) & (top > -np.inf)
    shifted = np.exp(0.5 * np.where(far, z - np.where(far, top, 0.0), 0.0))
    s, slope = router_scores(np.where(far, 0.0, z))
    s, slope = np.where(far, shifted, s), np.where(far, 0.5 * shifted, slope)
    whole = s.sum(axis=1, keepdims=True)
    whole = np.where(whole == 0, 1.0, whole)
    return s / whole, slope / whole


def router_probabilities(z, scoring):
    return router_softmax(z)[0] if scoring != "sqrtsoftplus" else router_shares(z)[0]


def balance_loss(logits, ids, scoring="softmax", bias=None, offsets=None):
    """(counts [S, E], mean probabilities [S, E], (balance loss, z-loss)) of a router's rows."""
    z = router_logits(logits, bias)
    t, e = z.shape
    k = np.shape(ids)[1]
    p, lse = router_probabilities(z, scoring), router_softmax(z)[1]
    ranges = _ranges(t, offsets)
    counts, probs = np.zeros((len(ranges), e), dtype=np.int64), np.zeros((len(ranges), e))
    per_sequence, square, rows = [], 0.0, 0
    for s, (a, b) in enumerate(ranges):
        if a == b:
            continue
        chosen = np.asarray(ids)[a:b].reshape(-1)
        counts[s] = np.bincount(chosen[(chosen >= 0) & (chosen < e)], minlength=e)
        probs[s] = p[a:b].mean(axis=0)
        per_sequence.append(float((e * counts[s] / (k * (b - a)) * probs[s]).sum()))
        square += float((lse[a:b] ** 2).sum())
        rows += b - a
    return counts, probs, (sum(per_sequence) / max(1, len(per_sequence)), square / max(1, rows))


def route_weights(logits, ids, scoring="softmax", bias=None, scale=1.0):
    """The router's weights [T, k] of given ids."""
    z = router_logits(logits, bias)
    zs = np.take_along_axis(z, np.asarray(ids, dtype=np.int64), axis=1)
    if scoring == "sqrtsoftplus":
        return scale * router_scores(zs)[0]
    ex = np.exp(zs - zs.max(axis=1, keepdims=True))
    return ex / ex.sum(axis=1, keepdims=True)


def route_backward(logits, ids, dweights, scoring="softmax", bias=None, scale=1.0, counts=None, dlosses=None,
                   offsets=None):
    """Gradient of <dweights, route_weights> + <dlosses, losses> with respect to the logits, [T, E]; NaN in
    rows of no sequence (not written)."""
    z = router_logits(logits, bias)
    t, e = z.shape
    ids = np.asarray(ids)
    k = ids.shape[1]
    d = np.zeros((t, e))
    soft, lse = router_softmax(z)
    slope, share = (router_scores(z)[1], router_shares(z)[1]) if scoring == "sqrtsoftplus" else (None, None)
    if dweights is not None:
        for r in range(t):
            on = [j for j in range(k) if 0 <= ids[r, j] < e]
            at = ids[r, on].astype(np.int64)
            dw = _f64(dweights)[r, on]
            if scoring == "sqrtsoftplus":
                g = scale * dw * slope[r, at]
            elif on and z[r, at].max() > -np.inf:
                ex = np.exp(z[r, at] - z[r, at].max())
                w = ex / ex.sum()
                g = w * (dw - (w * dw).sum())
            else:              # none, or all of them -inf: no gradient
                continue
            np.add.at(d[r], at, g)
    ranges = _ranges(t, offsets)
    if dlosses is not None:
        p = router_probabilities(z, scoring)
        used, rows = sum(b > a for a, b in ranges), sum(b - a for a, b in ranges)
        for s, (a, b) in enumerate(ranges):
            if a == b:
                continue
            weight = float(dlosses[0]) * e * _f64(counts)[s] / (k * (b - a)) / (b - a) / used
            inner = weight[None, :] - (p[a:b] * weight).sum(axis=1, keepdims=True)
            if scoring == "sqrtsoftplus":
                d[a:b] += share[a:b] * inner
            else:
                d[a:b] += p[a:b] * inner
            d[a:b] += 2 * float(dlosses[1]) / rows * lse[a:b] * soft[a:b]
    written = np.zeros(t, dtype=bool)
    for a, b in ranges:
        written[a:b] = True
    d[~written] = np.nan
    return d


# --------------------------------------------------------------------------
# The end of a product
# --------------------------------------------------------------------------

def activation(v, act):
    """none, silu, gelu (with erf), gelu_tanh, relu, relu2, or swiglu (halves of the last axis: gate, up)."""
    v = _f64(v)
    if act == "swiglu":
        gate, up = np.split(v, 2, axis=-1)
        return gate * sigmoid(gate) * up
    if act == "silu":
        return v * sigmoid(v)
    if act == "gelu":
        return 0.5 * v * np.vectorize(math.erfc)(-v * math.sqrt(0.5)) if v.size else v
    if act == "gelu_tanh":
        return v * sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "relu":
        return np.maximum(v, 0)
    if act == "relu2":
        return np.maximum(v, 0) ** 2
    if act == "none":
        return v
    raise ValueError(act)


def product_end(v, bias=None, act="none", scale=1.0, residual=None):
    """``scale * act(v + bias) + residual``; bias [n] or one row per row of v."""
    v = _f64(v) + (0.0 if bias is None else _f64(bias))
    v = scale * activation(v, act)
    return v if residual is None else v + _f64(residual)

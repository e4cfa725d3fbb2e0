"""Pins of the oracle's block-to-block, router-training and product-end functions (CPU): gradients
against central differences in fp64, closed forms, and rows that hold nothing."""
import numpy as np
import pytest

import oracle as O


def difference(f, x, d, step=1e-6):
    """Directional derivative of f at x along d."""
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


GATES = {"none": None, "token": (5, 1), "channel": (24,), "full": (5, 24)}


@pytest.mark.parametrize("kind", list(GATES))
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_gradients_against_differences(kind, sig, post):
    g = np.random.default_rng(3)
    t, h = 5, 24
    y, r, gain = g.standard_normal((t, h)), g.standard_normal((t, h)), g.uniform(0.5, 1.5, h)
    pg = g.uniform(0.5, 1.5, h) if post else None
    gate = None if GATES[kind] is None else g.standard_normal(GATES[kind])
    dh, dx = g.standard_normal((t, h)), g.standard_normal((t, h))
    more = dict(use_sigmoid=sig, scale=0.7, residual_scale=1.3, eps=1e-3)

    def loss(y=y, r=r, gain=gain, pg=pg, gate=gate):
        out, x = O.residual_norm(y, r, gain, pg, gate, **more)
        return (out * dh).sum() + (x * dx).sum()

    out, _ = O.residual_norm(y, r, gain, pg, gate, **more)
    found = O.residual_norm_backward(y, out, dh, dx, gain, pg, gate, **more)
    for name, key, at in (("y", "dy", y), ("r", "dh", r), ("gain", "dgain", gain), ("pg", "dpost_gain", pg),
                          ("gate", "dgate", gate)):
        if at is None:
            assert found[key] is None
            continue
        d = g.standard_normal(at.shape)
        assert difference(lambda v: loss(**{name: v}), at, d) == pytest.approx((found[key] * d).sum(), rel=1e-6, abs=1e-7)


def test_residual_norm_against_hand_values():
    out, x = O.residual_norm([[3.0, 4.0]], [[1.0, -1.0]], [2.0, 1.0], eps=0.0)
    np.testing.assert_allclose(out, [[4.0, 3.0]])
    np.testing.assert_allclose(x, [[8.0 / np.sqrt(12.5), 3.0 / np.sqrt(12.5)]])
    out, _ = O.residual_norm([[3.0, 4.0]], [[1.0, 0.0]], None, post_gain=[1.0, 2.0], gate=[[0.0]], use_sigmoid=True,
                             scale=2.0, residual_scale=0.5, eps=0.0)
    np.testing.assert_allclose(out, [[0.5 + 3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])


SCORINGS = ["softmax", "softmax_then_bias", "sqrtsoftplus"]


@pytest.mark.parametrize("scoring", SCORINGS)
@pytest.mark.parametrize("offsets", [None, [0, 4, 4, 9, 11], [1, 6, 12]])
def test_router_gradients_against_differences(scoring, offsets):
    g = np.random.default_rng(7)
    t, e, k = 12, 10, 3
    logits = g.standard_normal((t, e)).astype(np.float32).astype(np.float64) * 2
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32)
    dw, dl = g.standard_normal((t, k)), (1.7, 0.6)
    counts, _, _ = O.balance_loss(logits, ids, scoring, offsets=offsets)
    d = O.route_backward(logits, ids, dw, scoring, scale=2.5, counts=counts, dlosses=dl, offsets=offsets)
    inside = ~np.isnan(d[:, 0])
    lo, hi = (0, t) if offsets is None else (offsets[0], offsets[-1])
    assert inside.tolist() == [lo <= r < hi for r in range(t)]

    # differences need the logits in fp64: the oracle's own parts, without its fp32 add
    def total(z):
        p, lse = O.router_probabilities(z, scoring), O.router_softmax(z)[1]
        zs = np.take_along_axis(z, ids.astype(np.int64), axis=1)
        if scoring == "sqrtsoftplus":
            w = 2.5 * O.router_scores(zs)[0]
        else:
            w = np.exp(zs) / np.exp(zs).sum(axis=1, keepdims=True)
        o = [0, t] if offsets is None else offsets
        parts = [e * (counts[s] / (k * (b - a)) * p[a:b].mean(axis=0)).sum() for s, (a, b) in enumerate(zip(o[:-1], o[1:]))
                 if b > a]
        return (w * dw)[lo:hi].sum() + dl[0] * np.mean(parts) + dl[1] * np.mean(lse[lo:hi] ** 2)

    for _ in range(5):
        way = g.standard_normal((t, e))
        assert difference(total, logits, way) == pytest.approx((d[inside] * way[inside]).sum(), rel=1e-6, abs=1e-8)


@pytest.mark.parametrize("scoring", SCORINGS)
def test_an_even_load_has_balance_loss_one(scoring):
    t, e, k = 8, 8, 2
    ids = np.array([[i % e, (i + 1) % e] for i in range(t)], dtype=np.int32)
    counts, probs, (balance, z) = O.balance_loss(np.zeros((t, e)), ids, scoring)
    assert counts.tolist() == [[2] * e] and balance == pytest.approx(1.0)
    np.testing.assert_allclose(probs, 1 / e)
    assert z == pytest.approx(np.log(e) ** 2)


def test_rows_of_nothing_and_bad_ids():
    logits = np.zeros((3, 4), dtype=np.float32)
    logits[1] = -np.inf
    logits[2, :2] = -np.inf
    for scoring in SCORINGS:
        counts, probs, losses = O.balance_loss(logits, np.array([[0], [9], [-1]], dtype=np.int32), scoring)
        assert counts.tolist() == [[1, 0, 0, 0]] and np.isfinite(probs).all() and np.isfinite(losses).all()
        d = O.route_backward(logits, np.array([[0], [9], [3]], dtype=np.int32), np.ones((3, 1)), scoring, counts=counts,
                             dlosses=(1.0, 1.0))
        assert np.isfinite(d).all() and not d[1].any() and not d[2, :2].any()


@pytest.mark.parametrize("z", [-1e30, -700.0, -41.0, -39.0, -1.0, 0.0, 3.0, 80.0])
def test_score_and_slope_against_differences(z):
    s, slope = O.router_scores(np.array([z]))
    if z < -600:
        assert s[0] == pytest.approx(np.exp(z / 2)) and slope[0] == s[0] / 2
    else:
        step = 1e-5
        both = O.router_scores(np.array([z - step, z + step]))[0]
        assert slope[0] == pytest.approx((both[1] - both[0]) / (2 * step), rel=1e-6)


@pytest.mark.parametrize("act,at,value", [
    ("silu", 1.0, 1 / (1 + np.exp(-1))), ("gelu", 1.0, 0.8413447460685429), ("gelu", -40.0, 0.0), ("gelu", 0.0, 0.0),
    ("gelu_tanh", 1.0, 0.8411919906082768), ("relu", -2.0, 0.0), ("relu2", 3.0, 9.0), ("none", -2.0, -2.0)])
def test_activations(act, at, value):
    assert O.activation(np.array([at]), act)[0] == pytest.approx(value, abs=1e-15)


def test_product_end_order():
    v = O.product_end(np.array([[1.0, -3.0]]), bias=[1.0, 1.0], act="relu2", scale=0.5, residual=[[10.0, 20.0]])
    assert v.tolist() == [[12.0, 20.0]]
    assert O.product_end(np.array([[0.0, 2.0]]), act="swiglu").tolist() == [[0.0]]

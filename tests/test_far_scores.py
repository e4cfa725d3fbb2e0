"""Score routing of rows whose logits are all far below 0: the scores leave fp32's range (and fp64's), their shares of
the row's sum do not.

Tolerances as in the other tests of a router's training (u = 2^-24): P = (2 D + 160) u for a share, with D the largest
|z| of the row, or |z - max z| where the largest logit is below -20 and exp(max z / 2) is left out of the shares (z - max z
is exact to u |z - max z|; beyond 200 a share is below fp32's normal range, and may be 0)."""
import numpy as np
import pytest

import oracle as O

U = 2.0 ** -24
SUB = 2.0 ** -126
LOWEST = -float(np.finfo(np.float32).max)


@pytest.mark.parametrize("shift", [-85.0, -200.0, -1400.0, -1e4, -1e30])
def test_oracle_shares_are_those_of_half_the_logits(shift):
    g = np.random.default_rng(1)
    z = 3 * g.standard_normal((5, 12)) + shift
    share, slope = O.router_shares(z)
    np.testing.assert_allclose(share, O.router_softmax(z / 2)[0], rtol=1e-13)
    np.testing.assert_allclose(slope, share / 2, rtol=1e-13)
    assert O.router_probabilities(z, "sqrtsoftplus").sum(axis=1) == pytest.approx(1)


def test_oracle_shares_agree_where_both_forms_hold():
    z = 3 * np.random.default_rng(2).standard_normal((20, 12)) - np.linspace(70, 95, 20)[:, None]
    s, d = O.router_scores(z)
    share, slope = O.router_shares(z)
    np.testing.assert_allclose(share, s / s.sum(axis=1, keepdims=True), rtol=1e-12)
    np.testing.assert_allclose(slope, d / s.sum(axis=1, keepdims=True), rtol=1e-12)


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


SHIFTS = [0.0, -15.0, -19.0, -21.0, -60.0, -85.0, -170.0, -176.0, -200.0, -600.0, -1e4, -1e6]


def made(kind, t, e, k):
    g = np.random.default_rng(e)
    logits = 2 * g.standard_normal((t, e)) + 0.5 * g.standard_normal(e)
    if kind == "shifted":
        logits += np.resize(SHIFTS, t)[:, None]
    else:                                                  # masks of the type's lowest value, alone and beside others
        logits[:] = LOWEST
        logits[1::3] = -1e5 + g.standard_normal((len(logits[1::3]), e))
        logits[1::3, e // 2:] = LOWEST
        logits[2::3, e // 2:] = -np.inf
    logits = logits.astype(np.float32)
    return g, logits, np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32).copy()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["shifted", "lowest"])
@pytest.mark.parametrize("t,e,k,s", [(40, 8, 3, 0), (40, 48, 4, 3), (500, 128, 8, 5), (300, 256, 6, 0), (60, 700, 8, 2),
                                     (300, 1024, 8, 3)])
def test_statistics_and_gradients(lib, kind, t, e, k, s):
    import torch
    rule = lib.SCORE_SQRTSOFTPLUS
    g, logits, ids = made(kind, t, e, k)
    offsets = np.sort(g.integers(0, t + 1, s + 1)).astype(np.int32) if s else None
    z = O.router_logits(logits)
    top = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        far = np.where(np.isfinite(z), np.abs(np.where(top < -20, z - top, z)), 0.0)
    P = (2 * np.minimum(far, 200).max(axis=1, keepdims=True) + 160) * U

    n = max(1, s)
    counts, probs = torch.empty(n, e, dtype=torch.int32, device="cuda"), torch.empty(n, e, device="cuda")
    losses = torch.empty(2, device="cuda")
    lib.moe_balance_loss(dev(logits), dev(ids), counts, probs, losses,
                         torch.empty(lib.moe_balance_workspace_bytes(t, e, n), dtype=torch.uint8, device="cuda"), scoring=rule,
                         seq_offsets=None if s == 0 else dev(offsets))
    with np.errstate(over="ignore"):
        want_c, want_p, want_l = O.balance_loss(logits, ids, "sqrtsoftplus", offsets=offsets)
    np.testing.assert_array_equal(counts.cpu().numpy(), want_c)
    assert (np.abs(f64(probs) - want_p) <= (P.max() + 128 * U) * want_p + SUB).all()
    assert abs(float(losses[0]) - want_l[0]) <= (P.max() + 400 * U) * want_l[0]
    if not s:
        assert abs(float(probs.sum()) - 1) < 1e-4          # no row is lost

    dw = g.standard_normal((t, k)).astype(np.float32)
    dl = np.array([20.0, -3.0 if kind == "shifted" else 0.0], dtype=np.float32)
    d = torch.full((t, e), 7.0, device="cuda")
    lib.moe_route_backward(dev(logits), dev(ids), dev(dw), d, scoring=rule, scale=2.5, counts=counts, dlosses=dev(dl),
                           seq_offsets=None if s == 0 else dev(offsets))
    want = O.route_backward(logits, ids, dw, "sqrtsoftplus", scale=2.5, counts=want_c, dlosses=dl, offsets=offsets)
    at = ids.astype(np.int64)
    size = np.zeros((t, e))
    per = 2.5 * np.abs(dw) * O.router_scores(np.take_along_axis(z, at, axis=1))[1]
    for j in range(k):
        np.add.at(size, (np.arange(t), at[:, j]), per[:, j])
    own = (2 * np.minimum(np.where(np.isfinite(z), np.abs(z), 0.0), 200).max(axis=1, keepdims=True) + 160) * U
    bound = 4 * own * size                                 # the router's weights have no sum to be shares of
    (p, slope), (soft, lse) = O.router_shares(z), O.router_softmax(z)
    ranges = [(0, t)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
    used, rows = sum(b > a for a, b in ranges), sum(int(b - a) for a, b in ranges)
    for i, (a, b) in enumerate(ranges):
        if a < b:
            weight = 20.0 * e * want_c[i] / (k * (b - a) ** 2.0 * used)
            bound[a:b] += 4 * P[a:b] * slope[a:b] * (weight + (p[a:b] * weight).sum(axis=1, keepdims=True))
            wide = (2 * np.abs(np.where(np.isfinite(z[a:b]), z[a:b], 0.0)).max(axis=1, keepdims=True) + 160) * U
            bound[a:b] += 2 * abs(float(dl[1])) / rows * soft[a:b] * (4 * P[a:b] * np.abs(lse[a:b]) + wide)
    outside = np.isnan(want)
    got = f64(d)
    assert (got[outside] == 7.0).all()
    off = np.abs(got - np.where(outside, 7.0, want))
    assert (off <= 1.001 * bound + U * np.abs(np.where(outside, 0.0, want)) + 4 * SUB).all()
    if kind == "lowest":
        inside = ~outside[:, 0]
        assert not got[inside & (np.arange(t) % 3 == 2)][:, e // 2:].any()
    assert lib.device_status() == lib.DEV_OK

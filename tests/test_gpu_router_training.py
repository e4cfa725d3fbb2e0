"""GPU parity of the balance statistics and of the router's gradient against the fp64 oracle.

Tolerances (u = 2^-24).  z - m is off by u |z - m| and expf by 2 u, so a
probability is off by P = (2 max|z| + 160) u of itself: 32 additions in a lane,
the butterfly, the division; a score (log1pf, expf, sqrtf) by no more.  A mean
adds at most 64 rows in a warp, 16 warps, and 512 / 16 slots: 128 u more, and
the balance loss as much again over the experts (all terms positive).  A
log-sum-exp is off by L = (2 max|z| + 160) u, its mean square by
2 |lse| L + 256 u lse^2.  Gradients, with |.| sums of magnitudes: router weights
4 P w (|dw| + sum w |dw|) or 4 P scale |dw| s'; balance 4 P p (|a| + sum p |a|)
(s' / sum s in p's place); z-loss per_row p (4 P |lse| + L); and the output's
half step.  A bias gradient sums those bounds and 256 u of the magnitudes."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}   # expf may flush results below the normal range
RULES = ["softmax", "softmax_then_bias", "sqrtsoftplus"]


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def ragged(g, t, s):
    """Offsets of s sequences, some empty, that leave rows before and behind them."""
    o = np.sort(g.integers(0, t + 1, s + 1)).astype(np.int32)
    if s > 3:
        o[2] = o[1]
    return o


def inputs(g, t, e, k, spread=2.0):
    logits = (spread * g.standard_normal((t, e)) + 0.5 * g.standard_normal(e)).astype(np.float32)
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32).copy()
    return logits, ids, (0.3 * g.standard_normal(e)).astype(np.float32)


def balance(lib, logits, ids, rule, bias=None, offsets=None):
    import torch
    t, e = logits.shape
    s = 1 if offsets is None else len(offsets) - 1
    counts = torch.full((s, e), -7, dtype=torch.int32, device="cuda")
    probs, losses = torch.full((s, e), np.nan, device="cuda"), torch.full((2,), np.nan, device="cuda")
    ws = torch.full((lib.moe_balance_workspace_bytes(t, e, s),), 255, dtype=torch.uint8, device="cuda")
    lib.moe_balance_loss(dev(logits), dev(ids), counts, probs, losses, ws, bias=None if bias is None else dev(bias),
                         scoring=lib.SCORING_BY_NAME[rule], seq_offsets=None if offsets is None else dev(offsets))
    return counts, probs, losses


def part(z):
    """P and L of the tolerances, per row."""
    m = np.max(np.abs(np.where(np.isfinite(z), z, 0.0)), axis=1, keepdims=True)
    return (2 * m + 160) * U


def check_balance(lib, logits, ids, rule, bias=None, offsets=None):
    counts, probs, losses = balance(lib, logits, ids, rule, bias, offsets)
    want_c, want_p, want_l = O.balance_loss(logits, ids, rule, bias, offsets)
    z = O.router_logits(logits, bias)
    worst = part(z).max()
    np.testing.assert_array_equal(counts.cpu().numpy(), want_c)
    assert (np.abs(f64(probs) - want_p) <= (worst + 128 * U) * want_p + SUB["f32"]).all()
    lse = np.abs(O.router_softmax(z)[1]).max()
    got = f64(losses)
    assert abs(got[0] - want_l[0]) <= (worst + 400 * U) * want_l[0]
    assert abs(got[1] - want_l[1]) <= 2 * lse * worst + 256 * U * want_l[1]
    return want_c


def check_gradient(lib, g, logits, ids, rule, bias, offsets, counts, weights=True, losses=True, out="f32"):
    import torch
    t, e = logits.shape
    k = ids.shape[1]
    dw = g.standard_normal((t, k)).astype(np.float32) if weights else None
    dl = np.array([20.0, -3.0], dtype=np.float32) if losses else None
    d = torch.full((t, e), 7.0, dtype=torch_dtype(out), device="cuda")
    db = torch.full((e,), np.nan, device="cuda") if rule == "softmax" else None
    ws = torch.full((lib.moe_route_backward_workspace_bytes(t, e),), 255, dtype=torch.uint8, device="cuda")
    scale = 2.5 if rule == "sqrtsoftplus" else 1.0
    lib.moe_route_backward(dev(logits), dev(ids), None if dw is None else dev(dw), d,
                           bias=None if bias is None else dev(bias), scoring=lib.SCORING_BY_NAME[rule], scale=scale,
                           counts=dev(counts.astype(np.int32)) if losses else None, dlosses=None if dl is None else dev(dl),
                           seq_offsets=None if offsets is None else dev(offsets), dbias=db, workspace=ws)
    want = O.route_backward(logits, ids, dw, rule, bias, scale, counts, dl, offsets)
    z = O.router_logits(logits, bias)
    size = np.zeros((t, e))
    at = ids.astype(np.int64)
    if weights:
        zs = np.take_along_axis(z, at, axis=1)
        if rule == "sqrtsoftplus":
            per = scale * np.abs(dw) * O.router_scores(zs)[1]
        else:
            w = O.route_weights(logits, ids, rule, bias)
            per = w * (np.abs(dw) + (w * np.abs(dw)).sum(axis=1, keepdims=True))
        for j in range(k):
            np.add.at(size, (np.arange(t), at[:, j]), per[:, j])
    bound = 4 * part(z) * size
    if losses:
        p, (soft, lse) = O.router_probabilities(z, rule), O.router_softmax(z)
        ranges = [(0, t)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
        used, rows = sum(b > a for a, b in ranges), sum(int(b - a) for a, b in ranges)
        for s, (a, b) in enumerate(ranges):
            if a == b:
                continue
            weight = 20.0 * e * counts[s] / (k * (b - a) ** 2.0 * used)
            before = p[a:b]
            if rule == "sqrtsoftplus":
                score, slope = O.router_scores(z[a:b])
                before = slope / score.sum(axis=1, keepdims=True)
            here = before * (weight + (p[a:b] * weight).sum(axis=1, keepdims=True))
            there = 2 * 3.0 / rows * soft[a:b]
            size[a:b] += here + there * np.abs(lse[a:b])
            bound[a:b] += 4 * part(z[a:b]) * here + there * (4 * part(z[a:b]) * np.abs(lse[a:b]) + part(z[a:b]))
    got = f64(d)
    outside = np.isnan(want)
    assert (got[outside] == 7.0).all()
    off = np.abs(got - np.where(outside, 7.0, want))
    limit = bound * 1.001 + HALF[out] * np.abs(np.where(outside, 0.0, want)) + SUB[out]
    assert (off <= limit).all(), f"{np.max(off / limit)} of the bound"
    if db is not None:
        inside = ~outside[:, 0]
        limit = bound[inside].sum(axis=0) + 256 * U * size[inside].sum(axis=0) + SUB["f32"]
        assert (np.abs(f64(db) - want[inside].sum(axis=0)) <= limit).all()
    return d


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("t,e,k,s", [(1, 1, 1, 0), (3, 8, 8, 0), (129, 128, 8, 0), (40, 33, 5, 7), (1000, 256, 6, 3),
                                     (1025, 60, 4, 0), (5000, 100, 2, 70), (2500, 1024, 8, 5), (17, 700, 3, 40)])
def test_sizes(lib, rule, t, e, k, s):
    g = np.random.default_rng(t + e)
    logits, ids, bias = inputs(g, t, e, k)
    bias = bias if rule == "softmax" and e % 2 == 0 else None
    offsets = ragged(g, t, s) if s else None
    counts = check_balance(lib, logits, ids, rule, bias, offsets)
    for weights, losses, out in ((True, True, "f32"), (True, False, "bf16"), (False, True, "f16")):
        check_gradient(lib, g, logits, ids, rule, bias, offsets, counts, weights, losses, out)
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("rule", RULES)
def test_one_long_sequence_among_short_ones(lib, rule):
    g = np.random.default_rng(11)
    t, e, k = 4096, 64, 4
    logits, ids, _ = inputs(g, t, e, k)
    offsets = np.concatenate([np.arange(0, 100, 1), [100, 4000], np.arange(4001, 4090, 2)]).astype(np.int32)
    counts = check_balance(lib, logits, ids, rule, None, offsets)
    check_gradient(lib, g, logits, ids, rule, None, offsets, counts)


@pytest.mark.parametrize("rule", RULES)
def test_masked_and_extreme_logits(lib, rule):
    import torch
    g = np.random.default_rng(12)
    logits, ids, _ = inputs(g, 40, 48, 4)
    lowest = -np.finfo(np.float32).max
    logits[3, 5:] = -np.inf
    logits[4, 5:] = lowest
    logits[6] += 80
    logits[7] -= 85                     # the scores stay normal numbers, exp of the logits does not
    logits[8] = -np.inf                 # a row that holds nothing
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :4].astype(np.int32).copy()
    z = O.router_logits(logits)
    got_c, got_p, got_l = balance(lib, logits, ids, rule)
    want_c, want_p, want_l = O.balance_loss(logits, ids, rule)
    np.testing.assert_array_equal(got_c.cpu().numpy(), want_c)
    np.testing.assert_allclose(f64(got_p), want_p, rtol=(2 * 90 + 400) * U, atol=SUB["f32"])
    np.testing.assert_allclose(f64(got_l), want_l, rtol=(8 * 90 + 800) * U)
    d = torch.empty(40, 48, device="cuda")
    dl = np.array([20.0, 3.0], dtype=np.float32)
    lib.moe_route_backward(dev(logits), dev(ids), None, d, scoring=lib.SCORING_BY_NAME[rule],
                           counts=dev(want_c.astype(np.int32)), dlosses=dev(dl))
    want = O.route_backward(logits, ids, None, rule, counts=want_c, dlosses=dl)
    assert np.isfinite(f64(d)).all() and not d[8].any() and not d[3, 5:].any()
    p = O.router_probabilities(z, rule)
    np.testing.assert_allclose(f64(d), want, atol=float(1e-4 * np.abs(want).max()))
    assert np.isfinite(p).all()


@pytest.mark.parametrize("rule", RULES)
def test_selected_logits_of_minus_infinity(lib, rule):
    import torch
    logits = np.full((6, 40), -np.inf, dtype=np.float32)
    logits[1, 3], logits[2, :5] = 1.0, [1.0, 2.0, 3.0, -np.inf, 0.0]
    logits[4:] = np.random.default_rng(3).standard_normal((2, 40))
    ids = np.array([[0, 1, 2]] * 2 + [[0, 2, 3], [3, 0, 1], [5, 6, 7], [39, 0, 20]], dtype=np.int32)
    ids[1, 0] = 3
    dw = np.array([[1.0, 2.0, -1.0]] * 6, dtype=np.float32)
    counts = torch.ones(1, 40, dtype=torch.int32, device="cuda")
    for dl in (None, np.array([2.0, 0.5], dtype=np.float32)):
        d = torch.full((6, 40), np.nan, device="cuda")
        lib.moe_route_backward(dev(logits), dev(ids), dev(dw), d, scoring=lib.SCORING_BY_NAME[rule], counts=counts,
                               dlosses=None if dl is None else dev(dl))
        want = O.route_backward(logits, ids, dw, rule, counts=np.ones((1, 40)), dlosses=dl)
        np.testing.assert_allclose(f64(d), want, atol=1e-5)
    assert not d[0].any()


def test_bad_ids_and_offsets_are_reported(lib):
    import torch
    g = np.random.default_rng(13)
    logits, ids, _ = inputs(g, 30, 16, 2)
    ids[4, 0], ids[9, 1] = -1, 16
    counts, _, _ = balance(lib, logits, ids, "softmax")
    assert lib.device_status() == lib.DEV_BAD_EXPERT_ID
    np.testing.assert_array_equal(counts.cpu().numpy(), O.balance_loss(logits, ids)[0])
    d, dw = torch.empty(30, 16, device="cuda"), g.standard_normal((30, 2)).astype(np.float32)
    lib.moe_route_backward(dev(logits), dev(ids), dev(dw), d)
    assert lib.device_status() == lib.DEV_BAD_EXPERT_ID
    np.testing.assert_allclose(f64(d), O.route_backward(logits, ids, dw), atol=1e-5)
    ids = np.abs(ids) % 16
    for offsets in ([0, 20, 10, 30], [-3, 5, 30], [0, 10, 31]):
        balance(lib, logits, ids, "softmax", offsets=np.array(offsets, dtype=np.int32))
        assert lib.device_status() == lib.DEV_BAD_ROW
        lib.moe_route_backward(dev(logits), dev(ids), dev(dw), d, counts=torch.ones(len(offsets) - 1, 16, dtype=torch.int32,
                               device="cuda"), dlosses=torch.ones(2, device="cuda"),
                               seq_offsets=dev(np.array(offsets, dtype=np.int32)))
        assert lib.device_status() == lib.DEV_BAD_ROW


def test_an_expert_named_twice(lib):
    import torch
    g = np.random.default_rng(14)
    logits, ids, _ = inputs(g, 20, 40, 4)
    ids[:, 3] = ids[:, 1]
    dw = g.standard_normal((20, 4)).astype(np.float32)
    for rule in RULES:
        d = torch.empty(20, 40, device="cuda")
        lib.moe_route_backward(dev(logits), dev(ids), dev(dw), d, scoring=lib.SCORING_BY_NAME[rule])
        np.testing.assert_allclose(f64(d), O.route_backward(logits, ids, dw, rule), atol=1e-5)


def test_no_rows(lib):
    import torch
    counts, probs, losses = balance(lib, np.zeros((0, 32), np.float32), np.zeros((0, 2), np.int32), "softmax")
    assert not counts.any() and not probs.any() and not losses.any()
    counts, probs, losses = balance(lib, np.zeros((5, 32), np.float32), np.zeros((5, 2), np.int32), "sqrtsoftplus",
                                    offsets=np.array([2, 2, 2], dtype=np.int32))
    assert not counts.any() and not probs.any() and not losses.any()
    db = torch.full((32,), 3.0, device="cuda")
    ws = torch.empty(lib.moe_route_backward_workspace_bytes(0, 32), dtype=torch.uint8, device="cuda")
    lib.moe_route_backward(torch.empty(0, 32, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                           torch.empty(0, 2, device="cuda"), torch.empty(0, 32, device="cuda"), dbias=db, workspace=ws)
    assert not db.any()


def test_the_same_bits_again_and_captured(lib):
    import torch
    g = np.random.default_rng(15)
    for t, s in ((500, 0), (6000, 9)):
        logits, ids, bias = inputs(g, t, 128, 8)
        offsets = dev(ragged(g, t, s)) if s else None
        n = max(1, s)
        l, i, b, dw = dev(logits), dev(ids), dev(bias), dev(g.standard_normal((t, 8)).astype(np.float32))
        counts, probs = torch.empty(n, 128, dtype=torch.int32, device="cuda"), torch.empty(n, 128, device="cuda")
        losses, d, db = torch.empty(2, device="cuda"), torch.zeros(t, 128, device="cuda"), torch.empty(128, device="cuda")
        w1 = torch.empty(lib.moe_balance_workspace_bytes(t, 128, n), dtype=torch.uint8, device="cuda")
        w2 = torch.empty(lib.moe_route_backward_workspace_bytes(t, 128), dtype=torch.uint8, device="cuda")

        def both():
            lib.moe_balance_loss(l, i, counts, probs, losses, w1, bias=b, seq_offsets=offsets)
            lib.moe_route_backward(l, i, dw, d, bias=b, counts=counts, dlosses=losses, seq_offsets=offsets, dbias=db,
                                   workspace=w2)

        both()
        outputs = (counts, probs, losses, d, db)
        want = [o.clone() for o in outputs]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        for _ in range(3):
            for o in outputs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all((a == b).all() for a, b in zip(outputs, want))


def test_refusals(lib):
    import torch
    l, i = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    c, p, o = torch.zeros(1, 16, dtype=torch.int32, device="cuda"), torch.zeros(1, 16, device="cuda"), torch.zeros(2, device="cuda")
    ws = torch.empty(lib.moe_balance_workspace_bytes(4, 16, 1), dtype=torch.uint8, device="cuda")
    with pytest.raises(lib.BQError, match="WORKSPACE"):
        lib.moe_balance_loss(l, i, c, p, o, ws[:16])
    with pytest.raises(lib.BQError, match="only selects"):
        lib.moe_balance_loss(l, i, c, p, o, ws, bias=p[0], scoring=lib.SCORE_SQRTSOFTPLUS)
    with pytest.raises(lib.BQError, match="counts has shape"):
        lib.moe_balance_loss(l, i, c, p, o, ws, seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(lib.BQError, match="unknown scoring"):
        lib.moe_balance_loss(l, i, c, p, o, ws, scoring=3)
    with pytest.raises(lib.BQError, match="both NULL"):
        lib.moe_route_backward(l, i, None, torch.empty_like(l))
    with pytest.raises(lib.BQError, match="counts is NULL"):
        lib.moe_route_backward(l, i, None, torch.empty_like(l), dlosses=o)
    with pytest.raises(lib.BQError, match="WORKSPACE"):
        lib.moe_route_backward(l, i, torch.zeros(4, 2, device="cuda"), torch.empty_like(l), dbias=p[0])
    with pytest.raises(lib.BQError, match="no gradient"):
        lib.moe_route_backward(l, i, torch.zeros(4, 2, device="cuda"), torch.empty_like(l), dbias=p[0], scoring=1)
    with pytest.raises(lib.BQError, match="strides"):
        lib.moe_route_backward(l, i, torch.zeros(4, 2, device="cuda"), torch.empty(16, 4, device="cuda").t())

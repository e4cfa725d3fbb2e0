"""Pins of the oracle's FP8 row, product and row-move functions (CPU)."""
import math

import numpy as np
import pytest

import oracle as O


def test_e4m3_round_is_the_identity_on_every_value():
    v = O.e4m3_value(np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8))
    np.testing.assert_array_equal(O.e4m3_round(v), v)


@pytest.mark.parametrize("value,rounded", [(17, 16), (19, 20), (21, 20), (23, 24), (2 ** -10, 0), (3 * 2 ** -10, 2 ** -8),
                                           (-17, -16), (500, 448), (432, 448), (431.9, 416), (2 ** -10 + 1e-12, 2 ** -9)])
def test_e4m3_round_takes_the_nearest_and_ties_to_even(value, rounded):
    assert O.e4m3_round(np.array([value]))[0] == rounded


def test_e4m3_round_against_the_nearest_by_search():
    g = np.random.default_rng(1)
    v = g.standard_normal(2000) * np.exp2(g.integers(-12, 9, 2000))
    table = O.e4m3_value(np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8))
    near = np.abs(np.clip(v, -448, 448)[:, None] - table[None]).min(axis=1)
    np.testing.assert_array_equal(np.abs(O.e4m3_round(v) - np.clip(v, -448, 448)), near)


def test_quant_rows_scale_and_largest_code():
    x = np.zeros((3, 144))
    x[0, :128] = np.linspace(-7, 7, 128)
    x[1, 130] = 21.0
    q, s = O.quant_fp8_rows(x)
    assert s.shape == (3, 2) and s.dtype == np.float32
    assert s[0, 0] == np.float32(7 / 448) and q[0, 0] == -448 and q[0, 127] == 448
    assert s[1, 1] == np.float32(21 / 448) and q[1, 130] == 448 and s[1, 0] == np.float32(2.0 ** -126)
    assert not q[2].any()


def test_quant_rows_ties_of_sixteen_bit_values_are_exact():
    # 448 v / amax = 17 (between the codes 16 and 18) for v = 51/64, amax = 21, and 21 for v = 63/64
    x = np.zeros((1, 128))
    x[0, :3] = [21.0, 51 / 64, 63 / 64]
    q, _ = O.quant_fp8_rows(x)
    assert q[0, :3].tolist() == [448, 16, 20]


def test_quant_rows_do_not_hide_nan_or_infinity():
    x = np.ones((2, 128), dtype=np.float32)
    x[0, 5], x[1, 6] = np.nan, -np.inf
    q, s = O.quant_fp8_rows(x)
    assert np.isnan(s[0, 0]) and np.isnan(q[0]).all()
    assert np.isinf(s[1, 0]) and np.isnan(q[1, 6]) and not q[1, :6].any()


def test_mm_block_against_fsum():
    g = np.random.default_rng(2)
    m, n, k = 3, 130, 272
    x = O.e4m3_round(g.standard_normal((m, k)) * 50)
    xs = g.uniform(0.1, 1, (m, 3)).astype(np.float32)
    codes = g.integers(0, 127, (n, k)).astype(np.uint8)
    ws = g.uniform(0.1, 1, (2, 3)).astype(np.float32)
    w = O.e4m3_value(codes)
    y = O.mm_fp8_block(x, xs, codes, ws)
    for r in range(m):
        for c in (0, 1, 127, 128, 129):
            want = math.fsum(x[r, i] * float(xs[r, i // 128]) * w[c, i] * float(ws[c // 128, i // 128]) for i in range(k))
            assert abs(y[r, c] - want) <= 1e-12 * max(1, abs(want))


def test_row_moves_invert_and_adjoint():
    g = np.random.default_rng(3)
    t, k, h = 7, 3, 5
    inv = g.permutation(t * k).reshape(t, k).astype(np.int32)
    inv[2, 1] = -1
    x, ys = g.standard_normal((t, h)), g.standard_normal((t * k, h))
    w, dy = g.uniform(0.1, 1, (t, k)), g.standard_normal((t, h))
    xs = O.dispatch_rows(x, inv, np.full((t * k, h), 7.0))
    for a in range(t):
        for j in range(k):
            if inv[a, j] >= 0:
                assert (xs[inv[a, j]] == x[a]).all()
    assert (xs == 7.0).all(axis=1).sum() == 1
    # <dispatch(x), ys> = <x, combine(ys, 1)> over the rows in use
    used = np.zeros(t * k, dtype=bool)
    used[inv[inv >= 0]] = True
    assert abs((xs * ys)[used].sum() - (x * O.combine_rows(ys, inv, None)).sum()) < 1e-12
    # gradients of combine against differences
    dys, dw = O.combine_rows_backward(dy, ys, inv, w, np.zeros((t * k, h)))
    base, eps = (dy * O.combine_rows(ys, inv, w)).sum(), 1e-6
    for a, j in ((0, 0), (2, 1), (6, 2)):
        v = w.copy()
        v[a, j] += eps
        assert abs(((dy * O.combine_rows(ys, inv, v)).sum() - base) / eps - dw[a, j]) < 1e-6
    for r, c in ((0, 0), (11, 3)):
        v = ys.copy()
        v[r, c] += eps
        assert abs(((dy * O.combine_rows(v, inv, w)).sum() - base) / eps - dys[r, c]) < 1e-6

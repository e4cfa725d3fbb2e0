"""GPU parity: rows into expert order and back with their gradients, and the
FP8 row quantiser, against the fp64 oracle.

Tolerances (u = 2^-24, the fp32 half step; e = half step of the row type):
a sum of k products by fused multiply-adds is off by at most k u sum|terms|,
and the store by e |result|; a weight gradient adds H products, at most
H u sum|terms|; dys is one fp32 product and a store, (u + e) |result|.
Moves, codes and scales are exact."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}    # half a subnormal step (fp32: one step)


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rows(g, shape, dtype):
    """Random rows on the GPU and, exactly, as fp64."""
    import torch
    t = torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(torch_dtype(dtype))
    return t.cuda(), t.double().numpy()


def routing(g, t, k, drop=0.0):
    inv = g.permutation(t * k).reshape(t, k).astype(np.int32)
    inv[g.random((t, k)) < drop] = -1
    return inv


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


SHAPES = [(1, 6, 4096), (8, 6, 512), (3, 1, 16), (129, 8, 2048), (517, 5, 208), (2, 7, 8208)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,k,h", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_moves_and_gradients(lib, t, k, h, dtype, drop):
    import torch
    g = np.random.default_rng(t * 31 + k * 7 + h)
    inv = routing(g, t, k, drop)
    d_inv = dev(inv)
    x, x64 = rows(g, (t, h), dtype)
    # dispatch: exact, rows that no pair names stay
    xs = torch.full((t * k, h), 7.0, dtype=x.dtype, device="cuda")
    assert lib.moe_dispatch(x, d_inv, xs) is xs
    np.testing.assert_array_equal(f64(xs), O.dispatch_rows(x64, inv, np.full((t * k, h), 7.0)))
    # its gradient
    dxs, dxs64 = rows(g, (t * k, h), dtype)
    dx = torch.full_like(x, np.nan)
    lib.moe_dispatch_backward(dxs, d_inv.view(-1), dx)
    want = O.combine_rows(dxs64, inv, None)
    bound = k * U * O.combine_rows(np.abs(dxs64), inv, None) + HALF[dtype] * np.abs(want) + SUB[dtype]
    assert (np.abs(f64(dx) - want) <= bound * 1.001).all()
    # combine
    w = g.uniform(0.05, 1, (t, k)).astype(np.float32)
    ys, ys64 = rows(g, (t * k, h), dtype)
    y = torch.full_like(x, np.nan)
    lib.moe_combine(ys, d_inv, dev(w), y)
    want = O.combine_rows(ys64, inv, w)
    size = O.combine_rows(np.abs(ys64), inv, w)
    assert (np.abs(f64(y) - want) <= (k * U * size + HALF[dtype] * np.abs(want) + SUB[dtype]) * 1.001).all()
    # ... added to what y holds
    y = x.clone()
    lib.moe_combine(ys, d_inv, dev(w), y, accumulate=True)
    want = want + x64
    assert (np.abs(f64(y) - want) <= ((k + 1) * U * (size + np.abs(x64)) + HALF[dtype] * np.abs(want)
                                      + SUB[dtype]) * 1.001).all()
    # gradients of combine
    dys = torch.full((t * k, h), 7.0, dtype=x.dtype, device="cuda")
    dw = torch.full((t, k), np.nan, device="cuda")
    lib.moe_combine_backward(x, ys, d_inv, dev(w), dys, dw)
    want_s, want_w = O.combine_rows_backward(x64, ys64, inv, w, np.full((t * k, h), 7.0))
    assert (np.abs(f64(dys) - want_s) <= ((U + HALF[dtype]) * np.abs(want_s) + SUB[dtype]) * 1.001).all()
    _, size_w = O.combine_rows_backward(np.abs(x64), np.abs(ys64), inv, w, np.zeros((t * k, h)))
    assert (np.abs(f64(dw) - want_w) <= h * U * size_w).all()
    assert lib.device_status() == lib.DEV_OK


def test_one_gradient_alone_is_the_same(lib):
    import torch
    g = np.random.default_rng(5)
    t, k, h = 33, 4, 256
    d_inv, (dy, _), (ys, _) = dev(routing(g, t, k)), rows(g, (t, h), "bf16"), rows(g, (t * k, h), "bf16")
    w = dev(g.uniform(0, 1, (t, k)).astype(np.float32))
    dys, dw = torch.empty_like(ys), torch.empty_like(w)
    lib.moe_combine_backward(dy, ys, d_inv, w, dys, dw)
    only_s, only_w = torch.empty_like(ys), torch.empty_like(w)
    lib.moe_combine_backward(dy, None, d_inv, w, only_s, None)
    lib.moe_combine_backward(dy, ys, d_inv, None, None, only_w)
    assert torch.equal(only_s, dys) and torch.equal(only_w, dw)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_strided_rows_and_neighbours_untouched(lib, dtype):
    import torch
    g = np.random.default_rng(6)
    t, k, h = 19, 3, 64
    inv = routing(g, t, k)
    d_inv, w = dev(inv), dev(g.uniform(0, 1, (t, k)).astype(np.float32))
    wide, wide64 = rows(g, (t, 3 * h), dtype)
    x, x64 = wide[:, h:2 * h], wide64[:, h:2 * h]
    big = torch.full((t * k + 2, 2 * h), 7.0, dtype=wide.dtype, device="cuda")
    lib.moe_dispatch(x, d_inv, big[1:-1, :h])
    want = np.full((t * k + 2, 2 * h), 7.0)
    want[1:-1, :h] = O.dispatch_rows(x64, inv, want[1:-1, :h])
    np.testing.assert_array_equal(f64(big), want)
    # back from the strided rows, into strided rows
    out = torch.full((t + 2, 2 * h), 7.0, dtype=wide.dtype, device="cuda")
    dense = torch.empty(t, h, dtype=wide.dtype, device="cuda")
    lib.moe_combine(big[1:-1, :h], d_inv, w, out[1:-1, h:])
    lib.moe_combine(big[1:-1, :h].contiguous(), d_inv, w, dense)
    assert torch.equal(out[1:-1, h:], dense)
    assert (out[:, :h] == 7).all() and (out[0] == 7).all() and (out[-1] == 7).all()
    dys = torch.full_like(big, 7.0)
    lib.moe_combine_backward(x, big[1:-1, :h], d_inv, w, dys[1:-1, :h], torch.empty_like(w))
    assert (dys[:, h:] == 7).all() and (dys[0] == 7).all() and (dys[-1] == 7).all()


def test_bad_rows_are_reported_and_skipped(lib):
    import torch
    t, k, h = 4, 2, 64
    inv = np.arange(8, dtype=np.int32).reshape(t, k)
    inv[1, 0], inv[2, 1] = 8, -2
    x = torch.ones(t, h, device="cuda")
    buf = torch.full((12, h), 7.0, device="cuda")
    lib.moe_dispatch(x, dev(inv), buf[:8])
    assert lib.device_status() == lib.DEV_BAD_ROW and lib.device_status() == lib.DEV_OK
    assert (buf[[0, 1, 3, 4, 6, 7]] == 1).all() and (buf[[2, 5, 8, 9, 10, 11]] == 7).all()
    y, w = torch.empty(t, h, device="cuda"), torch.ones(t, k, device="cuda")
    lib.moe_combine(buf[:8], dev(inv), w, y)
    assert lib.device_status() == lib.DEV_BAD_ROW
    assert y[:, 0].tolist() == [2, 1, 1, 2]
    dys, dw = torch.full((8, h), 7.0, device="cuda"), torch.empty(t, k, device="cuda")
    lib.moe_combine_backward(x, buf[:8], dev(inv), w, dys, dw)
    assert lib.device_status() == lib.DEV_BAD_ROW
    assert dw.tolist() == [[h, h], [0, h], [h, 0], [h, h]] and (dys[[2, 5]] == 7).all()
    q, s = torch.zeros(8, h, dtype=torch.uint8, device="cuda"), torch.full((8, 1), 7.0, device="cuda")
    lib.moe_dispatch_fp8_b128(x, dev(inv), q, s)
    assert lib.device_status() == lib.DEV_BAD_ROW
    assert (s[[2, 5]] == 7).all() and (q[[2, 5]] == 0).all() and (s[[0, 1, 3, 4, 6, 7]] == np.float32(1 / 448)).all()


def test_a_dropped_pair_contributes_nothing_even_if_its_weight_is_nan(lib):
    import torch
    inv = dev(np.array([[0, -1], [-1, -1]], dtype=np.int32))
    ys = torch.ones(4, 16, device="cuda")
    ys[1:] = float("nan")
    w = torch.tensor([[2.0, float("nan")], [float("nan"), 1.0]], device="cuda")
    y = torch.full((2, 16), float("nan"), device="cuda")
    lib.moe_combine(ys, inv, w, y)
    assert (y[0] == 2).all() and (y[1] == 0).all()          # a token with no pair left gives zeros
    dw = torch.full((2, 2), 9.0, device="cuda")
    lib.moe_combine_backward(torch.ones(2, 16, device="cuda"), ys, inv, w, None, dw)
    assert dw.tolist() == [[16, 0], [0, 0]]


def test_no_tokens(lib):
    import torch
    e = torch.empty
    x, inv, w = e(0, 64, device="cuda"), e(0, 6, dtype=torch.int32, device="cuda"), e(0, 6, device="cuda")
    n = lib.launch_count()
    lib.moe_dispatch(x, inv, x)
    lib.moe_dispatch_backward(x, inv, x)
    lib.moe_combine(x, inv, w, x)
    lib.moe_combine_backward(x, x, inv, w, x, w)
    lib.moe_dispatch_fp8_b128(x, inv, e(0, 64, dtype=torch.uint8, device="cuda"), e(0, 1, device="cuda"))
    lib.quant_fp8_b128(x, e(0, 64, dtype=torch.uint8, device="cuda"), e(0, 1, device="cuda"))
    assert lib.launch_count() == n


# ---------------------------------------------------------------- FP8 rows
def quantised(lib, x, n_rows=None, fill=0xAA):
    import torch
    r, k = x.shape
    q = torch.full((r, k), fill, dtype=torch.uint8, device="cuda")
    s = torch.full((r, -(-k // 128)), 7.0, device="cuda")
    lib.quant_fp8_b128(x, q, s, n_rows=n_rows)
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("r,k", [(1, 16), (7, 4096), (33, 272), (300, 768), (5, 128), (2, 144), (1000, 1040)])
def test_quant_codes_and_scales_are_exact(lib, dtype, r, k):
    import torch
    g = np.random.default_rng(r + k)
    x = (g.standard_normal((r, k)) * np.exp(g.standard_normal(k))).astype(np.float32)
    x[:, ::37] = 0
    x = torch.from_numpy(x).to(torch_dtype(dtype))
    q, s = quantised(lib, x.cuda())
    want_q, want_s = O.quant_fp8_rows(x.double().numpy())
    np.testing.assert_array_equal(s, want_s)
    np.testing.assert_array_equal(O.e4m3_value(q), want_q)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quant_on_and_beside_every_border(lib, dtype):
    """Values whose quotient lies on a border between two codes, or one step of the type beside it."""
    import torch
    dt = torch_dtype(dtype)
    table = O.e4m3_value(np.arange(127, dtype=np.uint8))
    middles = (table[1:] + table[:-1]) / 2
    out = []
    for amax in (448.0, 1.0, 21.0, 7.0, 1.25, 0.0302734375, 1.5 * 2 ** -9, 60000.0):
        amax = float(torch.tensor(amax).to(dt))
        v = torch.tensor(middles * amax / 448.0, dtype=torch.float64).to(dt)
        inf = torch.full_like(v, float("inf"))
        step = lambda a, b: torch.nextafter(a, b) if dtype == "f32" else (  # noqa: E731
            (a.view(torch.int16) + (1 if b is inf else -1)).view(dt))
        for x in (v, step(v, inf), torch.where(v > 0, step(v.clamp(min=2.0 ** -14), None if dtype != "f32" else -inf), v)):
            row = torch.zeros(128, dtype=dt)
            row[:126] = x.clamp(max=amax)
            row[127] = amax
            out.append(row)
            out.append(-row)
    x = torch.stack(out)
    q, s = quantised(lib, x.cuda())
    want_q, want_s = O.quant_fp8_rows(x.double().numpy())
    np.testing.assert_array_equal(s, want_s)
    np.testing.assert_array_equal(O.e4m3_value(q), want_q)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quant_extremes(lib, dtype):
    import torch
    dt = torch_dtype(dtype)
    big, tiny = float(torch.finfo(dt).max), float(torch.finfo(dt).smallest_normal)
    x = torch.zeros(8, 256, dtype=dt)
    x[0, :128] = big
    x[0, 128:] = tiny
    x[1, 3], x[1, 200] = float("nan"), 1.0
    x[2, 4], x[2, 5], x[2, 130] = float("inf"), 2.0, 5.0
    x[3, 6] = -float("inf")
    x[5] = tiny / 4
    x[6, 0] = big
    x[6, 1:128] = tiny
    x[7] = -0.0
    q, s = quantised(lib, x.cuda())
    want_q, want_s = O.quant_fp8_rows(x.double().numpy())
    np.testing.assert_array_equal(s, want_s)
    np.testing.assert_array_equal(O.e4m3_value(q), want_q)


def test_quant_row_limit_on_the_device(lib):
    import torch
    x = torch.randn(37, 144, device="cuda").bfloat16()
    full_q, full_s = quantised(lib, x)
    for n, done in ((0, 0), (1, 1), (20, 20), (37, 37), (99, 37), (-5, 0)):
        q, s = quantised(lib, x, n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
        np.testing.assert_array_equal(q[:done], full_q[:done])
        np.testing.assert_array_equal(s[:done], full_s[:done])
        assert (q[done:] == 0xAA).all() and (s[done:] == 7).all()


def test_quant_strided_rows(lib):
    import torch
    wide = torch.randn(21, 768, device="cuda").half()
    q, s = quantised(lib, wide[:, 256:528])
    dq, ds = quantised(lib, wide[:, 256:528].contiguous())
    np.testing.assert_array_equal(q, dq)
    np.testing.assert_array_equal(s, ds)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,k,h", [(1, 6, 4096), (70, 8, 272), (300, 3, 128)])
def test_dispatch_fp8_is_dispatch_and_quant(lib, t, k, h, dtype):
    import torch
    g = np.random.default_rng(t + k)
    inv = routing(g, t, k, 0.2)
    x, x64 = rows(g, (t, h), dtype)
    q = torch.full((t * k, h), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((t * k, -(-h // 128)), 7.0, device="cuda")
    lib.moe_dispatch_fp8_b128(x, dev(inv), q.view(torch.float8_e4m3fn), s)
    want_q, want_s = O.quant_fp8_rows(x64)
    np.testing.assert_array_equal(s.cpu().numpy(), O.dispatch_rows(want_s, inv, np.full(s.shape, 7.0, np.float32)))
    fill = np.broadcast_to(O.e4m3_value(np.array([0x55], dtype=np.uint8)), q.shape)
    np.testing.assert_array_equal(O.e4m3_value(q.cpu().numpy()), O.dispatch_rows(want_q, inv, fill))


def test_the_binding_refuses_what_does_not_fit_on_the_gpu(lib):
    import torch
    x, xs = torch.zeros(4, 64, device="cuda"), torch.zeros(8, 64, device="cuda")
    inv, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    n = lib.launch_count()
    bad = [lambda: lib.moe_dispatch(x, inv, xs.half()), lambda: lib.moe_dispatch(x, inv, xs[:7]),
           lambda: lib.moe_dispatch(x[:, :62], inv, xs[:, :62]), lambda: lib.moe_dispatch(x, inv.t(), xs),
           lambda: lib.moe_combine(xs, inv, w.double(), x), lambda: lib.moe_combine(xs, inv, w[:3], x),
           lambda: lib.moe_combine(xs.t(), inv, w, x), lambda: lib.moe_dispatch_backward(xs, inv[:3], x),
           lambda: lib.quant_fp8_b128(x, xs, w), lambda: lib.moe_dispatch(x[:1].expand(4, 64), inv, xs),
           lambda: lib.moe_dispatch(x, torch.zeros(4, 9, dtype=torch.int32, device="cuda"),
                                    torch.zeros(36, 64, device="cuda"))]
    for call in bad:
        with pytest.raises(lib.BQError):
            call()
    assert lib.launch_count() == n


def test_gradients_against_differences(lib):
    """The forward calls are linear in rows and weights, so a difference over a whole step equals the gradient up to
    rounding: (k + 2) u of the sums' size on either side of the step, and H u for the weights' gradient."""
    import torch
    g = np.random.default_rng(12)
    t, k, h = 9, 4, 128
    inv = routing(g, t, k, 0.2)
    d_inv = dev(inv)
    (ys, ys64), (dy, dy64), (x, _), (dxs, dxs64) = (rows(g, s, "f32") for s in ((t * k, h), (t, h), (t, h), (t * k, h)))
    w = dev(g.uniform(0.1, 1, (t, k)).astype(np.float32))
    dys, dw = torch.zeros_like(ys), torch.empty_like(w)
    lib.moe_combine_backward(dy, ys, d_inv, w, dys, dw)

    def loss(ys_, w_):
        y = torch.empty_like(dy)
        lib.moe_combine(ys_, d_inv, w_, y)
        return (y.double() * dy.double()).sum().item()

    size = (O.combine_rows(np.abs(ys64), inv, np.full((t, k), 2.0)) * np.abs(dy64)).sum()
    base = loss(ys, w)
    for a, j in ((0, 0), (4, 2), (8, 3)):
        w2 = w.clone()
        w2[a, j] += 1
        step = (w2 - w)[a, j].item()
        assert abs((loss(ys, w2) - base) - step * dw[a, j].item()) <= 4 * (h + k + 2) * U * size
    for r, c in ((0, 0), (17, 5), (35, 127)):
        y2 = ys.clone()
        y2[r, c] += 1
        step = (y2.double() - ys.double())[r, c].item()
        assert abs((loss(y2, w) - base) - step * dys[r, c].item()) <= 4 * (k + 2) * U * (size + 2 * np.abs(dy64).max())
    # dispatch: <dispatch(x + e), dxs> - <dispatch(x), dxs> = <e, dx>
    dx = torch.empty_like(x)
    lib.moe_dispatch_backward(dxs, d_inv, dx)
    xs, xs2 = torch.zeros_like(ys), torch.zeros_like(ys)
    e = torch.randn_like(x)
    lib.moe_dispatch(x, d_inv, xs)
    lib.moe_dispatch(x + e, d_inv, xs2)
    step = (x + e).double() - x.double()
    got = ((xs2.double() - xs.double()) * dxs.double()).sum().item()
    bound = k * U * (np.abs(step.cpu().numpy()) * O.combine_rows(np.abs(dxs64), inv, None)).sum()
    assert abs(got - (step * dx.double()).sum().item()) <= 2 * bound


def test_rows_beyond_32_bit_offsets(lib):
    """Sorted matrices of more than 2^31 elements: every row against the token's row it came from."""
    import torch
    t, k, h = 270_000, 4, 2048                     # 2.2 G elements, 4.4 GB
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, h, generator=gen, device="cuda", dtype=torch.bfloat16)
    inv = torch.randperm(t * k, generator=gen, device="cuda").int().view(t, k)
    xs = torch.empty(t * k, h, device="cuda", dtype=torch.bfloat16)
    lib.moe_dispatch(x, inv, xs)
    for j in range(k):
        for a in range(0, t, 90_000):
            assert torch.equal(xs[inv[a:a + 90_000, j].long()], x[a:a + 90_000])
    w = torch.rand(t, k, generator=gen, device="cuda")
    y = torch.empty_like(x)
    lib.moe_combine(xs, inv, w, y)                 # every term is x[t]: y = (sum of weights) x, fp32, rounded once
    some = torch.tensor([0, 1, t // 2, t - 2, t - 1], device="cuda")
    want = (w[some].double().sum(1, keepdim=True) * x[some].double())
    assert ((y[some].double() - want).abs() <= (HALF["bf16"] + 2 * k * U) * want.abs() * 1.001 + SUB["bf16"]).all()
    dys, dw = xs, torch.empty_like(w)              # the last rows of dys and dw
    ys = torch.empty_like(xs)
    lib.moe_dispatch(x, inv, ys)
    lib.moe_combine_backward(x, ys, inv, w, dys, dw)
    want = (w[some].double()[..., None] * x[some].double()[:, None])
    assert ((dys[inv[some].long()].double() - want).abs() <= (HALF["bf16"] + U) * want.abs() * 1.001 + SUB["bf16"]).all()
    sq = x[some].double().square().sum(1, keepdim=True).expand(-1, k)
    assert ((dw[some].double() - sq).abs() <= h * U * sq).all()
    del dys, xs
    q, s = torch.empty(t * k, h, dtype=torch.uint8, device="cuda"), torch.empty(t * k, h // 128, device="cuda")
    lib.quant_fp8_b128(ys, q, s)
    for r in (0, t * k // 2, t * k - 3):
        want_q, want_s = O.quant_fp8_rows(ys[r:r + 3].double().cpu().numpy())
        np.testing.assert_array_equal(s[r:r + 3].cpu().numpy(), want_s)
        np.testing.assert_array_equal(O.e4m3_value(q[r:r + 3].cpu().numpy()), want_q)

"""GPU: the ends of the FP8 products' and the row kernels' ranges (the largest
sizes, malformed offsets, scales whose product leaves fp32, waits that run out
in a part of a cluster, neighbours of every code's border)."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

ONE = 0x38      # the e4m3 code of 1


def needs(gb):
    import torch
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB of free device memory")


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def e4m3_table():
    import torch
    return torch.from_numpy(O.e4m3_value(np.arange(256, dtype=np.uint8))).float().cuda()


@pytest.mark.parametrize("grouped", [False, True])
def test_as_many_rows_as_the_products_take(lib, grouped):
    """2^31 - 256 rows of 16: y is the first value of each row (times scales of 1), exact."""
    import torch
    needs(72)
    rows, k = 2 ** 31 - 256, 16
    x = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    piece = 1 << 26
    codes = (torch.arange(piece, device="cuda") % 113).to(torch.uint8)      # e4m3 codes of 0 .. 2^7
    for a in range(0, rows, piece):
        x[a:a + piece, 0] = codes[:min(piece, rows - a)]
    xs = torch.ones(rows, 1, device="cuda")
    w = torch.zeros(2, 1, k, dtype=torch.uint8, device="cuda")
    w[:, 0, 0] = ONE
    ws = torch.ones(2, 1, 1, device="cuda")
    y = torch.full((rows, 1), float("nan"), dtype=torch.float16, device="cuda")
    if grouped:
        off = torch.tensor([0, 200, rows], dtype=torch.int32, device="cuda")
        lib.moe_mm_fp8_b128(x, xs, off, w, ws, y)
    else:
        lib.mm_fp8_b128(x, xs, w[0], ws[0], y)
    assert lib.device_status() == lib.DEV_OK
    want = e4m3_table()[codes.long()].half()
    for a in range(0, rows, piece):
        assert torch.equal(y[a:a + piece, 0], want[:min(piece, rows - a)]), f"rows from {a}"


def test_ranges_that_overlap_leave_whole_experts_out(lib):
    """Offsets 0, 1024, 0, 1024: expert 1 descends, and expert 2's chunks are more than ascending offsets can make."""
    import torch
    g = np.random.default_rng(50)
    rows, n, k = 1024, 1024, 256
    x = dev(g.integers(0, 0x7F, (rows, k), dtype=np.uint8))
    xs, ws = torch.ones(rows, 2, device="cuda"), torch.ones(3, 8, 2, device="cuda")
    w = dev(g.integers(0, 0x7F, (3, n, k), dtype=np.uint8))
    y, want = torch.full((rows, n), 7.0, device="cuda"), torch.empty(rows, n, device="cuda")
    off = torch.tensor([0, rows, 0, rows], dtype=torch.int32, device="cuda")
    lib.moe_mm_fp8_b128(x, xs, off, w, ws, y)
    assert lib.device_status() == lib.DEV_BAD_ROW
    lib.mm_fp8_b128(x, xs, w[0], ws[0], want)      # the same tile, so the same sums
    assert torch.equal(y, want)


def test_ranges_that_overlap_more_often_than_an_int_counts(lib):
    """512 experts of all of 1.1e9 rows (of one weight, so that it does not matter which one a row gets): 4.4e9 chunks."""
    import torch
    needs(40)
    rows, k, e = 1_100_000_000, 16, 1024
    x = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    x[::1000, 0] = ONE
    xs = torch.ones(rows, 1, device="cuda")
    w = torch.zeros(e, 1, k, dtype=torch.uint8, device="cuda")
    w[:, 0, 0] = ONE
    y = torch.full((rows, 1), float("nan"), dtype=torch.float16, device="cuda")
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    lib.moe_mm_fp8_b128(x, xs, off, w, torch.ones(e, 1, 1, device="cuda"), y)
    assert lib.device_status() == lib.DEV_BAD_ROW
    assert (y[::1000] == 1).all() and int((y == 0).sum()) == rows - rows // 1000


@pytest.mark.parametrize("op", ["quant", "dispatch"])
def test_the_longest_row_the_quantiser_takes(lib, op):
    """One row of 2^31 - 16 values: the last group has 112."""
    import torch
    needs(24)
    k = 2 ** 31 - 16
    x = torch.ones(1, k, dtype=torch.float16, device="cuda")
    x[0, 1] = 7.0                  # group 0: 1 -> code of 64, scale 7 / 448
    x[0, k - 3] = 28.0             # the last group: 1 -> code of 16
    q = torch.zeros(1, k, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, 2 ** 24, device="cuda")
    if op == "quant":
        lib.quant_fp8_b128(x, q, s)
    else:
        lib.moe_dispatch_fp8_b128(x, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), q, s)
    assert lib.device_status() == lib.DEV_OK
    want_s = torch.full_like(s, np.float32(1 / 448))
    want_s[0, 0], want_s[0, -1] = float(np.float32(7 / 448)), float(np.float32(28 / 448))
    assert torch.equal(s, want_s)
    top = 0x7E                     # the code of 448
    assert q[0, 1] == top and q[0, k - 3] == top and (q[0, 128:-112] == top).all()
    assert (e4m3_table()[q[0, 2:128].long()] == 64).all()
    last = e4m3_table()[q[0, -112:].long()]
    assert int((last == 16).sum()) == 111 and last[-3] == 448


@pytest.mark.parametrize("m,n,k,swiglu", [(1, 4096, 4096, False), (3, 256, 1024, False), (32, 512, 1024, True),
                                          (8, 8192, 2048, False)])
def test_a_wait_that_runs_out_in_one_part_of_a_split_leaves_y(lib, m, n, k, swiglu):
    """K split over 4, 8, 8 and 2 parts, the odd ones without copies: the others have their sums, y is not written."""
    import torch
    g = np.random.default_rng(51)
    x, w = dev(g.integers(0, 0x7F, (m, k), dtype=np.uint8)), dev(g.integers(0, 0x7F, (n, k), dtype=np.uint8))
    xs, ws = torch.ones(m, k // 128, device="cuda"), torch.ones(n // 128, k // 128, device="cuda")
    y, want = (torch.full((m, n // 2 if swiglu else n), 7.0, device="cuda") for _ in range(2))
    lib.test_set_wait_probe(True, 2_000_000, odd_parts_only=True)
    try:
        lib.mm_fp8_b128(x, xs, w, ws, y, swiglu=swiglu)
        assert lib.device_status() == lib.DEV_WAIT_TIMEOUT
    finally:
        lib.test_set_wait_probe(False)
    assert (y == 7).all()
    lib.mm_fp8_b128(x, xs, w, ws, y, swiglu=swiglu)
    lib.mm_fp8_b128(x, xs, w, ws, want, swiglu=swiglu)
    assert lib.device_status() == lib.DEV_OK
    assert torch.equal(y, want) and (y != 7).all()


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (100, 256, 1024), (2048, 2048, 512)])
def test_calls_queued_behind_one_whose_waits_run_out(lib, m, n, k):
    """No synchronisation in between: the next calls take the shared memory and TMEM that the failed one left."""
    import torch
    g = np.random.default_rng(52)
    x, w = dev(g.integers(0, 0x7F, (m, k), dtype=np.uint8)), dev(g.integers(0, 0x7F, (n, k), dtype=np.uint8))
    xs, ws = torch.ones(m, k // 128, device="cuda"), torch.ones(n // 128, k // 128, device="cuda")
    y, z, want = (torch.full((m, n), 7.0, device="cuda") for _ in range(3))
    lib.mm_fp8_b128(x, xs, w, ws, want)
    for odd in (False, True) * 3:
        lib.test_set_wait_probe(True, 1_000_000, odd_parts_only=odd)
        try:
            lib.mm_fp8_b128(x, xs, w, ws, z)
        finally:
            lib.test_set_wait_probe(False)
        y.fill_(7.0)
        for _ in range(4):
            lib.mm_fp8_b128(x, xs, w, ws, y)
        assert lib.device_status() == lib.DEV_WAIT_TIMEOUT
        assert torch.equal(y, want) and (z == 7).all()


def products(lib, x, xs, w, ws, swiglu, grouped):
    """y (fp32) of the codes' product, dense or with every row in the second of three experts."""
    import torch
    m, n = x.shape[0], w.shape[0]
    y = torch.full((m, n // 2 if swiglu else n), 7.0, device="cuda")
    if grouped:
        off = torch.tensor([0, 0, m, m], dtype=torch.int32, device="cuda")
        lib.moe_mm_fp8_b128(dev(x), dev(xs), off, dev(np.stack([w] * 3)), dev(np.stack([ws] * 3)), y, swiglu=swiglu)
    else:
        lib.mm_fp8_b128(dev(x), dev(xs), dev(w), dev(ws), y, swiglu=swiglu)
    assert lib.device_status() == lib.DEV_OK
    return y


def bound(x, xs, w, ws):
    """(exact product, bound of the error of fp32 sums): (259 + kb) u S as for scales of ordinary size, and half a
    subnormal step for each block where a sum comes out below the normal numbers."""
    kb = xs.shape[1]
    size = O.mm_fp8_block(np.abs(O.e4m3_value(x)), np.abs(xs), w & 0x7F, np.abs(ws))
    exact = O.mm_fp8_block(O.e4m3_value(x), xs, w, ws)
    return exact, (260 + kb) * 2.0 ** -24 * size + (kb + 1) * 2.0 ** -150


# rows that take the split lanes, the lanes, and the wide tile
RANGE = [(1, 256, 1024), (7, 512, 272), (32, 4096, 256), (45, 384, 512), (700, 1280, 400)]


def scaled_case(m, n, k, ex, ew):
    """Random codes of both signs; row scales of about 2^ex, weight scales of about 2^ew, of both signs."""
    g = np.random.default_rng(10000 + ex * 31 + ew + m)
    kb, nb = -(-k // 128), -(-n // 128)
    x, w = (g.integers(0, 0x7F, s, dtype=np.uint8) | (g.integers(0, 2, s, dtype=np.uint8) << 7) for s in ((m, k), (n, k)))
    xs, ws = (np.float32(g.choice([-1.0, 1.0], s) * np.exp2(e + g.uniform(-1, 1, s))) for e, s in
              ((ex, (m, kb)), (ew, (nb, kb))))
    assert (xs != 0).all() and (ws != 0).all() and np.isfinite(xs).all() and np.isfinite(ws).all()
    return x, xs, w, ws


def assert_within(got, want, err):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / err).max()
    assert worst <= 1.0, f"{worst:.2f} times the bound"


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("m,n,k", RANGE)
@pytest.mark.parametrize("ex,ew", [(-126, 4), (-126, 126), (126, -126), (-140, 30), (30, -140), (-62, -60), (50, 48)])
def test_scales_of_any_size_whose_product_is_normal(lib, m, n, k, ex, ew, grouped):
    x, xs, w, ws = scaled_case(m, n, k, ex, ew)
    exact, err = bound(x, xs, w, ws)
    assert_within(products(lib, x, xs, w, ws, False, grouped), exact, err)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("m,n,k", RANGE)
@pytest.mark.parametrize("ex,ew", [(-126, -1), (-126, -14), (-126, -24), (-100, -40), (-8, -130), (-120, -100)])
def test_scales_whose_product_is_below_the_normal_numbers(lib, m, n, k, ex, ew, grouped):
    """The product of the scales is off by half a subnormal step, 2^-150, and a block's sum is below 2^25."""
    x, xs, w, ws = scaled_case(m, n, k, ex, ew)
    exact, err = bound(x, xs, w, ws)
    assert_within(products(lib, x, xs, w, ws, False, grouped), exact, err + xs.shape[1] * 2.0 ** -125)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m,n,k", [(8, 512, 1024), (45, 512, 512), (700, 1280, 400)])
def test_zero_rows_are_zero_and_change_no_other(lib, m, n, k, swiglu):
    """A padded batch: rows of zeros get the smallest scale, whose product with the weight's is subnormal."""
    import torch
    g = np.random.default_rng(61)
    rows = torch.randn(m, k, device="cuda")
    padded = rows.clone()
    padded[2::3] = 0.0
    w, ws = g.integers(0, 0x7F, (n, k), dtype=np.uint8), np.float32(g.uniform(1e-5, 1e-4, (-(-n // 128), -(-k // 128))))
    y = []
    for r in (rows, padded):
        q, s = torch.empty(m, k, dtype=torch.uint8, device="cuda"), torch.empty(m, -(-k // 128), device="cuda")
        lib.quant_fp8_b128(r, q, s)
        y.append(products(lib, q.cpu().numpy(), s.cpu().numpy(), w, ws, swiglu, False))
    assert (y[1][2::3] == 0).all()
    keep = torch.arange(m, device="cuda") % 3 != 2
    assert torch.equal(y[0][keep], y[1][keep])


@pytest.mark.parametrize("m,n,k", RANGE)
def test_scales_whose_product_is_beyond_fp32_show_in_their_rows_only(lib, m, n, k):
    x, xs, w, ws = scaled_case(m, n, k, -5, 10)
    x[0], xs[0, 0] = 0, 2.0 ** 127          # zeros: NaN, as the header says
    got = products(lib, x, xs, w, ws, False, False)
    assert not got[0].isfinite().any()
    if m > 1:
        exact, err = bound(x[1:], xs[1:], w, ws)
        assert_within(got[1:], exact, err)


HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("amax", [448.0, 1.0, 21.0, 7.0, 1.25, 0.0302734375, 1.5 * 2 ** -9, 60000.0, 3.0 * 2.0 ** -14])
def test_quotients_one_step_beside_every_border(lib, dtype, amax):
    """For each border of two codes the value of the type nearest to it, and the values one step above and below that."""
    import torch
    dt = torch_type(dtype)
    bits = {"f32": torch.int32}.get(dtype, torch.int16)
    amax = torch.tensor(amax).to(dt)
    table = O.e4m3_value(np.arange(127, dtype=np.uint8))
    at = torch.from_numpy((table[1:] + table[:-1]) / 2 * amax.double().item() / 448.0).to(dt)
    at = at[at > 0]                                   # fp16 has no value beside the smallest borders of a small amax
    assert at.numel() >= 100
    up, down = ((at.view(bits) + d).to(bits).view(dt) for d in (1, -1))    # neighbours of a positive value
    assert (up > at).all() and (down < at).all() and (down >= 0).all()
    rows = []
    for v in (at, up, down):
        row = torch.zeros(128, dtype=dt)
        row[:at.numel()] = v.clamp(max=amax.item())
        row[127] = amax
        rows += [row, -row]
    x = torch.stack(rows)
    q, s = torch.empty(6, 128, dtype=torch.uint8, device="cuda"), torch.empty(6, 1, device="cuda")
    lib.quant_fp8_b128(x.cuda(), q, s)
    want_q, want_s = O.quant_fp8_rows(x.double().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(O.e4m3_value(q.cpu().numpy()), want_q)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,ld", [(5000, 101, 104), (5000, 101, 112), (2500, 357, 360), (2500, 260, 264), (4, 101, 104)])
def test_rows_of_y_on_16_byte_boundaries_that_end_inside_a_vector(lib, m, n, ld, out):
    import torch
    k = 144
    x, xs, w, ws = scaled_case(m, n, k, -9, -9)
    big = torch.full((m, ld), 7.0, dtype=torch_type(out), device="cuda")
    y = big[:, :n]
    lib.mm_fp8_b128(dev(x), dev(xs), dev(w), dev(ws), y)
    exact, err = bound(x, xs, w, ws)
    assert_within(y, exact, err + HALF_STEP[out] * np.abs(exact) + 2.0 ** -25)     # fp16's half subnormal step
    assert (big[:, n:] == 7).all() and lib.device_status() == lib.DEV_OK


def test_backward_and_fp8_rows_beyond_32_bit_offsets(lib):
    """Sorted matrices of more than 2^31 elements: the sort's gradient, and the sort into FP8 rows."""
    import torch
    needs(24)
    t, k, h = 270_000, 4, 2048
    gen = torch.Generator(device="cuda").manual_seed(2)
    dxs = torch.randn(t * k, h, generator=gen, device="cuda", dtype=torch.bfloat16)
    inv = torch.randperm(t * k, generator=gen, device="cuda").int().view(t, k)
    dx = torch.full((t, h), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.moe_dispatch_backward(dxs, inv, dx)
    for a in range(0, t, 30_000):
        terms = dxs[inv[a:a + 30_000].long()].double()
        err = k * 2.0 ** -24 * terms.abs().sum(1) + 2.0 ** -8 * terms.sum(1).abs() * 1.001 + 2.0 ** -134
        assert ((dx[a:a + 30_000].double() - terms.sum(1)).abs() <= err).all()
    q = torch.empty(t * k, h, dtype=torch.uint8, device="cuda")
    s = torch.empty(t * k, h // 128, device="cuda")
    lib.moe_dispatch_fp8_b128(dx, inv, q, s)
    one_q, one_s = torch.empty(t, h, dtype=torch.uint8, device="cuda"), torch.empty(t, h // 128, device="cuda")
    lib.quant_fp8_b128(dx, one_q, one_s)
    for j in range(k):
        for a in range(0, t, 90_000):
            at = inv[a:a + 90_000, j].long()
            assert torch.equal(q[at], one_q[a:a + 90_000]) and torch.equal(s[at], one_s[a:a + 90_000])
    assert lib.device_status() == lib.DEV_OK

"""GPU parity: the FP8 x FP8 block-scaled product, dense and over rows sorted
by expert, and the FP8 MoE layer made of these operators.

Tolerance of one element (u = 2^-24, S = sum|terms|, e = half step of y's
type): products of two e4m3 values are exact in fp32; a block's 128 terms are
added with at most one fp32 step (2 u) lost each; the two scales and their
product are three roundings; the kb blocks are added by fused multiply-adds.
So |y - exact| <= (256 + 3 + kb) u S + e |exact|.  SwiGLU: |silu'| <= 1.1 and
|silu(g)| <= |g|, so errors dg, du of its inputs give 1.1 |u| dg + |g| du, and
the function itself (exp, division, two products) at most 16 u |y|, to which
the exponent's argument adds u |g| |y|.

Largest of all the weights' and rows' scales here keep y within fp16."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def fp8_rows(g, m, k):
    """Codes (uint8), their values and scales of random rows."""
    codes = g.integers(0, 254, (m, k), dtype=np.uint8)
    codes += codes >= 0x7F                     # every byte but the two NaNs
    return codes, O.e4m3_value(codes), g.uniform(1e-3, 4e-3, (m, -(-k // 128))).astype(np.float32)


def fp8_weight(g, mats, n, k):
    codes = g.integers(0, 254, (mats, n, k), dtype=np.uint8)
    codes += codes >= 0x7F
    return codes, g.uniform(5e-5, 2e-4, (mats, -(-n // 128), -(-k // 128))).astype(np.float32)


def expected(x, xs, w, ws, out, swiglu=False):
    """(exact y, bound of the error) of one product in fp64."""
    y = O.mm_fp8_block(x, xs, w, ws)
    size = O.mm_fp8_block(np.abs(x), xs, w & 0x7F, ws)
    err = (259 + xs.shape[1]) * U * size
    if swiglu:
        n = y.shape[1] // 2
        g, u, dg, du = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
        y = g / (1 + np.exp(-g)) * u
        err = 1.1 * np.abs(u) * dg + np.abs(g) * du + dg * du + (16 + np.abs(g)) * U * np.abs(y)
    return y, err + HALF[out] * np.abs(y) + 2.0 ** -24


def check(got, want, err, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    worst = (np.abs(got - want) / err).max() if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"


MM = [(1, 128, 128), (1, 4096, 4096), (8, 256, 2048), (32, 256, 2048), (33, 200, 272), (7, 1, 16), (64, 1000, 144),
      (129, 384, 512), (130, 4096, 768), (257, 511, 1040), (300, 130, 128), (1000, 640, 384), (16, 4096, 4096),
      (5, 129, 8208), (65, 2048, 640), (2, 5000, 2048), (700, 2050, 272), (5000, 100, 144),
      (1153, 1024, 128)]


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", MM)
def test_dense_product(lib, m, n, k, out):
    import torch
    g = np.random.default_rng(m * 7 + n * 3 + k)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    y = torch.full((m, n), float("nan"), dtype=torch_dtype(out), device="cuda")
    assert lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y) is y
    check(y, *expected(x, xs, w[0], ws[0], out), f"{m}x{n}x{k}")
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 256, 128), (8, 1536, 2048), (40, 768, 272), (130, 512, 1040), (300, 1280, 512),
                                   (520, 256, 384), (3, 4096, 4096), (1200, 1024, 384), (3333, 256, 16)])
def test_dense_product_with_swiglu(lib, m, n, k, out):
    import torch
    g = np.random.default_rng(m + n + k)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    y = torch.full((m, n // 2), float("nan"), dtype=torch_dtype(out), device="cuda")
    lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y, swiglu=True)
    check(y, *expected(x, xs, w[0], ws[0], out, True), f"swiglu {m}x{n}x{k}")


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m", [1, 8, 31])
@pytest.mark.parametrize("n", [14 * 128, 15 * 128, 16 * 128, 36 * 128, 38 * 128, 76 * 128, 78 * 128])
@pytest.mark.parametrize("k", [640, 656, 912, 1936])
def test_borders_of_the_split_over_k(lib, m, n, k, swiglu):
    """Parts of one block, of unequal sizes and with a short last block; a part's adds and those over the cluster are
    together at most kb, the bound's count."""
    import torch
    g = np.random.default_rng(m + n + k)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    y = torch.full((m, n // 2 if swiglu else n), float("nan"), dtype=torch.float32, device="cuda")
    if swiglu and n % 256:   # gate and up halves would not start on a block of scales
        with pytest.raises(lib.BQError, match="BQ_ERR_SHAPE"):
            lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y, swiglu=True)
        assert torch.isnan(y).all()
        return
    lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y, swiglu=swiglu)
    check(y, *expected(x, xs, w[0], ws[0], "f32", swiglu), f"{m}x{n}x{k}")
    assert lib.device_status() == lib.DEV_OK


def run_grouped(lib, g, counts, n, k, out, swiglu, behind=0, first=0):
    """The grouped product over experts of `counts` rows, rows 0..first and the last `behind` outside every expert."""
    import torch
    e, used = len(counts), int(np.sum(counts))
    rows = first + used + behind
    codes, x, xs = fp8_rows(g, rows, k)
    w, ws = fp8_weight(g, e, n, k)
    off = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    cols = n // 2 if swiglu else n
    y = torch.full((rows, cols), 7.0, dtype=torch_dtype(out), device="cuda")
    lib.moe_mm_fp8_b128(dev(codes), dev(xs), dev(off), dev(w), dev(ws), y, swiglu=swiglu)
    torch.cuda.synchronize()
    for i in range(e):
        a, b = off[i], off[i + 1]
        if a < b:
            check(y[a:b], *expected(x[a:b], xs[a:b], w[i], ws[i], out, swiglu), f"expert {i} of {b - a} rows")
    assert (y[:first] == 7).all() and (y[first + used:] == 7).all()
    assert lib.device_status() == lib.DEV_OK


GROUPS = [
    ([1, 0, 2, 1, 0, 0, 1, 3], 384, 256),
    ([0, 0, 5, 0], 128, 272),
    ([33, 1, 130, 0, 64, 7], 512, 384),
    ([300, 0, 1, 257, 16], 256, 640),
    ([1], 256, 4096),
    ([700], 768, 144),
    ([17] * 40, 256, 128),
    ([0] * 30 + [2] + [0] * 33, 1536, 2048),
    ([40] * 30, 512, 384),
    ([200, 0, 1, 300, 77, 0, 129, 128], 1024, 272),
    ([3, 0, 1, 17] * 40, 2048, 144),
]


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped_product(lib, case, swiglu, out):
    counts, n, k = GROUPS[case]
    g = np.random.default_rng(case + 10 * swiglu)
    run_grouped(lib, g, counts, 256 * -(-n // 256) if swiglu else n, k, out, swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_rows_outside_every_expert_stay(lib, swiglu):
    run_grouped(lib, np.random.default_rng(3), [3, 0, 70, 9], 256, 256, "bf16", swiglu, behind=200, first=5)
    run_grouped(lib, np.random.default_rng(3), [130, 0, 700, 9], 1024, 256, "bf16", swiglu, behind=200, first=5)


def test_grouped_odd_columns(lib):
    run_grouped(lib, np.random.default_rng(2), [500, 0, 333, 150], 1001, 144, "f16", False)
    for n in (1, 127, 129, 1000):
        run_grouped(lib, np.random.default_rng(n), [4, 0, 33, 150], n, 144, "f32", False)


def test_grouped_many_experts_and_none_with_rows(lib):
    run_grouped(lib, np.random.default_rng(4), [0] * 8, 256, 128, "f32", False, behind=6)
    counts = np.zeros(1024, dtype=int)
    counts[[0, 5, 511, 1022, 1023]] = [2, 1, 20, 1, 3]
    run_grouped(lib, np.random.default_rng(5), counts, 128, 128, "f32", False)


def test_grouped_bad_offsets_are_reported_and_skipped(lib):
    import torch
    g = np.random.default_rng(6)
    n, k, rows = 128, 128, 12
    codes, x, xs = fp8_rows(g, rows, k)
    w, ws = fp8_weight(g, 4, n, k)
    # experts 1 (descends) and 3 (past the end) are skipped; the others keep their rows
    off = np.array([0, 4, 2, 8, 13], dtype=np.int32)
    y = torch.full((rows, n), 7.0, device="cuda")
    lib.moe_mm_fp8_b128(dev(codes), dev(xs), dev(off), dev(w), dev(ws), y)
    assert lib.device_status() == lib.DEV_BAD_ROW and lib.device_status() == lib.DEV_OK
    want = np.full((rows, n), 7.0)
    for e, a, b in ((0, 0, 4), (2, 2, 8)):
        want[a:b] = O.mm_fp8_block(x[a:b], xs[a:b], w[e], ws[e])
    got = y.double().cpu().numpy()
    assert np.abs(got[[0, 1, 4, 5, 6, 7]] - want[[0, 1, 4, 5, 6, 7]]).max() < 1e-4 and (got[8:] == 7).all()


@pytest.mark.parametrize("m", [3, 200, 2000])
def test_nan_and_infinite_scales_stay_in_their_rows_and_columns(lib, m):
    import torch
    g = np.random.default_rng(7)
    n, k = 384, 384
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    codes[1, 130] = 0x7F          # a NaN code
    xs[2, 1] = np.inf
    w[0, 140, 7] = 0xFF
    ws[0, 2, 0] = np.nan          # columns 256..383
    y = torch.zeros(m, n, device="cuda")
    lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y)
    y = y.cpu().numpy()
    assert np.isnan(y[1]).all() and not np.isfinite(y[2]).any()
    assert np.isnan(y[:, 140]).all() and np.isnan(y[:, 256:]).all()
    rest = np.delete(np.delete(y, [1, 2], 0), np.r_[140, 256:384], 1)
    want, err = expected(np.delete(x, [1, 2], 0), np.delete(xs, [1, 2], 0), w[0], np.nan_to_num(ws[0]), "f32")
    keep = np.delete(np.arange(n), np.r_[140, 256:384])
    assert (np.abs(rest - want[:, keep]) <= err[:, keep]).all()


@pytest.mark.parametrize("m", [2, 70, 300, 3000])
def test_strided_output(lib, m):
    import torch
    g = np.random.default_rng(8)
    n, k = 200, 256
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    for dt in ("f16", "f32"):
        big = torch.full((m + 2, 413), 7.0, dtype=torch_dtype(dt), device="cuda")
        lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), big[1:-1, 3:203])
        check(big[1:-1, 3:203], *expected(x, xs, w[0], ws[0], dt))
        assert (big[0] == 7).all() and (big[-1] == 7).all() and (big[:, :3] == 7).all() and (big[:, 203:] == 7).all()


def test_no_rows(lib):
    import torch
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    n = lib.launch_count()
    lib.mm_fp8_b128(e(0, 128, dt=torch.uint8), e(0, 1), e(128, 128, dt=torch.uint8), e(1, 1), e(0, 128))
    lib.moe_mm_fp8_b128(e(0, 128, dt=torch.uint8), e(0, 1), torch.zeros(3, dtype=torch.int32, device="cuda"),
                        e(2, 128, 128, dt=torch.uint8), e(2, 1, 1), e(0, 128))
    assert lib.launch_count() == n


@pytest.mark.parametrize("m", [1, 33, 260, 1500])
def test_two_runs_agree_bit_for_bit(lib, m):
    import torch
    g = np.random.default_rng(9)
    codes, _, xs = fp8_rows(g, m, 2048)
    w, ws = fp8_weight(g, 1, 512, 2048)
    a = [dev(codes), dev(xs), dev(w[0]), dev(ws[0])]
    y, z = torch.empty(m, 512, device="cuda"), torch.empty(m, 512, device="cuda")
    lib.mm_fp8_b128(*a, y)
    lib.mm_fp8_b128(*a, z)
    assert torch.equal(y, z)


def test_input_gradient_is_the_product_with_the_transposed_weight(lib):
    """dx = q(dy) W: 128 x 128 blocks and their scales transpose exactly."""
    import torch
    g = np.random.default_rng(10)
    m, n, k = 40, 384, 256
    w, ws = fp8_weight(g, 1, n, k)
    dy = torch.from_numpy(g.standard_normal((m, n)).astype(np.float32)).cuda().bfloat16()
    q = torch.empty(m, n, dtype=torch.uint8, device="cuda")
    s = torch.empty(m, 3, device="cuda")
    lib.quant_fp8_b128(dy, q, s)
    dx = torch.empty(m, k, device="cuda")
    lib.mm_fp8_b128(q, s, dev(w[0].T), dev(ws[0].T), dx)
    v, sv = O.quant_fp8_rows(dy.double().cpu().numpy())
    full = v * np.repeat(sv.astype(np.float64), 128, 1)
    want = full @ O.dequant_fp8_block(w[0], ws[0])
    _, err = expected(v, sv, np.ascontiguousarray(w[0].T), np.ascontiguousarray(ws[0].T), "f32")
    check(dx, want, err)


def fp8_layer(lib, t, h, inter, e, k, seed, graph=False):
    """One MoE layer of FP8 experts through the public entry points; returns every intermediate."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    x = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    logits = torch.randn(t, e, generator=g, device="cuda")
    rng = np.random.default_rng(seed)
    gu, gus = fp8_weight(rng, e, 2 * inter, h)
    dn, dns = fp8_weight(rng, e, h, inter)
    d = {"x": x, "gu": gu, "gus": gus, "dn": dn, "dns": dns, "ids": z(t, k, dt=torch.int32), "w": z(t, k),
         "off": z(e + 1, dt=torch.int32), "inv": z(t, k, dt=torch.int32), "q1": z(t * k, h, dt=torch.uint8),
         "s1": z(t * k, -(-h // 128)), "act": z(t * k, inter, dt=torch.bfloat16), "q2": z(t * k, inter, dt=torch.uint8),
         "s2": z(t * k, -(-inter // 128)), "ys": z(t * k, h), "y": z(t, h)}
    d_gu, d_gus, d_dn, d_dns = dev(gu), dev(gus), dev(dn), dev(dns)
    cnt, pt, ps = z(e, dt=torch.int32), z(t * k, dt=torch.int32), z(t * k, dt=torch.int32)
    ws = z(lib.moe_permute_workspace_bytes(t, k, e), dt=torch.uint8)

    def layer(stream=None):
        lib.moe_route(logits, None, k, d["ids"], d["w"], stream=stream)
        lib.moe_permute(d["ids"], e, cnt, d["off"], pt, ps, d["inv"], ws, stream=stream)
        lib.moe_dispatch_fp8_b128(x, d["inv"], d["q1"], d["s1"], stream=stream)
        lib.moe_mm_fp8_b128(d["q1"], d["s1"], d["off"], d_gu, d_gus, d["act"], swiglu=True, stream=stream)
        lib.quant_fp8_b128(d["act"], d["q2"], d["s2"], n_rows=d["off"][e:], stream=stream)
        lib.moe_mm_fp8_b128(d["q2"], d["s2"], d["off"], d_dn, d_dns, d["ys"], stream=stream)
        lib.moe_combine(d["ys"], d["inv"], d["w"], d["y"], stream=stream)

    d["layer"], d["logits"], d["keep"] = layer, logits, (d_gu, d_gus, d_dn, d_dns, cnt, pt, ps, ws)
    return d


def check_layer(d, t, h, inter, e, k):
    """Each stage against the oracle on the device's own inputs of that stage."""
    n = lambda name: d[name].cpu().numpy()  # noqa: E731
    ids, w = O.route(d["logits"].cpu().numpy(), k, None)
    np.testing.assert_array_equal(n("ids"), ids)
    ref = O.permute(ids, e)
    inv, off = n("inv"), ref["offsets"]
    np.testing.assert_array_equal(inv.reshape(-1), ref["inv"])
    x64 = d["x"].double().cpu().numpy()
    q1, s1 = O.quant_fp8_rows(x64)
    np.testing.assert_array_equal(O.e4m3_value(n("q1")), O.dispatch_rows(q1, inv, np.zeros((t * k, h))))
    q2, s2 = O.quant_fp8_rows(d["act"].double().cpu().numpy())
    np.testing.assert_array_equal(O.e4m3_value(n("q2")), q2)
    np.testing.assert_array_equal(n("s2"), s2)
    v1 = O.e4m3_value(n("q1"))
    for i in range(e):
        a, b = off[i], off[i + 1]
        if a < b:
            check(d["act"][a:b], *expected(v1[a:b], n("s1")[a:b], d["gu"][i], d["gus"][i], "bf16", True), f"gate/up {i}")
            check(d["ys"][a:b], *expected(q2[a:b], s2[a:b], d["dn"][i], d["dns"][i], "f32"), f"down {i}")
    ys = n("ys").astype(np.float64)
    want, size = O.combine_rows(ys, inv, n("w")), O.combine_rows(np.abs(ys), inv, n("w"))
    assert (np.abs(n("y") - want) <= (k + 1) * U * size * 1.001).all()


@pytest.mark.parametrize("t,h,inter,e,k", [(1, 512, 256, 8, 3), (8, 384, 128, 16, 6), (200, 256, 384, 8, 2),
                                           (400, 512, 128, 4, 2)])
def test_fp8_layer_stage_by_stage(lib, t, h, inter, e, k):
    import torch
    d = fp8_layer(lib, t, h, inter, e, k, 11 + t)
    d["layer"]()
    torch.cuda.synchronize()
    assert lib.device_status() == lib.DEV_OK
    check_layer(d, t, h, inter, e, k)


def test_fp8_layer_captured_replayed_and_on_another_stream(lib):
    import torch
    shape = (40, 256, 128, 8, 2)
    a, b = fp8_layer(lib, *shape, 21), fp8_layer(lib, *shape, 22)
    a["layer"](), b["layer"]()
    torch.cuda.synchronize()
    want_a, want_b = a["y"].clone(), b["y"].clone()
    side = torch.cuda.Stream()
    graphs = []
    for d in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            d["layer"]()
        graphs.append(gr)
    for name in ("act", "ys", "y"):
        a[name].fill_(float("nan")), b[name].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):       # the two graphs overlap
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(a["y"], want_a) and torch.equal(b["y"], want_b)
    # a graph takes the contents of its buffers at replay: other logits
    a["logits"].neg_()
    graphs[0].replay()
    torch.cuda.synchronize()
    check_layer(a, *shape)
    other = torch.cuda.Stream()
    a["y"].zero_()
    other.wait_stream(torch.cuda.current_stream())
    a["layer"](stream=other)
    other.synchronize()
    check_layer(a, *shape)
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("m,n,k", [(3, 256, 1024), (300, 512, 1024), (2048, 2048, 512)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(lib, m, n, k):
    import torch
    g = np.random.default_rng(30)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    a = [dev(codes), dev(xs), dev(w[0]), dev(ws[0]), torch.empty(m, n, device="cuda")]
    lib.test_set_wait_probe(True, 2_000_000)
    try:
        lib.mm_fp8_b128(*a)
        assert lib.device_status() == lib.DEV_WAIT_TIMEOUT
    finally:
        lib.test_set_wait_probe(False)
    lib.mm_fp8_b128(*a)
    assert lib.device_status() == lib.DEV_OK
    check(a[-1], *expected(x, xs, w[0], ws[0], "f32"))


@pytest.mark.parametrize("experts", [0, 1000])
def test_rows_and_outputs_beyond_32_bit_offsets(lib, experts):
    """x of more than 2^32 bytes and y of more than 2^31 bytes, of one weight and of 1000: rows from the start, the middle
    and the end."""
    import torch
    m, n, k = 4_300_000, 256, 1008
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    g = np.random.default_rng(40)
    kb = 8
    base, x, xs = fp8_rows(g, 1000, k)
    codes, scales = dev(base).repeat(m // 1000, 1), dev(xs).repeat(m // 1000, 1)
    e = max(experts, 1)
    w, ws = fp8_weight(g, e, n, k)
    y = torch.empty(m, n, dtype=torch.float16, device="cuda")
    if experts:
        off = torch.arange(0, m + 1, m // e, device="cuda", dtype=torch.int32)      # 4300 rows each
        lib.moe_mm_fp8_b128(codes, scales, off, dev(w), dev(ws), y)
    else:
        lib.mm_fp8_b128(codes, scales, dev(w[0]), dev(ws[0]), y)
    assert scales.shape[1] == kb
    for r in (0, 2_150_000, m - 1000):
        for a in range(r, r + 1000, 100):      # pieces of 100 rows lie within one expert
            i = a // (m // e) if experts else 0
            check(y[a:a + 100], *expected(x[a - r:a - r + 100], xs[a - r:a - r + 100], w[i], ws[i], "f16"), f"row {a}")
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("each", [1, 45])
def test_weights_beyond_32_bit_offsets(lib, each):
    """300 experts of 4096 x 4096: 5 GB; the first, the last and one behind 2^32 bytes hold values, the others zeros.
    A row each takes the tile with the weights on the lanes, 45 the wide one."""
    import torch
    e, n, k = 300, 4096, 4096
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free device memory")
    g = np.random.default_rng(41)
    some, (codes, scales) = [0, 270, 299], fp8_weight(g, 3, n, k)
    w = torch.zeros(e, n, k, dtype=torch.uint8, device="cuda")
    ws = torch.ones(e, 32, 32, device="cuda")
    for j, i in enumerate(some):
        w[i], ws[i] = dev(codes[j]), dev(scales[j])
    xc, x, xs = fp8_rows(g, e * each, k)
    off = torch.arange(0, e * each + 1, each, dtype=torch.int32, device="cuda")
    y = torch.full((e * each, n), 7.0, device="cuda")
    lib.moe_mm_fp8_b128(dev(xc), dev(xs), off, w, ws, y)
    zero = torch.ones(e * each, dtype=torch.bool, device="cuda")
    for j, i in enumerate(some):
        a, b = i * each, (i + 1) * each
        zero[a:b] = False
        check(y[a:b], *expected(x[a:b], xs[a:b], codes[j], scales[j], "f32"), f"expert {i}")
    assert (y[zero] == 0).all()

"""GPU parity: FP8 products that end in a bias, an activation, a scale and a residual.

Tolerance (u = 2^-24): the product v as in the plain products' tests,
(259 + kb) u S, and u |v| for the bias.  An activation passes an error on by at
most its largest slope (silu 1.1, gelu and its tanh form 1.13, relu 1, relu2
2 |v|) and adds its own: silu (16 + |v|) u |y| (the exponent's argument, exp, the
reciprocal), gelu 2 u |v| (an approximation of Phi off by 0.75e-7 = 1.3 u at
most) + 16 u |y|, its tanh form (16 + 8 |w|) u |y| with w the exponent's argument;
then two roundings, 2 u (|scale y| + |residual|), and the output's half step."""
import numpy as np
import pytest

import oracle as O
from test_gpu_fp8_mm import HALF, U, check, dev, fp8_rows, fp8_weight, torch_dtype

pytestmark = pytest.mark.gpu

SLOPE = {"silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13, "relu": 1.0, "none": 1.0}


def expected(x, xs, w, ws, out, act, bias, scale, residual):
    v = O.mm_fp8_block(x, xs, w, ws)
    size = O.mm_fp8_block(np.abs(x), xs, w & 0x7F, ws)
    v = v + (0.0 if bias is None else bias.astype(np.float64))
    err = (259 + xs.shape[1]) * U * size + U * np.abs(v)
    y = O.activation(v, act)
    if act == "swiglu":
        n = v.shape[1] // 2
        g, up, dg, du = v[:, :n], v[:, n:], err[:, :n], err[:, n:]
        err = 1.1 * np.abs(up) * dg + np.abs(g) * du + dg * du + (16 + np.abs(g)) * U * np.abs(y)
    elif act == "relu2":
        err = 2 * np.abs(v) * err + err * err + 2 * U * np.abs(y)
    else:
        own = {"silu": 16 + np.abs(v), "gelu": 16.0 + 2 * np.abs(v) / np.maximum(np.abs(y), 1e-30),
               "gelu_tanh": 16 + 8 * np.abs(1.6 * (v + 0.045 * v ** 3)), "relu": 0.0,
               "none": 0.0}[act]
        err = SLOPE[act] * err + own * U * np.abs(y)
    y, err = scale * y, abs(scale) * err + 2 * U * abs(scale) * np.abs(y)
    if residual is not None:
        y, err = y + residual, err + 2 * U * np.abs(residual)
    return y, err + HALF[out] * np.abs(y) + 2.0 ** -24


def made_residual(g, shape, out):
    import torch
    t = torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(torch_dtype(out))
    return t.cuda(), t.double().numpy()


ACTS = ["none", "swiglu", "silu", "gelu", "gelu_tanh", "relu", "relu2"]
# weights on the lanes, with K split over a cluster (the first four) and not; rows on the lanes
SIZES = [(1, 4096, 4096), (8, 1536, 2048), (32, 512, 1040), (31, 256, 768), (3, 5120, 272), (33, 256, 272), (300, 1280, 512),
         (1200, 1024, 384), (2500, 256, 144)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_activations_at_every_path(lib, m, n, k, act):
    import torch
    g = np.random.default_rng(m + n + k)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    bias = g.standard_normal(n).astype(np.float32)
    cols = n // 2 if act == "swiglu" else n
    for out in ("f32", "f16", "bf16"):
        res, res64 = made_residual(g, (m, cols), out)
        y = torch.full((m, cols), float("nan"), dtype=torch_dtype(out), device="cuda")
        lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y, act=act, bias=dev(bias), residual=res, scale=0.5)
        check(y, *expected(x, xs, w[0], ws[0], out, act, bias, 0.5, res64), f"{act} {out}")
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("m,n,k", [(1, 129, 528), (40, 4095, 144), (7, 1, 16), (130, 4095, 272), (700, 2050, 128),
                                   (260, 4097, 16)])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_parts_alone_odd_sizes_strides_and_in_place(lib, m, n, k, out):
    import torch
    g = np.random.default_rng(m * n + k)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    args = (dev(codes), dev(xs), dev(w[0]), dev(ws[0]))
    bias = g.standard_normal(n).astype(np.float32)
    res, res64 = made_residual(g, (m, n), out)
    new = (lambda: torch.full((m, n), float("nan"), dtype=res.dtype, device="cuda"))
    check(lib.mm_fp8_b128(*args, new(), bias=dev(bias)), *expected(x, xs, w[0], ws[0], out, "none", bias, 1.0, None), "bias")
    check(lib.mm_fp8_b128(*args, new(), act="relu"), *expected(x, xs, w[0], ws[0], out, "relu", None, 1.0, None), "act")
    check(lib.mm_fp8_b128(*args, new(), scale=-2.0), *expected(x, xs, w[0], ws[0], out, "none", None, -2.0, None), "scale")
    want = expected(x, xs, w[0], ws[0], out, "gelu", bias, 0.25, res64)
    for before, behind in ((0, 0), (1, 2), (16, 16)):       # rows on no boundary, and on one
        wide = torch.full((m + 1, before + n + behind), 7.0, dtype=res.dtype, device="cuda")
        y = wide[:-1, before:before + n]
        y.copy_(res)
        lib.mm_fp8_b128(*args, y, act="gelu", bias=dev(bias), residual=y, scale=0.25)
        check(y, *want, f"in place, {before} columns before")
        assert (wide[-1] == 7).all() and (wide[:, :before] == 7).all() and (wide[:, before + n:] == 7).all()
    assert torch.equal(lib.mm_fp8_b128(*args, new()), lib.mm_fp8_b128(*args, new(), act="none", scale=1.0))


GROUPS = [([1, 0, 2, 1, 0, 0, 1, 3], 512, 256), ([33, 1, 130, 0, 64, 7], 512, 384), ([300, 0, 1, 257, 16], 256, 640),
          ([17] * 40, 256, 128), ([0] * 30 + [2] + [0] * 33, 1536, 2048), ([0, 0], 256, 128)]


@pytest.mark.parametrize("act", ["none", "swiglu", "silu"])
@pytest.mark.parametrize("counts,n,k", GROUPS)
def test_experts_with_biases(lib, counts, n, k, act):
    import torch
    g = np.random.default_rng(sum(counts) + n)
    e, used, first, behind = len(counts), int(np.sum(counts)), 3, 5
    rows = first + used + behind
    codes, x, xs = fp8_rows(g, rows, k)
    w, ws = fp8_weight(g, e, n, k)
    bias = g.standard_normal((e, n)).astype(np.float32)
    off = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    cols = n // 2 if act == "swiglu" else n
    for out in ("bf16", "f32"):
        res, res64 = made_residual(g, (rows, cols), out)
        y = torch.full((rows, cols), 7.0, dtype=res.dtype, device="cuda")
        lib.moe_mm_fp8_b128(dev(codes), dev(xs), dev(off), dev(w), dev(ws), y, act=act, bias=dev(bias), residual=res,
                            scale=0.5)
        for i in range(e):
            a, b = off[i], off[i + 1]
            if a < b:
                check(y[a:b], *expected(x[a:b], xs[a:b], w[i], ws[i], out, act, bias[i], 0.5, res64[a:b]), f"expert {i}")
        assert (y[:first] == 7).all() and (y[first + used:] == 7).all()
    assert lib.device_status() == lib.DEV_OK


def test_nan_is_not_hidden(lib):
    import torch
    g = np.random.default_rng(3)
    for m in (4, 300):
        codes, _, xs = fp8_rows(g, m, 256)
        w, ws = fp8_weight(g, 1, 256, 256)
        codes[2, 7] = 0x7F
        bias = np.zeros(256, dtype=np.float32)
        bias[5] = np.nan
        for act in ("none", "silu", "gelu", "gelu_tanh", "relu", "relu2"):
            y = torch.zeros(m, 256, device="cuda")
            lib.mm_fp8_b128(dev(codes), dev(xs), dev(w[0]), dev(ws[0]), y, act=act, bias=dev(bias))
            nan = torch.isnan(y).cpu().numpy()
            assert nan[2].all() and nan[:, 5].all()
            assert not np.delete(np.delete(nan, 2, axis=0), 5, axis=1).any()


def test_captured(lib):
    import torch
    g = np.random.default_rng(4)
    codes, _, xs = fp8_rows(g, 8, 1024)
    w, ws = fp8_weight(g, 1, 512, 1024)
    args = [dev(codes), dev(xs), dev(w[0]), dev(ws[0])]
    bias = torch.randn(512, device="cuda")
    start = torch.randn(8, 512, device="cuda")
    y, want = start.clone(), start.clone()
    for _ in range(2):
        lib.mm_fp8_b128(*args, want, act="silu", bias=bias, residual=want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.mm_fp8_b128(*args, y, act="silu", bias=bias, residual=y)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_refusals(lib):
    import torch
    x, xs = torch.zeros(4, 128, dtype=torch.uint8, device="cuda"), torch.ones(4, 1, device="cuda")
    w, ws, y = torch.zeros(256, 128, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, device="cuda"), torch.zeros(4, 256, device="cuda")
    with pytest.raises(lib.BQError, match="unknown activation"):
        lib.mm_fp8_b128(x, xs, w, ws, y, act="tanh")
    with pytest.raises(lib.BQError, match="exclude each other"):
        lib.mm_fp8_b128(x, xs, w, ws, y, swiglu=True, act="silu")
    with pytest.raises(lib.BQError, match="bias has shape"):
        lib.mm_fp8_b128(x, xs, w, ws, y, bias=torch.zeros(128, device="cuda"))
    with pytest.raises(lib.BQError, match="bias has type"):
        lib.mm_fp8_b128(x, xs, w, ws, y, bias=torch.zeros(256, device="cuda", dtype=torch.float16))
    with pytest.raises(lib.BQError, match="residual has type"):
        lib.mm_fp8_b128(x, xs, w, ws, y, residual=y.half())
    with pytest.raises(lib.BQError, match="residual has shape"):
        lib.mm_fp8_b128(x, xs, w, ws, y[:, :128], act="swiglu", residual=y)

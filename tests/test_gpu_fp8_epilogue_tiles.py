"""GPU parity: FP8 products with an end, where the CTAs of the wide kernel take several tiles each.

There are more tiles than SMs, and many a CTA meets a chunk of few rows (some of
its warps have none of them) before a fuller one of another expert, whose bias is
far from the first's.  K is one block or a few, so that little separates the
tiles.  Every row is compared, with the bounds of the other products with an end."""
import numpy as np
import pytest

import oracle as O
from test_gpu_fp8_epilogue import expected, made_residual
from test_gpu_fp8_mm import check, dev, fp8_rows, fp8_weight, torch_dtype

pytestmark = pytest.mark.gpu

SMS = 152


def meets(tiles_of_chunk):
    """Does a CTA meet a chunk of 96 rows or fewer, then one of more rows than that?  Tiles as their chunks' rows."""
    return any(tiles_of_chunk[i] <= 96 < tiles_of_chunk[i + SMS] for i in range(len(tiles_of_chunk) - SMS))


# the rows of the experts in turn, the columns of y's tiles beside them
@pytest.mark.parametrize("k", [16, 128, 400])
@pytest.mark.parametrize("act", ["none", "swiglu", "gelu"])
@pytest.mark.parametrize("counts", [[5, 128] * 10, [33, 1, 128, 0, 97, 64] * 4])
def test_short_experts_before_full_ones(lib, counts, act, k):
    import torch
    n = 4096
    per_chunk = n // 256
    assert meets([c for c in counts if c for _ in range(per_chunk)])
    g = np.random.default_rng(sum(counts) + k)
    e, first, behind = len(counts), 2, 3
    rows = first + sum(counts) + behind
    codes, x, xs = fp8_rows(g, rows, k)
    w, ws = fp8_weight(g, e, n, k)
    bias = (g.standard_normal((e, n)) + np.where(np.arange(e) % 2, 3.0, -3.0)[:, None]).astype(np.float32)
    off = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    cols = n // 2 if act == "swiglu" else n
    args = [dev(codes), dev(xs), dev(off), dev(w), dev(ws)]
    for out, with_residual in (("bf16", True), ("f32", True), ("f16", False), ("f32", False)):
        res, res64 = made_residual(g, (rows, cols), out)
        y = torch.full((rows, cols), 7.0, dtype=res.dtype, device="cuda")
        lib.moe_mm_fp8_b128(*args, y, act=act, bias=dev(bias), residual=res if with_residual else None, scale=0.5)
        for i in range(e):
            a, b = off[i], off[i + 1]
            if a < b:
                want = expected(x[a:b], xs[a:b], w[i], ws[i], out, act, bias[i], 0.5, res64[a:b] if with_residual else None)
                check(y[a:b], *want, f"{act} {out}, expert {i} of {b - a} rows")
        assert (y[:first] == 7).all() and (y[off[-1]:] == 7).all()
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("k", [16, 128])
@pytest.mark.parametrize("act", ["none", "swiglu", "silu"])
def test_a_last_chunk_of_fewer_rows(lib, act, k):
    import torch
    m, cols = 289, 14336                                   # chunks of 97, 97 and 95 rows
    n = 2 * cols if act == "swiglu" else cols
    tiles = cols // (128 if act == "swiglu" else 256)
    assert meets([97, 97, 95] * tiles)                     # the chunks of a tile of columns one after the other
    g = np.random.default_rng(k)
    codes, x, xs = fp8_rows(g, m, k)
    w, ws = fp8_weight(g, 1, n, k)
    bias = (3 * g.standard_normal(n)).astype(np.float32)
    args = [dev(codes), dev(xs), dev(w[0]), dev(ws[0])]
    for out, with_residual in (("bf16", True), ("f32", False)):
        res, res64 = made_residual(g, (m, cols), out)
        y = torch.full((m, cols), float("nan"), dtype=torch_dtype(out), device="cuda")
        lib.mm_fp8_b128(*args, y, act=act, bias=dev(bias), residual=res if with_residual else None)
        want = expected(x, xs, w[0], ws[0], out, act, bias, 1.0, res64 if with_residual else None)
        check(y, *want, f"{act} {out}")
    assert lib.device_status() == lib.DEV_OK

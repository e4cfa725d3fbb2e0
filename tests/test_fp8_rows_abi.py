"""Refusals of the row-move, FP8 row and FP8 product entry points (no GPU needed):
each is made on the host, before any launch."""
import ctypes
import os

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300")
P = ctypes.c_void_p(4096)         # an aligned address that no call below dereferences
ODD = ctypes.c_void_p(4104)       # 8-byte aligned only
OK, NULL, SHAPE, ALIGN, FORMAT = 0, 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def bq():
    if not os.path.exists(os.path.join(PKG, "libbq.so")):
        import __graft_entry__
        __graft_entry__.build()
    import block_quantized_moe_gather_gb300 as m
    return m


@pytest.mark.parametrize("call,status", [
    (lambda L: L.bq_moe_dispatch(P, 3, 4, 64, 64, P, 2, P, 64, None), FORMAT),
    (lambda L: L.bq_moe_dispatch(P, F16, -1, 64, 64, P, 2, P, 64, None), SHAPE),
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 0, 64, P, 2, P, 64, None), SHAPE),
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 64, P, 0, P, 64, None), SHAPE),
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 64, P, 9, P, 64, None), SHAPE),
    (lambda L: L.bq_moe_dispatch(P, F16, 2 ** 30, 64, 64, P, 2, P, 64, None), SHAPE),       # T * k beyond int32
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 63, P, 2, P, 64, None), SHAPE),             # ld < H
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 60, 64, P, 2, P, 64, None), ALIGN),             # 120-byte rows
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 68, P, 2, P, 64, None), ALIGN),
    (lambda L: L.bq_moe_dispatch(ODD, F16, 4, 64, 64, P, 2, P, 64, None), ALIGN),
    (lambda L: L.bq_moe_dispatch(None, F16, 4, 64, 64, P, 2, P, 64, None), NULL),
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 64, None, 2, P, 64, None), NULL),
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 64, ctypes.c_void_p(4098), 2, P, 64, None), ALIGN),
    (lambda L: L.bq_moe_dispatch(P, F16, 4, 64, 64, P, 2, None, 64, None), NULL),
    (lambda L: L.bq_moe_dispatch(None, F16, 0, 64, 64, None, 2, None, 64, None), OK),       # no tokens
    (lambda L: L.bq_moe_dispatch_backward(P, F32, 4, 64, 64, P, 2, None, 64, None), NULL),
    (lambda L: L.bq_moe_dispatch_backward(P, F32, 4, 62, 64, P, 2, P, 64, None), ALIGN),
    (lambda L: L.bq_moe_dispatch_backward(None, F32, 0, 64, 64, None, 2, None, 64, None), OK),
    (lambda L: L.bq_moe_combine(P, BF16, 4, 64, 64, P, None, 2, 0, P, 64, None), NULL),     # weights
    (lambda L: L.bq_moe_combine(P, BF16, 4, 64, 64, P, P, 2, 2, P, 64, None), SHAPE),       # accumulate
    (lambda L: L.bq_moe_combine(P, BF16, 4, 64, 64, P, P, 2, 0, P, 8, None), SHAPE),
    (lambda L: L.bq_moe_combine(None, BF16, 0, 64, 64, None, None, 2, 0, None, 64, None), OK),
    (lambda L: L.bq_moe_combine_backward(P, 64, P, 64, F32, 4, 64, P, P, 2, None, 0, None, None), NULL),
    (lambda L: L.bq_moe_combine_backward(P, 64, None, 0, F32, 4, 64, P, P, 2, P, 64, P, None), NULL),   # ys
    (lambda L: L.bq_moe_combine_backward(P, 64, P, 64, F32, 4, 64, P, None, 2, P, 64, P, None), NULL),  # weights
    (lambda L: L.bq_moe_combine_backward(P, 64, P, 64, 5, 4, 64, P, P, 2, P, 64, P, None), FORMAT),
    (lambda L: L.bq_moe_combine_backward(P, 64, P, 32, F32, 4, 64, P, P, 2, P, 64, P, None), SHAPE),
    (lambda L: L.bq_quant_fp8_b128(P, F16, 4, 72, 72, None, P, P, None), SHAPE),            # k not a multiple of 16
    (lambda L: L.bq_quant_fp8_b128(P, F16, 4, 0, 72, None, P, P, None), SHAPE),
    (lambda L: L.bq_quant_fp8_b128(P, 7, 4, 64, 64, None, P, P, None), FORMAT),
    (lambda L: L.bq_quant_fp8_b128(P, F16, 4, 64, 32, None, P, P, None), SHAPE),
    (lambda L: L.bq_quant_fp8_b128(P, F16, 4, 64, 64, None, None, P, None), NULL),
    (lambda L: L.bq_quant_fp8_b128(P, F16, 4, 64, 64, None, ODD, P, None), ALIGN),
    (lambda L: L.bq_quant_fp8_b128(P, F16, 4, 64, 64, ctypes.c_void_p(4097), P, P, None), ALIGN),
    (lambda L: L.bq_quant_fp8_b128(None, F16, 0, 64, 64, None, None, None, None), OK),
    (lambda L: L.bq_moe_dispatch_fp8_b128(P, F16, 4, 64, 64, None, 2, P, P, None), NULL),
    (lambda L: L.bq_moe_dispatch_fp8_b128(P, F16, 4, 64, 64, P, 9, P, P, None), SHAPE),
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 128, 72, 0, P, F16, 128, None), SHAPE),      # k not a multiple of 16
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 0, 64, 0, P, F16, 128, None), SHAPE),
    (lambda L: L.bq_mm_fp8_b128(P, P, -4, P, P, 128, 64, 0, P, F16, 128, None), SHAPE),
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 128, 64, 1, P, F16, 128, None), SHAPE),      # gate/up n % 256
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 128, 64, 2, P, F16, 128, None), SHAPE),
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 128, 64, 0, P, 3, 128, None), FORMAT),
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 128, 64, 0, P, F16, 127, None), SHAPE),
    (lambda L: L.bq_mm_fp8_b128(ODD, P, 4, P, P, 128, 64, 0, P, F16, 128, None), ALIGN),
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, None, 128, 64, 0, P, F16, 128, None), NULL),
    (lambda L: L.bq_mm_fp8_b128(P, P, 4, P, P, 128, 64, 0, ctypes.c_void_p(4098), F32, 128, None), ALIGN),
    (lambda L: L.bq_mm_fp8_b128(None, None, 0, None, None, 128, 64, 0, None, F16, 128, None), OK),
    (lambda L: L.bq_moe_mm_fp8_b128(P, P, 4, None, 8, P, P, 128, 64, 0, P, F16, 128, None), NULL),
    (lambda L: L.bq_moe_mm_fp8_b128(P, P, 4, P, 0, P, P, 128, 64, 0, P, F16, 128, None), SHAPE),
    (lambda L: L.bq_moe_mm_fp8_b128(P, P, 4, P, 1025, P, P, 128, 64, 0, P, F16, 128, None), SHAPE),
    (lambda L: L.bq_moe_mm_fp8_b128(P, P, 4, P, 1024, P, P, 2 ** 22, 64, 0, P, F16, 2 ** 22, None), SHAPE),
])
def test_refused_before_any_launch(bq, call, status):
    assert call(bq._lib) == status
    if status != OK:
        assert bq.last_error()


def test_the_binding_refuses_tensors_that_do_not_fit(bq):
    import torch
    x, xs, inv = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(bq.BQError, match="not on a CUDA device"):
        bq.moe_dispatch(x, inv, xs)
    where = "w"
    with pytest.raises(bq.BQError, match="shape"):
        bq._rows_of(where, "x", x, rows=5)
    with pytest.raises(bq.BQError, match="not contiguous"):
        bq._rows_of(where, "x", x.t())
    with pytest.raises(bq.BQError, match="FORMAT"):
        bq._rows_of(where, "x", x.double())
    with pytest.raises(bq.BQError, match="FORMAT"):
        bq._rows_of(where, "x", x, dtype=bq.DT_F16)
    with pytest.raises(bq.BQError, match="FORMAT"):
        bq._pairs(where, inv.long(), 4)
    with pytest.raises(bq.BQError, match="SHAPE"):
        bq._pairs(where, inv, 3)
    with pytest.raises(bq.BQError, match="SHAPE"):
        bq._dense(where, "weights", x.t(), (64, 4), "f32")
    with pytest.raises(bq.BQError, match="FORMAT"):
        bq._dense(where, "q", x, (4, 64), "fp8")
    assert bq._pairs(where, inv.view(-1), 4) == (inv.data_ptr(), 2)
    assert bq._rows_of(where, "x", torch.zeros(4, 128)[:, 64:])[2:] == (4, 64, 128)
    assert bq._rows_of(where, "x", torch.zeros(1, 64).expand(4, 64))[4] == 0      # the library refuses the stride

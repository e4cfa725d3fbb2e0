"""Sizes next to 2^31 at the FP8 entry points: what the kernels cannot count is
refused on the host (no GPU needed; every pointer is NULL, so a size that is
taken ends as BQ_ERR_NULL)."""
import os

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300")
NULL, SHAPE = 1, 2
F16 = 1
MOST = 2 ** 31 - 256


@pytest.fixture(scope="module")
def bq():
    if not os.path.exists(os.path.join(PKG, "libbq.so")):
        import __graft_entry__
        __graft_entry__.build()
    import block_quantized_moe_gather_gb300 as m
    return m


@pytest.mark.parametrize("m,n,k,status", [
    (MOST, 1, 16, NULL), (MOST + 1, 1, 16, SHAPE), (2 ** 31 - 1, 1, 16, SHAPE),
    (1, MOST, 16, NULL), (1, MOST + 1, 16, SHAPE), (1, 2 ** 31 - 1, 16, SHAPE),
    (1, 1, MOST, NULL), (1, 1, MOST + 16, SHAPE), (1, 1, 2 ** 31 - 16, SHAPE),
])
def test_products_refuse_sizes_they_cannot_count(bq, m, n, k, status):
    assert bq._lib.bq_mm_fp8_b128(None, None, m, None, None, n, k, 0, None, F16, n, None) == status
    # offsets: any address, nothing reads it
    assert bq._lib.bq_moe_mm_fp8_b128(None, None, m, 4096, 1, None, None, n, k, 0, None, F16, n, None) == status


def test_the_wait_probe_for_parts_of_a_split(bq):
    assert bq._lib.bq_test_set_wait_probe(3, 0) == 0
    for bad in (-1, 2, 4, 5):
        assert bq._lib.bq_test_set_wait_probe(bad, 0) == SHAPE
    assert bq._lib.bq_test_set_wait_probe(0, 0) == 0

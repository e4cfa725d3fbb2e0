"""The chunk arithmetic of the FP8 products (csrc/row_chunks.cuh), compiled for
the host: no GPU needed."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300", "csrc")
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def chunks(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("row_chunks")
    (d / "c.cpp").write_text(
        '#include "row_chunks.cuh"\n'
        'extern "C" int row_chunks(int rows, int most) { return bq::row_chunks(rows, most); }\n'
        'extern "C" void row_chunk(int rows, int chunks, int i, int* out) {\n'
        '    const bq::RowChunk c = bq::row_chunk(rows, chunks, i);\n'
        '    out[0] = c.first; out[1] = c.rows;\n'
        '}\n'
        'extern "C" int add_chunks(int a, int b, int limit) { return bq::add_chunks(a, b, limit); }\n')
    subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(d / "c.cpp"), "-o",
                    str(d / "c.so")], check=True)
    return ctypes.CDLL(str(d / "c.so"))


def part(lib, rows, n, i):
    out = (ctypes.c_int * 2)()
    lib.row_chunk(rows, n, i, out)
    return out[0], out[1]


@pytest.mark.parametrize("most", [32, 128])
@pytest.mark.parametrize("rows", [0, 1, 31, 32, 33, 127, 128, 129, 1000, 16385, 2 ** 30, 2 ** 31 - 2 ** 24, 2 ** 31 - 256,
                                  INT_MAX - 126, INT_MAX])
def test_chunks_cover_the_rows(chunks, rows, most):
    n = chunks.row_chunks(rows, most)
    assert n == -(-rows // most)
    if rows == 0:
        return
    # every chunk where there are few, else the first, some in the middle and the last ones
    some = range(n) if n <= 1000 else [0, 1, n // 3, n // 2, n - 2, n - 1]
    size = -(-rows // n)
    for i in some:
        first, count = part(chunks, rows, n, i)
        assert first == i * size and count == min(size, rows - first) and 1 <= count <= most


@pytest.mark.parametrize("rows", [1000, 2 ** 30, 1_100_000_000, 2 ** 31 - 256])
@pytest.mark.parametrize("experts", [3, 300, 600, 1024])
def test_sums_of_overlapping_ranges_stop_at_the_limit(chunks, rows, experts):
    """Offsets 0, rows, 0, rows, ...: every other expert has all rows.  The sums ascend, are exact up to the limit and
    stay one above it, added one after the other or as a scan does."""
    most = 128
    each = [chunks.row_chunks(rows, most) if e % 2 == 0 else 0 for e in range(experts)]
    limit = chunks.row_chunks(rows, most) + min(experts, rows)     # what ascending offsets can make
    serial, exact = [0], [0]
    for c in each:
        serial.append(chunks.add_chunks(serial[-1], c, limit))
        exact.append(exact[-1] + c)
    assert serial == [min(v, limit + 1) for v in exact]
    scan = each[:]
    off = 1
    while off < experts:
        scan = [chunks.add_chunks(scan[i], scan[i - off], limit) if i >= off else scan[i] for i in range(experts)]
        off *= 2
    assert scan == serial[1:]


def test_sums_at_the_largest_limit(chunks):
    limit = 2 ** 30 - 1
    assert chunks.add_chunks(limit + 1, limit + 1, limit) == limit + 1
    assert chunks.add_chunks(limit, 1, limit) == limit + 1 and chunks.add_chunks(limit, 0, limit) == limit

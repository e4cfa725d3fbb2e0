"""Refusals of the residual norm, the router's training calls and the products' ends (no GPU needed):
each is made on the host, before any launch; and the layout of the host structs that the binding packs."""
import ctypes
import os

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300")
P = ctypes.c_void_p(4096)         # an aligned address that no call below dereferences
ODD = ctypes.c_void_p(4104)       # 8-byte aligned only
A = 4096
OK, NULL, SHAPE, ALIGN, FORMAT, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def bq():
    if not os.path.exists(os.path.join(PKG, "libbq.so")):
        import __graft_entry__
        __graft_entry__.build()
    import block_quantized_moe_gather_gb300 as m
    return m


def desc(bq, T=4, H=64, y=F16, h=F16, x=F16, gain_t=F16, gate_t=F16, kind=0, sigmoid=0, scale=1.0, rs=1.0, eps=1e-6,
         gain=A, post=0, gate=0, ldgate=64):
    return bq._RESIDUAL_NORM_DESC.pack(T, H, y, h, x, gain_t, gate_t, kind, sigmoid, scale, rs, eps, gain, post, gate, ldgate)


def forward(bq, d, y=P, ldy=64, h=P, ldh=64, out=P, ldo=64, x=P, ldx=64):
    return bq._lib.bq_residual_norm(d, y, ldy, h, ldh, out, ldo, x, ldx, None)


@pytest.mark.parametrize("make,more,status", [
    (dict(T=-1), {}, SHAPE), (dict(H=60), {}, SHAPE), (dict(H=0), {}, SHAPE), (dict(H=16392), {}, SHAPE),
    (dict(y=3), {}, FORMAT), (dict(h=-1), {}, FORMAT), (dict(x=7), {}, FORMAT), (dict(gain_t=9), {}, FORMAT),
    (dict(kind=4), {}, SHAPE), (dict(sigmoid=2), {}, SHAPE), (dict(kind=2, gate_t=5, gate=A), {}, FORMAT),
    (dict(eps=-1.0), {}, SHAPE), (dict(eps=float("nan")), {}, SHAPE), (dict(eps=float("inf")), {}, SHAPE),
    (dict(gain=0), {}, NULL), (dict(kind=1), {}, NULL), (dict(gain=A + 8), {}, ALIGN), (dict(post=A + 2), {}, ALIGN),
    (dict(kind=2, gate=A + 8), {}, ALIGN), (dict(kind=1, gate=A + 1), {}, ALIGN),
    (dict(kind=3, gate=A, ldgate=56), {}, SHAPE), (dict(kind=3, gate=A, ldgate=68), {}, ALIGN),
    ({}, dict(y=None), NULL), ({}, dict(h=ODD), ALIGN), ({}, dict(out=None), NULL), ({}, dict(ldx=8), SHAPE),
    ({}, dict(ldy=68), ALIGN), ({}, dict(ldh=1 << 36), SHAPE),
    (dict(T=0, gain=0), dict(y=None, h=None, out=None, x=None), OK),
])
def test_residual_norm_is_refused(bq, make, more, status):
    assert forward(bq, desc(bq, **make), **more) == status
    if status != OK:
        assert bq.last_error()


def backward(bq, d, y=P, h=P, dh_out=P, dx=P, dy=P, dh=P, dgain=None, dpost=None, dgate=None, ld=64, ws=None, n=0):
    return bq._lib.bq_residual_norm_backward(d, y, ld, h, ld, dh_out, ld, dx, ld, dy, ld, dh, ld, dgain, dpost, dgate, ld, ws,
                                             n, None)


@pytest.mark.parametrize("make,more,status", [
    ({}, dict(dx=None, dh_out=None), NULL), ({}, dict(dy=None), NULL), ({}, dict(dh=None), NULL), ({}, dict(h=None), NULL),
    ({}, dict(dgain=P), WORKSPACE), ({}, dict(dgain=P, ws=P, n=100), WORKSPACE), ({}, dict(dgain=P, ws=ODD, n=1 << 20), ALIGN),
    ({}, dict(dgain=ctypes.c_void_p(4098), ws=P, n=1 << 20), ALIGN), ({}, dict(dgain=P, dx=None), NULL),
    ({}, dict(dpost=P), NULL), ({}, dict(dgate=P), NULL), (dict(kind=3, gate=A), dict(dgate=ODD), ALIGN),
    (dict(kind=2, gate=A), dict(dgate=P), WORKSPACE), (dict(T=0), dict(y=None, h=None, dy=None, dh=None), OK),
])
def test_residual_norm_backward_is_refused(bq, make, more, status):
    assert backward(bq, desc(bq, **make), **more) == status


def test_a_null_descriptor(bq):
    assert forward(bq, None) == NULL and backward(bq, None) == NULL


def balance(bq, logits=P, bias=None, T=4, E=16, ids=P, k=2, scoring=0, off=None, S=1, counts=P, probs=P, losses=P, ws=P,
            n=1 << 30):
    return bq._lib.bq_moe_balance_loss(logits, bias, T, E, ids, k, scoring, off, S, counts, probs, losses, ws, n, None)


@pytest.mark.parametrize("more,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=9), SHAPE),
    (dict(E=4, k=5), SHAPE), (dict(T=2 ** 30, k=8), SHAPE), (dict(scoring=3), SHAPE), (dict(S=0), SHAPE), (dict(S=2), SHAPE),
    (dict(off=P, S=65537), SHAPE), (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(counts=None), NULL),
    (dict(probs=None), NULL), (dict(losses=None), NULL), (dict(bias=P, scoring=1), SHAPE), (dict(ws=None), WORKSPACE),
    (dict(n=64), WORKSPACE), (dict(ws=ctypes.c_void_p(4112)), ALIGN), (dict(ids=ctypes.c_void_p(4098)), ALIGN)])
def test_balance_is_refused(bq, more, status):
    assert balance(bq, **more) == status


def gradient(bq, logits=P, bias=None, T=4, E=16, ids=P, k=2, scoring=0, scale=1.0, dw=P, counts=None, dl=None, off=None, S=1,
             d=P, dtype=F32, db=None, ws=None, n=0):
    return bq._lib.bq_moe_route_backward(logits, bias, T, E, ids, k, scoring, scale, dw, counts, dl, off, S, d, dtype, db, ws,
                                         n, None)


@pytest.mark.parametrize("more,status", [
    (dict(dtype=3), FORMAT), (dict(dw=None), NULL), (dict(dl=P), NULL), (dict(ids=None), NULL), (dict(d=None), NULL),
    (dict(d=ctypes.c_void_p(4098)), ALIGN), (dict(db=P), WORKSPACE), (dict(db=P, scoring=2), SHAPE),
    (dict(bias=P, scoring=1), SHAPE), (dict(k=9), SHAPE), (dict(S=3), SHAPE), (dict(T=0, logits=None, ids=None, d=None), OK)])
def test_route_backward_is_refused(bq, more, status):
    assert gradient(bq, **more) == status


def test_workspace_queries(bq):
    assert bq.residual_norm_backward_workspace_bytes(4, 60) == 0 and bq.residual_norm_backward_workspace_bytes(-1, 64) == 0
    assert bq.residual_norm_backward_workspace_bytes(0, 64) > 0
    assert bq.moe_balance_workspace_bytes(10, 0, 1) == 0 and bq.moe_balance_workspace_bytes(10, 8, 0) == 0
    assert bq.moe_route_backward_workspace_bytes(10, 1025) == 0 and bq.moe_route_backward_workspace_bytes(0, 8) > 0


def product(bq, epi, m=4, n=256, k=64, dtype=F16, ldy=256, y=P):
    return bq._lib.bq_mm_fp8_b128_epilogue(P, P, m, P, P, n, k, epi, y, dtype, ldy, None)


@pytest.mark.parametrize("epi,more,status", [
    (None, {}, NULL), ((7, 1.0, 0, 0, 0), {}, SHAPE), ((-1, 1.0, 0, 0, 0), {}, SHAPE), ((1, 1.0, A, 0, 0), dict(n=128), SHAPE),
    ((2, 1.0, A + 2, 0, 0), {}, ALIGN), ((2, 1.0, 0, A + 1, 256), {}, ALIGN), ((2, 1.0, 0, A, 255), {}, SHAPE),
    ((1, 1.0, 0, A, 127), dict(ldy=128), SHAPE), ((2, 1.0, A, A, 256), dict(dtype=4), FORMAT), ((2, 1.0, A, 0, 0), dict(m=0), OK)])
def test_ends_are_refused(bq, epi, more, status):
    assert product(bq, None if epi is None else bq._EPILOGUE.pack(*epi), **more) == status
    if epi is not None and status == SHAPE:
        assert bq.last_error().startswith("bq_mm_fp8_b128_epilogue")


def test_host_structs_have_the_size_that_the_header_gives(bq, tmp_path):
    """The packed layouts against the compiler's."""
    import shutil
    import subprocess
    cc = shutil.which("cc") or shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "bq.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(bq_epilogue), '
                   'offsetof(bq_epilogue, residual), offsetof(bq_epilogue, ldr), sizeof(bq_residual_norm_desc), '
                   'offsetof(bq_residual_norm_desc, scale), offsetof(bq_residual_norm_desc, ldgate)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run([cc, "-I", os.path.join(os.path.dirname(PKG), "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [bq._EPILOGUE.size, 16, 24, bq._RESIDUAL_NORM_DESC.size, 36, 72]


def test_more_rows_than_an_int_steps_over_are_refused(bq):
    n = 2 ** 31 - 1
    assert balance(bq, T=n, E=1, k=1, n=1 << 40) == SHAPE
    assert gradient(bq, T=n, E=1, k=1) == SHAPE
    assert bq.moe_balance_workspace_bytes(n, 1, 1) == 0 and bq.moe_route_backward_workspace_bytes(n, 1) == 0
    assert bq.moe_balance_workspace_bytes(n - 64, 1, 1) > 0

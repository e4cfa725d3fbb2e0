"""GPU: the activations of the FP8 products' ends by themselves: rows of zeros, so that a product's value is its bias,
to the bit, and y = act(bias) in fp32.

Bounds (u = 2^-24, relative to the value, as the header states them).  exp2 and reciprocal are off by 4 u each, a
rounding by u; the exponent's argument w comes with two or three roundings, so that exp is off by 2.2 u |w| at most with
|w| = |v| (silu), v^2 / 2 (gelu), or the argument of the tanh form, whose sum of two products adds as much again.
gelu's polynomial with its own roundings is 8 u.  A reciprocal or an exponential below 2^-126 becomes 0, and with it a
result of up to 90 times as much."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUB = 2.0 ** -119


def values():
    """Dense from -14 to 14, around 0, and far from it, as fp32; a multiple of 256 of them."""
    v = np.concatenate([np.linspace(-14, 14, 30001), np.linspace(-100, 100, 4001), [0.0, -0.0, 1e30, -1e30],
                        np.geomspace(1e-30, 1, 2000), -np.geomspace(1e-30, 1, 2000)]).astype(np.float32)
    return np.concatenate([v, np.ones(-len(v) % 256, dtype=np.float32)])


def relative(act, v):
    if act == "silu":
        return 16 + 2.2 * np.abs(v)
    if act == "gelu":
        return 24 + 2.2 * 0.5 * v * v
    return 16 + 8 * np.abs(1.6 * (v + 0.045 * v ** 3))


def run(lib, m, act, bias, residual=False):
    import torch
    n, k = len(bias), 16
    zeros = (lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda"))
    b = torch.from_numpy(bias).cuda()
    cols = n // 2 if act == "swiglu" else n
    y = torch.full((m, cols), 7.0, device="cuda")
    lib.mm_fp8_b128(zeros(m, k), torch.ones(m, 1, device="cuda"), zeros(n, k), torch.ones(-(-n // 128), 1, device="cuda"), y,
                    act=act, bias=b, residual=torch.zeros_like(y) if residual else None)
    assert (y == y[:1]).all() or torch.isnan(y).any()
    return y[0].double().cpu().numpy()


@pytest.mark.parametrize("m,residual", [(1, False), (1, True), (200, False), (200, True)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_relative_error(lib, act, m, residual):
    v = values()
    got = run(lib, m, act, v, residual)
    v = v.astype(np.float64)
    with np.errstate(over="ignore"):
        want = O.activation(v, act)
        off = np.abs(got - want)
        limit = relative(act, np.clip(v, -200, 200)) * U * np.abs(want) + SUB
    assert (off <= limit).all(), f"{v[np.argmax(off / limit)]}: {np.max(off / limit)} of the bound"


@pytest.mark.parametrize("m", [1, 200])
def test_relative_error_of_swiglu(lib, m):
    v = values()
    up = np.random.default_rng(1).uniform(0.5, 2, len(v)).astype(np.float32)
    got = run(lib, m, "swiglu", np.concatenate([v, up]))
    v = v.astype(np.float64)
    want = O.activation(v, "silu") * up
    off = np.abs(got - want)
    limit = (1 + relative("silu", np.clip(v, -200, 200))) * U * np.abs(want) + 2 * SUB
    assert (off <= limit).all(), f"{v[np.argmax(off / limit)]}: {np.max(off / limit)} of the bound"


@pytest.mark.parametrize("m", [1, 200])
def test_infinities_and_nan(lib, m):
    v = np.ones(256, dtype=np.float32)
    v[:3] = np.inf, -np.inf, np.nan
    for act in ("silu", "gelu", "gelu_tanh", "relu", "relu2"):
        got = run(lib, m, act, v)
        assert got[0] == np.inf and np.isnan(got[2]) and np.isfinite(got[3:]).all()
        assert not got[1] > 0
        if act in ("gelu", "relu", "relu2"):
            assert got[1] == 0


@pytest.mark.parametrize("dtype,rows", [("f32", 1), ("bf16", 3), ("f32", 700)])
def test_relative_error_of_the_gates_sigmoid(lib, dtype, rows):
    """A stream of zeros and a block's output of ones: h_out is the gate's sigmoid."""
    import torch
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    v = torch.from_numpy(np.concatenate([np.linspace(-100, 100, 4000), np.linspace(-2, 2, 4096)]).astype(np.float32)).cuda()
    gate = v.expand(rows, -1).to(dt).contiguous()
    out = torch.empty(rows, v.numel(), device="cuda")
    lib.residual_norm(torch.ones_like(out), torch.zeros_like(out), out, gate=gate, gate_sigmoid=True)
    lib.device_status()
    v = gate[0].double().cpu().numpy()
    want, got = O.sigmoid(v), out.double().cpu().numpy()
    assert (np.abs(got - want) <= (16 + 2.2 * np.abs(v)) * U * want + 2.0 ** -126).all()

"""GPU parity of the norms between two blocks and their gradients against the fp64 oracle.

Tolerances (u = 2^-24, the fp32 half step; e = half step of an output's type).
A sum over a row adds at most 64 values in a thread, 5 in a butterfly and 32
over warps and CTAs, so a sum of n terms is off by at most 128 u sum|terms|, and
1 / rms, whose terms are all positive, by 64 u and the 2 u of rsqrtf.  With the
few products and the sigmoid (4 u and 2 u of the gate's magnitude, 16 u here) behind it:
  h':  96 u (|residual_scale h| + |scale g b|) + e |h'|
  x:   gain / rms * (bound of h' before rounding) + |x| (96 u + the rms of that
       bound over the rms of h') + e |x|
Backward, with A = |dh'| + |r gain dx| + |h' r^3| mean|gain dx h'| and
B = s |post g| scale A + |y s^3| mean(post scale |g| A |y|):
  dh:  400 u |residual_scale| A + e |dh|      (r^3: 200 u; the mean: 128 u; products)
  dy:  900 u B + e |dy|                       (the same over D, s^3 and its mean)
  sums over rows add up to 40 rows in a thread, 512 / 16 parts and 16 warps: 128 u;
  dgain: 256 u sum|dx h' r|;  dpost: 700 u sum|scale g| A |y s|;  dgate: 700 u sum scale A |b| (+ e)"""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 2.0 ** -148, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def made(g, shape, dtype, add=0.0, times=1.0):
    import torch
    t = torch.from_numpy((add + times * g.standard_normal(shape)).astype(np.float32)).to(torch_dtype(dtype))
    return t.cuda(), t.double().numpy()


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, bound, dtype, what):
    got = f64(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    limit = bound * 1.001 + HALF[dtype] * np.abs(want) + SUB[dtype]
    assert np.isfinite(got).all() and (off <= limit).all(), f"{what}: {np.max(off / limit)} of the bound"


class Case:
    def __init__(self, seed, t, h, types, gain, post, gate, sig, scale, residual_scale):
        g = np.random.default_rng(seed)
        self.types, self.t, self.h, self.gate_kind = types, t, h, gate
        ty, th, tx = types
        self.y, self.y64 = made(g, (t, h), ty, times=1.5)
        self.h_in, self.h64 = made(g, (t, h), th, times=2.0)
        self.gain, self.gain64 = made(g, h, gain, 1.0, 0.2)
        self.post, self.post64 = made(g, h, gain, 1.0, 0.2) if post else (None, None)
        shape, self.gate_type = {"none": (None, None), "token": ((t, 1), "f32"), "channel": ((h,), gain),
                                 "full": ((t, h), ty)}[gate]
        self.gate, self.gate64 = (None, None) if gate == "none" else made(g, shape, self.gate_type)
        self.more = dict(scale=scale, residual_scale=residual_scale, eps=1e-5)
        self.sig = sig
        self.dh_out, self.dh64 = made(g, (t, h), th)
        self.dx, self.dx64 = made(g, (t, h), tx)

    def args(self):
        return dict(gain=self.gain, post_gain=self.post, gate=self.gate, gate_sigmoid=self.sig, **self.more)

    def factor(self):
        return 1.0 if self.gate is None else np.abs(O.sigmoid(self.gate64) if self.sig else self.gate64)


def check_forward(lib, c):
    import torch
    out, x = torch.full_like(c.h_in, np.nan), torch.full((c.t, c.h), np.nan, dtype=torch_dtype(c.types[2]), device="cuda")
    got = lib.residual_norm(c.y, c.h_in, out, x, **c.args())
    assert got[0] is out and got[1] is x
    want, want_x = O.residual_norm(c.y64, c.h64, c.gain64, c.post64, c.gate64, c.sig, **c.more)
    rs, sc = c.more["residual_scale"], c.more["scale"]
    off = 96 * U * (np.abs(rs * c.h64) + np.abs(want - rs * c.h64))
    close(out, want, off, c.types[1], "h_out")
    inv = 1 / np.sqrt(np.mean(want ** 2, axis=1, keepdims=True) + c.more["eps"])
    spread = np.sqrt(np.mean(off ** 2, axis=1, keepdims=True)) * inv
    close(x, want_x, np.abs(c.gain64) * inv * off + np.abs(want_x) * (96 * U + spread), c.types[2], "x")
    assert sc is not None
    return out


def check_backward(lib, c, h_out, with_dx=True, with_dh=True):
    import torch
    h64, eps = f64(h_out), c.more["eps"]
    dy, dh = torch.full_like(c.y, np.nan), torch.full_like(c.h_in, np.nan)
    new = (lambda *s: torch.full(s, np.nan, device="cuda"))
    dgain = new(c.h) if with_dx else None
    dpost = new(c.h) if c.post is not None else None
    dgate = None
    if c.gate is not None:
        dgate = torch.full_like(c.gate, np.nan, dtype=c.gate.dtype if c.gate_kind == "full" else torch.float32)
    ws = torch.full((lib.residual_norm_backward_workspace_bytes(c.t, c.h),), 255, dtype=torch.uint8, device="cuda")
    lib.residual_norm_backward(c.y, h_out if with_dx else None, c.dh_out if with_dh else None, c.dx if with_dx else None,
                               dy, dh, **(c.args() if with_dx else dict(c.args(), gain=None)), dgain=dgain,
                               dpost_gain=dpost, dgate=dgate, workspace=ws)
    want = O.residual_norm_backward(c.y64, h64, c.dh64 if with_dh else None, c.dx64 if with_dx else None, c.gain64, c.post64,
                                    c.gate64, c.sig, **c.more)
    r = 1 / np.sqrt(np.mean(h64 ** 2, axis=1, keepdims=True) + eps)
    s = 1 / np.sqrt(np.mean(c.y64 ** 2, axis=1, keepdims=True) + eps)
    size = np.abs(c.dh64) if with_dh else np.zeros((c.t, c.h))
    if with_dx:
        gd = np.abs(c.gain64 * c.dx64)
        size = size + r * gd + np.abs(h64) * r ** 3 * np.mean(gd * np.abs(h64), axis=1, keepdims=True)
    sc, rs = abs(c.more["scale"]), abs(c.more["residual_scale"])
    close(dh, want["dh"], 400 * U * rs * size, c.types[1], "dh")
    d = sc * c.factor() * size
    if c.post is None:
        close(dy, want["dy"], 900 * U * d, c.types[0], "dy")
        b = np.abs(c.y64)
    else:
        pd, ay = np.abs(c.post64) * d, np.abs(c.y64)
        close(dy, want["dy"], 900 * U * (s * pd + ay * s ** 3 * np.mean(pd * ay, axis=1, keepdims=True)), c.types[0], "dy")
        close(dpost, want["dpost_gain"], 700 * U * (d * ay * s).sum(axis=0), "f32", "dpost_gain")
        b = np.abs(c.post64) * ay * s
    if with_dx:
        close(dgain, want["dgain"], 256 * U * np.abs(c.dx64 * h64 * r).sum(axis=0), "f32", "dgain")
    if c.gate is not None:
        size = sc * size * b * (O.sigmoid(c.gate64) if c.sig else 1.0)   # sigmoid' <= sigmoid
        if c.gate_kind != "full":
            size = size.sum(axis=1, keepdims=True) if c.gate_kind == "token" else size.sum(axis=0)
        close(dgate, want["dgate"], 700 * U * size, c.gate_type if c.gate_kind == "full" else "f32", "dgate")
    return [t for t in (dy, dh, dgain, dpost, dgate) if t is not None]


TYPES = [("f16",) * 3, ("bf16",) * 3, ("f32",) * 3, ("f32", "f16", "f16"), ("bf16", "f32", "bf16"), ("f16", "bf16", "f32")]
SIZES = [(1, 4096), (7, 8), (3, 264), (33, 2048), (517, 136), (5, 4104), (2, 16384), (9, 8200)]


@pytest.mark.parametrize("t,h", SIZES)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_sizes_and_types(lib, t, h, types):
    n = t + h
    c = Case(n, t, h, types, types[2] if n % 2 else "f32", n % 3 != 0, ["none", "token", "channel", "full"][n % 4], n % 5 < 2,
             0.5, 1.25)
    check_backward(lib, c, check_forward(lib, c))


@pytest.mark.parametrize("gate,sig", [("none", False)] + [(g, s) for g in ("token", "channel", "full") for s in (False, True)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("t,h,types", [(37, 512, TYPES[1]), (700, 1024, TYPES[4]), (1, 40, TYPES[3]), (41, 10000, TYPES[2])])
def test_gates_and_norms(lib, gate, sig, post, t, h, types):
    c = Case(t + 2 * post, t, h, types, "bf16", post, gate, sig, 0.25, 1.0)
    out = check_forward(lib, c)
    for with_dx, with_dh in ((True, True), (True, False), (False, True)):
        check_backward(lib, c, out, with_dx, with_dh)


@pytest.mark.parametrize("types", [TYPES[2], TYPES[4], TYPES[5]], ids="-".join)
@pytest.mark.parametrize("t,h,gate,post", [(330, 8192, "full", True), (400, 4096, "full", True), (310, 8192, "channel", True),
                                           (311, 8200, "full", True), (305, 2056, "token", False), (900, 64, "full", True)])
def test_many_wide_rows(lib, types, t, h, gate, post):
    """Rows of which few, or none ahead, fit into shared memory; more rows than blocks."""
    c = Case(t, t, h, types, "f32", post, gate, True, 0.5, 1.0)
    check_backward(lib, c, check_forward(lib, c))


@pytest.mark.parametrize("h", [4096, 9000])
@pytest.mark.parametrize("which", ["y", "h"])
def test_gradients_of_tiny_rows_without_eps(lib, which, h):
    """1 / rms is 2^45: its cube leaves fp32's range, what it is multiplied with brings the product back."""
    c = Case(3, 9, h, TYPES[2], "f32", True, "channel", True, 0.5, 1.25)
    c.more["eps"] = 0.0
    if which == "y":
        c.y, c.y64 = c.y * 2.0 ** -46, c.y64 * 2.0 ** -46
    else:
        c.h_in, c.h64 = c.h_in * 2.0 ** -46, c.h64 * 2.0 ** -46
    check_backward(lib, c, c.h_in)


@pytest.mark.parametrize("types", [TYPES[1], TYPES[3], TYPES[5]], ids="-".join)
@pytest.mark.parametrize("t,h,gate,post", [(40001, 64, "token", True), (5003, 520, "channel", False), (1301, 2056, "full", True),
                                           (622, 4104, "none", True), (313, 8000, "token", False)])
def test_more_rows_than_fit_at_once(lib, types, t, h, gate, post):
    """Blocks of one to eight rows that walk over the rows, and end inside a block's rows."""
    check_forward(lib, Case(t, t, h, types, types[2], post, gate, True, 0.5, 1.25))


def test_many_rows_of_few_values(lib):
    c = Case(5, 9001, 72, TYPES[4], "f32", True, "channel", True, 0.5, 1.0)
    check_backward(lib, c, check_forward(lib, c))


def test_a_prefill_batch(lib):
    c = Case(1, 2047, 4096, TYPES[1], "bf16", True, "channel", False, 1.0, 1.0)
    out = check_forward(lib, c)
    first = check_backward(lib, c, out)
    for a, b in zip(first, check_backward(lib, c, out)):
        assert (a == b).all()       # the same bits again


def test_strides_and_in_place(lib):
    import torch
    c = Case(4, 19, 256, TYPES[1], "bf16", True, "full", True, 0.5, 1.0)
    plain = lib.residual_norm(c.y, c.h_in, torch.empty_like(c.h_in), torch.empty_like(c.y), **c.args())

    def wide(t):
        w = torch.full((t.shape[0] + 1, t.shape[1] + 24), 7.0, dtype=t.dtype, device="cuda")
        v = w[:-1, 8:8 + t.shape[1]]
        v.copy_(t)
        return w, v

    (_, y), (hw, h), (_, gate), (xw, x) = wide(c.y), wide(c.h_in), wide(c.gate), wide(torch.zeros_like(c.y))
    lib.residual_norm(y, h, h, x, **dict(c.args(), gate=gate))          # h_out is h
    assert (h == plain[0]).all() and (x == plain[1]).all()
    for w in (hw, xw):                                                     # nothing beside the rows was written
        assert (w[-1] == 7).all() and (w[:, :8] == 7).all() and (w[:, 8 + 256:] == 7).all()

    def back(y, h_out, dh_out, dx, dy, dh, gate, dgate):
        dg, dp = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
        ws = torch.empty(lib.residual_norm_backward_workspace_bytes(19, 256), dtype=torch.uint8, device="cuda")
        lib.residual_norm_backward(y, h_out, dh_out, dx, dy, dh, **dict(c.args(), gate=gate), dgain=dg, dpost_gain=dp,
                                   dgate=dgate, workspace=ws)
        return dy, dh, dg, dp, dgate

    e = torch.empty_like
    want = back(c.y, plain[0], c.dh_out, c.dx, e(c.y), e(c.h_in), c.gate, e(c.gate))
    (dyw, dy), (dgw, dgate), (dhw, dh) = wide(c.y), wide(c.gate), wide(c.dh_out)
    got = back(y, h, dh, wide(c.dx)[1], dy, dh, gate, dgate)               # dh is dh_out
    for a, b in zip(want, got):
        assert (a == b).all()
    for w in (dyw, dgw, dhw):
        assert (w[-1] == 7).all() and (w[:, :8] == 7).all() and (w[:, 8 + 256:] == 7).all()


@pytest.mark.parametrize("t,h", [(400, 8192), (320, 16384)])
def test_wide_rows_in_place(lib, t, h):
    """Rows fetched ahead (one at a time, and by a cluster) are not those that are written."""
    import torch
    c = Case(t, t, h, TYPES[2], "f32", True, "channel", True, 0.5, 1.0)
    e = torch.empty_like
    out, x = lib.residual_norm(c.y, c.h_in, e(c.h_in), e(c.y), **c.args())
    ws = torch.empty(lib.residual_norm_backward_workspace_bytes(t, h), dtype=torch.uint8, device="cuda")

    def back(dh):
        sums = [torch.full((h,), np.nan, device="cuda") for _ in range(3)]
        dy, _ = lib.residual_norm_backward(c.y, out, c.dh_out, c.dx, e(c.y), dh, **c.args(), dgain=sums[0], dpost_gain=sums[1],
                                           dgate=sums[2], workspace=ws)
        return [dy, dh, *sums]

    want = back(e(c.dh_out))
    for a, b in zip(want, back(c.dh_out)):      # dh is dh_out
        assert (a == b).all()
    lib.residual_norm(c.y, c.h_in, c.h_in, x2 := e(x), **c.args())      # h_out is h
    assert (c.h_in == out).all() and (x2 == x).all()


def test_no_rows_and_no_x(lib):
    import torch
    h, h_out = torch.randn(4, 64, device="cuda"), torch.empty(4, 64, device="cuda")
    y = torch.randn(4, 64, device="cuda")
    assert lib.residual_norm(y, h, h_out)[1] is None
    torch.testing.assert_close(h_out, h + y, rtol=2 * U, atol=0)
    empty = torch.empty(0, 64, device="cuda")
    lib.residual_norm(empty, empty, empty, empty, gain=torch.ones(64, device="cuda"))
    dgain, dgate = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    ws = torch.empty(lib.residual_norm_backward_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    lib.residual_norm_backward(empty, empty, empty, empty, empty, empty, gain=torch.ones(64, device="cuda"),
                               gate=torch.ones(64, device="cuda"), dgain=dgain, dgate=dgate, workspace=ws)
    assert not dgain.any() and not dgate.any()


def test_infinities_and_nan_stay_in_their_rows(lib):
    import torch
    c = Case(8, 6, 512, TYPES[2], "f32", True, "token", True, 1.0, 1.0)
    out, x = torch.empty_like(c.h_in), torch.empty_like(c.y)
    lib.residual_norm(c.y, c.h_in, out, x, **c.args())
    y = c.y.clone()
    y[2, 5], y[4, 7] = np.nan, np.inf
    out2, x2 = torch.empty_like(out), torch.empty_like(x)
    lib.residual_norm(y, c.h_in, out2, x2, **c.args())
    for r in range(6):
        if r in (2, 4):
            assert not torch.isfinite(x2[r]).all()
        else:
            assert (out2[r] == out[r]).all() and (x2[r] == x[r]).all()


def test_captured_and_on_another_stream(lib):
    import torch
    c = Case(9, 65, 1024, TYPES[3], "f16", True, "channel", True, 0.5, 1.0)
    out, x = torch.empty_like(c.h_in), torch.empty(65, 1024, dtype=torch.float16, device="cuda")
    dy, dh = torch.empty_like(c.y), torch.empty_like(c.h_in)
    dg, dp, dgate = (torch.empty(1024, device="cuda") for _ in range(3))
    ws = torch.empty(lib.residual_norm_backward_workspace_bytes(65, 1024), dtype=torch.uint8, device="cuda")

    def both():
        lib.residual_norm(c.y, c.h_in, out, x, **c.args())
        lib.residual_norm_backward(c.y, out, c.dh_out, c.dx, dy, dh, **c.args(), dgain=dg, dpost_gain=dp, dgate=dgate,
                                   workspace=ws)

    outputs = (out, x, dy, dh, dg, dp, dgate)
    both()
    want = [t.clone() for t in outputs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in outputs:
        t.fill_(3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            graph.replay()
    side.synchronize()
    assert all((a == b).all() for a, b in zip(outputs, want))
    for t in outputs:
        t.fill_(3.0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    assert all((a == b).all() for a, b in zip(outputs, want))


def test_refusals(lib):
    import torch
    rows, gain = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    new = torch.empty_like
    with pytest.raises(lib.BQError, match="gain is NULL"):
        lib.residual_norm(rows, rows, new(rows), new(rows))
    with pytest.raises(lib.BQError, match="FORMAT"):
        lib.residual_norm(rows, rows, new(rows), new(rows), gain=gain, post_gain=gain.half())
    with pytest.raises(lib.BQError, match="gate has shape"):
        lib.residual_norm(rows, rows, new(rows), new(rows), gain=gain, gate=torch.ones(4, 2, device="cuda"))
    with pytest.raises(lib.BQError, match="multiple of 8"):
        lib.residual_norm(rows[:, :60], rows[:, :60], new(rows)[:, :60])
    with pytest.raises(lib.BQError, match="both NULL"):
        lib.residual_norm_backward(rows, rows, None, None, new(rows), new(rows), gain=gain)
    with pytest.raises(lib.BQError, match="WORKSPACE"):
        lib.residual_norm_backward(rows, rows, rows, rows, new(rows), new(rows), gain=gain, dgain=new(gain))
    with pytest.raises(lib.BQError, match="without what it belongs to"):
        lib.residual_norm_backward(rows, rows, rows, None, new(rows), new(rows), gain=gain, dgain=new(gain))
    with pytest.raises(lib.BQError, match="dgate has shape"):
        lib.residual_norm_backward(rows, rows, rows, rows, new(rows), new(rows), gain=gain, dgate=new(gain))

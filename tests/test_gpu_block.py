"""GPU: the operators of a block run together as a program runs them, and at sizes beyond 32-bit offsets.

Tolerances.  Serving: against the same steps as separate calls whose 32-bit
results go through 64-bit arithmetic, so that only the fused step's own fp32
roundings (below 64 u of the magnitudes) and the half step of the 16-bit result
are left; fp16 intermediate rows are the fused calls' own.  Training: central
differences of the 64-bit loss, whose error (step^2) is below 1e-6 of it, against
fp32 gradients of sums of 64 to 4096 terms, 1e-4 of the magnitudes."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def fp8_weight(g, *shape):
    import torch
    w = torch.from_numpy((g.standard_normal(shape) * 60).clip(-448, 448).astype(np.float32)).to(torch.float8_e4m3fn).cuda()
    blocks = shape[:-2] + (-(-shape[-2] // 128), -(-shape[-1] // 128))
    return w, dev(g.uniform(2e-4, 6e-4, blocks).astype(np.float32))


@pytest.mark.parametrize("t", [1, 7, 400])
def test_a_block_of_an_fp16_stream(lib, t):
    """norm -> FP8 rows -> first projection (bias, gelu) -> FP8 rows -> last projection into the stream -> next norm,
    then experts with biases from router to combine; the dense part and the experts against separate calls."""
    import torch
    g = np.random.default_rng(t)
    H, F, E, k, I = 512, 1024, 16, 4, 256
    half = (lambda *s: dev(g.standard_normal(s).astype(np.float16)))
    h, y0 = half(t, H), dev(g.standard_normal((t, H)).astype(np.float32))     # y0: a layer's fp32 output
    gain = dev((1 + 0.1 * g.standard_normal(H)).astype(np.float16))
    w1, s1 = fp8_weight(g, F, H)
    w2, s2 = fp8_weight(g, H, F)
    b1, b2 = dev(g.standard_normal(F).astype(np.float32)), dev(g.standard_normal(H).astype(np.float32))
    x = torch.empty_like(h)
    stream = torch.empty_like(h)
    lib.residual_norm(y0, h, stream, x, gain=gain, scale=0.5)

    def quantised(rows):
        q = torch.empty(rows.shape, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(rows.shape[0], -(-rows.shape[1] // 128), device="cuda")
        lib.quant_fp8_b128(rows, q, s)
        return q, s

    up = torch.empty(t, F, dtype=torch.float16, device="cuda")
    lib.mm_fp8_b128(*quantised(x), w1, s1, up, act="gelu", bias=b1)
    plain = torch.empty(t, F, device="cuda")
    lib.mm_fp8_b128(*quantised(x), w1, s1, plain)
    want = O.product_end(f64(plain), f64(b1), "gelu")
    size = np.abs(f64(plain)) + np.abs(f64(b1))
    assert (np.abs(f64(up) - want) <= 64 * U * size + 2.0 ** -11 * np.abs(want) + 2.0 ** -24).all()
    before = stream.clone()
    down = torch.empty(t, H, device="cuda")
    lib.mm_fp8_b128(*quantised(up), w2, s2, down)
    lib.mm_fp8_b128(*quantised(up), w2, s2, stream, bias=b2, residual=stream, scale=0.5)
    want = O.product_end(f64(down), f64(b2), "none", 0.5, f64(before))
    size = np.abs(f64(down)) + np.abs(f64(b2)) + np.abs(f64(before))
    assert (np.abs(f64(stream) - want) <= 64 * U * size + 2.0 ** -11 * np.abs(want) + 2.0 ** -24).all()

    # the experts: route, sort, gate/up and down with biases, combine, back into the stream under a gate per token
    wr = dev((g.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32))
    logits = x.float() @ wr.t()
    ids, weights = torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(t, k, device="cuda")
    lib.moe_route(logits, None, k, ids, weights)
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    tok, slot, inv = (torch.empty(t * k, dtype=torch.int32, device="cuda") for _ in range(3))
    ws = torch.empty(lib.moe_permute_workspace_bytes(t, k, E), dtype=torch.uint8, device="cuda")
    lib.moe_permute(ids, E, counts, offsets, tok, slot, inv, ws)
    q = torch.empty(t * k, H, dtype=torch.float8_e4m3fn, device="cuda")
    qs = torch.empty(t * k, H // 128, device="cuda")
    lib.moe_dispatch_fp8_b128(x, inv, q, qs)
    wg, sg = fp8_weight(g, E, 2 * I, H)
    wd, sd = fp8_weight(g, E, H, I)
    bg, bd = dev(g.standard_normal((E, 2 * I)).astype(np.float32)), dev(g.standard_normal((E, H)).astype(np.float32))
    act = torch.empty(t * k, I, dtype=torch.bfloat16, device="cuda")
    lib.moe_mm_fp8_b128(q, qs, offsets, wg, sg, act, act="swiglu", bias=bg)
    plain = torch.empty(t * k, 2 * I, device="cuda")
    lib.moe_mm_fp8_b128(q, qs, offsets, wg, sg, plain)
    expert = np.repeat(np.arange(E), counts.cpu().numpy())
    v = f64(plain) + f64(bg)[expert]
    want = O.activation(v, "swiglu")
    size = (1 + np.abs(v[:, :I])) * (1 + np.abs(v[:, I:]))
    assert (np.abs(f64(act) - want) <= 64 * U * size + 2.0 ** -8 * np.abs(want) + 2.0 ** -24).all()
    ys, yc = torch.empty(t * k, H, device="cuda"), torch.empty(t, H, device="cuda")
    q, qs = quantised(act)
    lib.moe_mm_fp8_b128(q, qs, offsets, wd, sd, ys, bias=bd)
    lib.moe_combine(ys, inv, weights, yc)
    gate = dev(g.standard_normal((t, 1)).astype(np.float32))
    out, x2 = torch.empty_like(stream), torch.empty_like(stream)
    lib.residual_norm(yc, stream, out, x2, gain=gain, gate=gate, gate_sigmoid=True)
    want, want_x = O.residual_norm(f64(yc), f64(stream), f64(gain), None, f64(gate), True)
    size = np.abs(f64(yc)) + np.abs(f64(stream))
    assert (np.abs(f64(out) - want) <= 96 * U * size + 2.0 ** -11 * np.abs(want) + 2.0 ** -24).all()
    np.testing.assert_allclose(f64(x2), want_x, rtol=2.0 ** -10, atol=2e-5)
    # the statistics of the same routing
    probs, losses, c = torch.empty(1, E, device="cuda"), torch.empty(2, device="cuda"), torch.empty(1, E, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.moe_balance_workspace_bytes(t, E), dtype=torch.uint8, device="cuda")
    lib.moe_balance_loss(logits, ids, c, probs, losses, ws)
    assert torch.equal(c[0], counts)                  # the same counts that the sort found
    assert lib.device_status() == lib.DEV_OK


@pytest.mark.parametrize("rule", ["softmax", "softmax_then_bias", "sqrtsoftplus"])
def test_training_gradients_against_differences(lib, rule):
    """From the gradients of a block's outputs back to the logits of its router, the expert outputs, the gate and the
    gains: every call of the library in turn, against central differences of the whole in 64 bits."""
    import torch
    g = np.random.default_rng(5)
    t, H, E, k, scale = 64, 128, 12, 3, 1.5
    offsets = np.array([0, 20, 20, 61], dtype=np.int32)
    logits = (1.5 * g.standard_normal((t, E))).astype(np.float32)
    ys, h = g.standard_normal((t * k, H)).astype(np.float32), g.standard_normal((t, H)).astype(np.float32)
    gate, gain, post = (g.standard_normal((t, 1)).astype(np.float32), (1 + 0.1 * g.standard_normal(H)).astype(np.float32),
                        (1 + 0.1 * g.standard_normal(H)).astype(np.float32))
    dh, dx = g.standard_normal((t, H)).astype(np.float32), g.standard_normal((t, H)).astype(np.float32)
    dh[61:], dx[61:] = 0, 0                                     # rows of no sequence take no part
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32).copy()
    order = np.argsort(ids.reshape(-1), kind="stable")
    inv = np.empty(t * k, dtype=np.int32)
    inv[order] = np.arange(t * k)
    dl = (3.0, 0.2)
    counts, _, _ = O.balance_loss(logits, ids, rule, offsets=offsets)

    def total(logits=logits.astype(np.float64), ys=ys.astype(np.float64), gate=gate, gain=gain, post=post, h=h):
        z = logits
        zs = np.take_along_axis(z, ids.astype(np.int64), axis=1)
        if rule == "sqrtsoftplus":
            w = scale * O.router_scores(zs)[0]
        else:
            w = np.exp(zs - zs.max(axis=1, keepdims=True))
            w = w / w.sum(axis=1, keepdims=True)
        y = O.combine_rows(ys, inv.reshape(t, k), w)
        out, x = O.residual_norm(y, h, gain, post, gate, True, 0.5, 1.25, 1e-5)
        p, lse = O.router_probabilities(z, rule), O.router_softmax(z)[1]
        parts = [E * (counts[s] / (k * (b - a)) * p[a:b].mean(axis=0)).sum()
                 for s, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])) if b > a]
        return (out * dh).sum() + (x * dx).sum() + dl[0] * np.mean(parts) + dl[1] * np.mean(lse[:61] ** 2)

    # forward and backward on the GPU
    new = (lambda *s: torch.empty(*s, device="cuda"))
    zl, zi = dev(logits), dev(ids)
    w = dev(O.route_weights(logits, ids, rule, None, scale).astype(np.float32))
    y, out, x = new(t, H), new(t, H), new(t, H)
    lib.moe_combine(dev(ys), dev(inv), w, y)
    args = dict(gain=dev(gain), post_gain=dev(post), gate=dev(gate), gate_sigmoid=True, scale=0.5, residual_scale=1.25, eps=1e-5)
    lib.residual_norm(y, dev(h), out, x, **args)
    c, probs, losses = torch.empty(3, E, dtype=torch.int32, device="cuda"), new(3, E), new(2)
    lib.moe_balance_loss(zl, zi, c, probs, losses, torch.empty(lib.moe_balance_workspace_bytes(t, E, 3), dtype=torch.uint8,
                         device="cuda"), scoring=lib.SCORING_BY_NAME[rule], seq_offsets=dev(offsets))
    np.testing.assert_array_equal(c.cpu().numpy(), counts)
    dy, dhin, dgain, dpost, dgate = new(t, H), new(t, H), new(H), new(H), new(t, 1)
    lib.residual_norm_backward(y, out, dev(dh), dev(dx), dy, dhin, **args, dgain=dgain, dpost_gain=dpost, dgate=dgate,
                               workspace=torch.empty(lib.residual_norm_backward_workspace_bytes(t, H), dtype=torch.uint8,
                                                     device="cuda"))
    dys, dw = new(t * k, H), new(t, k)
    lib.moe_combine_backward(dy, dev(ys), dev(inv), w, dys, dw)
    d = torch.zeros(t, E, device="cuda")
    lib.moe_route_backward(zl, zi, dw, d, scoring=lib.SCORING_BY_NAME[rule], scale=scale, counts=c,
                           dlosses=dev(np.array(dl, dtype=np.float32)), seq_offsets=dev(offsets))
    for name, at, got in (("logits", logits, d), ("ys", ys, dys), ("gate", gate, dgate), ("gain", gain, dgain),
                          ("post", post, dpost), ("h", h, dhin)):
        got = f64(got).reshape(at.shape)
        for _ in range(3):
            way = g.standard_normal(at.shape)
            step = 1e-5
            there = (total(**{name: at + step * way}) - total(**{name: at - step * way})) / (2 * step)
            assert abs(there - (got * way).sum()) <= 1e-4 * np.sqrt((got ** 2).sum() * at.size) + 1e-6, name


def test_rows_beyond_32_bit_offsets(lib):
    import torch
    t, H = 270001, 8192                                   # 4.4 GB a matrix
    y = torch.empty(t, H, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    h = torch.empty_like(y).uniform_(-2, 2)
    gain = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out, x = torch.empty_like(h), torch.empty_like(h)
    lib.residual_norm(y, h, out, x, gain=gain)
    dy, dh = torch.empty_like(y), torch.empty_like(h)
    lib.residual_norm_backward(y, out, h, x, dy, dh, gain=gain)
    for at in (0, 1000, t - 3):
        rows = slice(at, at + 3)
        want, want_x = O.residual_norm(f64(y[rows]), f64(h[rows]), f64(gain))
        np.testing.assert_allclose(f64(out[rows]), want, rtol=2.0 ** -8, atol=1e-6)
        np.testing.assert_allclose(f64(x[rows]), want_x, rtol=2.0 ** -8, atol=1e-5)
        back = O.residual_norm_backward(f64(y[rows]), f64(out[rows]), f64(h[rows]), f64(x[rows]), f64(gain))
        np.testing.assert_allclose(f64(dy[rows]), back["dy"], rtol=2.0 ** -8, atol=1e-4)
        np.testing.assert_allclose(f64(dh[rows]), back["dh"], rtol=2.0 ** -8, atol=1e-4)


def test_logits_beyond_32_bit_offsets(lib):
    import torch
    t, e, k = 1100003, 1024, 2                            # 4.5 GB of logits
    logits = torch.empty(t, e, device="cuda").uniform_(-3, 3)
    ids = torch.randint(0, e // 2, (t, k), dtype=torch.int32, device="cuda")
    ids[:, 1] += e // 2
    counts, probs, losses = torch.empty(1, e, dtype=torch.int32, device="cuda"), torch.empty(1, e, device="cuda"), torch.empty(2, device="cuda")
    ws = torch.empty(lib.moe_balance_workspace_bytes(t, e), dtype=torch.uint8, device="cuda")
    lib.moe_balance_loss(logits, ids, counts, probs, losses, ws)
    assert torch.equal(counts[0].long(), torch.bincount(ids.view(-1).long(), minlength=e))
    assert abs(float(probs.double().sum()) - 1) < 1e-4
    dw, d = torch.randn(t, k, device="cuda"), torch.empty(t, e, device="cuda")
    dl = torch.tensor([0.0, 1.0], device="cuda")
    lib.moe_route_backward(logits, ids, dw, d, counts=counts, dlosses=dl)
    for at in (0, t // 2, t - 2):
        rows = slice(at, at + 2)
        z, i = logits[rows].cpu().numpy(), ids[rows].cpu().numpy()
        want = O.route_backward(z, i, dw[rows].cpu().numpy())
        soft, lse = O.router_softmax(O.router_logits(z))
        np.testing.assert_allclose(f64(d[rows]), want + 2 / t * lse * soft, rtol=1e-4, atol=1e-9)


def test_a_residual_beyond_32_bit_offsets(lib):
    import torch
    m, n, k = 530001, 4096, 16                            # 2^31 values and more
    g = np.random.default_rng(9)
    x = torch.randint(0, 100, (m, k), dtype=torch.uint8, device="cuda")
    xs = torch.full((m, 1), 2e-2, device="cuda")
    w, ws = fp8_weight(g, n, k)
    bias = torch.randn(n, device="cuda")
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda").uniform_(-2, 2)
    places = [0, 300000, m - 2]
    before = [f64(y[a:a + 2]) for a in places]
    lib.mm_fp8_b128(x, xs, w, ws, y, act="relu", bias=bias, residual=y, scale=0.5)
    for a, r in zip(places, before):
        v = O.mm_fp8_block(O.e4m3_value(x[a:a + 2].cpu().numpy()), xs[a:a + 2].cpu().numpy(), w.view(torch.uint8).cpu().numpy(),
                           ws.cpu().numpy())
        want = O.product_end(v, f64(bias), "relu", 0.5, r)
        np.testing.assert_allclose(f64(y[a:a + 2]), want, rtol=2.0 ** -8, atol=1e-5)
    assert lib.device_status() == lib.DEV_OK


def test_calls_behind_what_writes_their_inputs(lib):
    """Second kernels read the gate, the gains and the offsets while the first is ending: written by a kernel or a copy just
    before the call, on the same stream, they are the new ones; on two streams at once too."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    t, h, e, k, n = 500, 1024, 64, 4, 6
    rows = [torch.randn(t, h, generator=g, device="cuda") for _ in range(4)]
    gates = torch.randn(n, h, generator=g, device="cuda")
    logits = torch.randn(t, e, generator=g, device="cuda")
    ids = torch.topk(logits, k).indices.int()
    cuts = torch.randint(0, t + 1, (n, 4), generator=g, device="cuda").sort(1).values.int()

    def state():
        new = (lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda"))
        return dict(gate=new(h), post=new(h), off=new(4, d=torch.int32), dy=new(t, h), dh=new(t, h), dgain=new(h), dpost=new(h),
                    dgate=new(h), counts=new(3, e, d=torch.int32), probs=new(3, e), losses=new(2),
                    ws=new(lib.residual_norm_backward_workspace_bytes(t, h), d=torch.uint8),
                    wb=new(lib.moe_balance_workspace_bytes(t, e, 3), d=torch.uint8))

    def step(s, i):
        torch.mul(gates[i], 1.0, out=s["gate"])
        torch.add(gates[i], 2.0, out=s["post"])
        lib.residual_norm_backward(*rows, s["dy"], s["dh"], gain=gates[0], post_gain=s["post"], gate=s["gate"], gate_sigmoid=True,
                                   dgain=s["dgain"], dpost_gain=s["dpost"], dgate=s["dgate"], workspace=s["ws"])
        s["off"].copy_(cuts[i])
        lib.moe_balance_loss(logits, ids, s["counts"], s["probs"], s["losses"], s["wb"], seq_offsets=s["off"])
        return [s[x].clone() for x in ("dy", "dh", "dgain", "dpost", "dgate", "counts", "probs", "losses")]

    alone, one = [], state()
    for i in range(n):
        alone.append(step(one, i))
        torch.cuda.synchronize()
    streams, states = [torch.cuda.Stream(), torch.cuda.Stream()], [state(), state()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for i in range(n):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                got[j].append(step(states[j], i if j == 0 else n - 1 - i))
    torch.cuda.synchronize()
    for i in range(n):
        for a, b, c in zip(alone[i], got[0][i], got[1][n - 1 - i]):
            assert torch.equal(a, b) and torch.equal(a, c)

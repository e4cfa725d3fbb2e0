"""GPU: small inputs that a call's second kernel reads (gate, gains, offsets), rewritten in place just before each of
many calls, where the call's first kernel runs on few SMs: every result is that of the new values, bit for bit what
the call gives alone with fresh tensors."""
import pytest

pytestmark = pytest.mark.gpu

REWRITES = 40


def new(*shape, dtype=None):
    import torch
    return torch.empty(*shape, dtype=dtype or torch.float32, device="cuda")


def compare(step, values, inputs):
    """step(inputs) -> outputs, after each rewrite of the inputs; against fresh tensors, one call at a time."""
    import torch
    got = []
    for i in range(REWRITES):
        for name, t in inputs.items():
            if i % 2:
                t.copy_(values[i][name])
            else:
                torch.add(values[i][name], 0, out=t)          # by a kernel
        got.append([o.clone() for o in step(inputs)])
    torch.cuda.synchronize()
    for i in range(REWRITES):
        want = step({name: v.clone() for name, v in values[i].items()})
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want)), f"rewrite {i}"


@pytest.mark.parametrize("t,h,dtype", [(1, 64, "f32"), (1, 4096, "bf16"), (16, 2048, "bf16"), (40, 1024, "f16"), (9, 12288, "bf16")])
def test_gate_and_gains_of_the_norm_gradients(lib, t, h, dtype):
    import torch
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(t + h)
    rand = (lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt))
    rows = [rand(t, h) for _ in range(4)]
    values = [{"gain": 1 + rand(h), "post_gain": 1 + rand(h), "gate": rand(h)} for _ in range(REWRITES)]
    ws = new(lib.residual_norm_backward_workspace_bytes(t, h), dtype=torch.uint8)

    def step(x):
        dy, dh, sums = torch.empty_like(rows[0]), torch.empty_like(rows[1]), [new(h) for _ in range(3)]
        lib.residual_norm_backward(*rows, dy, dh, **x, gate_sigmoid=True, dgain=sums[0], dpost_gain=sums[1], dgate=sums[2],
                                   workspace=ws)
        return [dy, dh, *sums]

    compare(step, values, {n: torch.empty_like(v) for n, v in values[0].items()})


@pytest.mark.parametrize("t,e,s", [(257, 32, 2), (300, 128, 5), (500, 64, 3), (2000, 40, 9)])
def test_offsets_of_the_balance_statistics(lib, t, e, s):
    import torch
    g = torch.Generator(device="cuda").manual_seed(t + e)
    logits = torch.randn(t, e, generator=g, device="cuda")
    ids = torch.topk(logits, 4).indices.int()
    values = [{"seq_offsets": torch.randint(0, t + 1, (s + 1,), generator=g, device="cuda").sort().values.int()}
              for _ in range(REWRITES)]
    ws = new(lib.moe_balance_workspace_bytes(t, e, s), dtype=torch.uint8)

    def step(x):
        out = [new(s, e, dtype=torch.int32), new(s, e), new(2)]
        lib.moe_balance_loss(logits, ids, *out, ws, **x)
        return out

    compare(step, values, {"seq_offsets": torch.empty_like(values[0]["seq_offsets"])})
    assert lib.device_status() == lib.DEV_OK

"""GPU: host threads whose router calls differ in the number of experts, on streams and with workspaces of their own.
All numbers need more shared memory than a kernel gets without asking, and take the same kernel.  The threads are a C++
program's, which make their calls through the C functions as fast as they can: Python's own would take turns."""
import ctypes
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

CALLS = 4000
EXPERTS = (1024, 800)

SOURCE = r"""
#include "bq.h"
#include <thread>
#include <vector>

struct Call {   // one thread's
    int32_t T, E, k;
    const float* logits;
    const int32_t* ids;
    const float* dweights;
    int32_t* counts;
    float *probs, *losses, *dlogits, *dbias;
    const float* dlosses;
    void* workspace;
    size_t bytes;
    bq_stream_t stream;
    int32_t kind, errors, status;
};

typedef decltype(&bq_moe_balance_loss) Balance;
typedef decltype(&bq_moe_route_backward) Gradient;

extern "C" void run_calls(Balance balance, Gradient gradient, Call* calls, int n, int times) {
    std::vector<std::thread> threads;
    for (int i = 0; i < n; ++i)
        threads.emplace_back([=] {
            Call& c = calls[i];
            for (int j = 0; j < times; ++j) {
                const bq_status s =
                    c.kind == 0 ? balance(c.logits, nullptr, c.T, c.E, c.ids, c.k, 0, nullptr, 1, c.counts, c.probs, c.losses,
                                          c.workspace, c.bytes, c.stream)
                                : gradient(c.logits, nullptr, c.T, c.E, c.ids, c.k, 0, 1.f, c.dweights, c.counts, c.dlosses,
                                           nullptr, 1, c.dlogits, 0, c.dbias, c.workspace, c.bytes, c.stream);
                if (s != BQ_OK) { ++c.errors; c.status = s; }
            }
        });
    for (auto& t : threads) t.join();
}
"""


class Call(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "E", "k")] +
                [(n, ctypes.c_void_p) for n in ("logits", "ids", "dweights", "counts", "probs", "losses", "dlogits", "dbias",
                                                "dlosses", "workspace")] +
                [("bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)] +
                [(n, ctypes.c_int32) for n in ("kind", "errors", "status")])


@pytest.fixture(scope="module")
def runner(tmp_path_factory, lib):
    import os
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    where = tmp_path_factory.mktemp("threads")
    (where / "run.cpp").write_text(SOURCE)
    include = os.path.join(os.path.dirname(os.path.dirname(lib.LIB_PATH)), "include")
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", include, str(where / "run.cpp"), "-o",
                    str(where / "run.so")], check=True)
    return ctypes.CDLL(str(where / "run.so"))


def tensors(lib, kind, e):
    import torch
    g = torch.Generator(device="cuda").manual_seed(e)
    t, k = 40, 4
    new = (lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda"))
    logits = torch.randn(t, e, generator=g, device="cuda")
    x = {"logits": logits, "ids": torch.topk(logits, k).indices.int().contiguous(),
         "dweights": torch.randn(t, k, generator=g, device="cuda"), "counts": new(1, e, dtype=torch.int32) + 1}
    if kind == "statistics":
        x.update(probs=new(1, e), losses=new(2), workspace=new(lib.moe_balance_workspace_bytes(t, e), dtype=torch.uint8))
    else:
        x.update(dlogits=new(t, e), dbias=new(e), workspace=new(lib.moe_route_backward_workspace_bytes(t, e), dtype=torch.uint8))
        if kind == "weights and losses":
            x["dlosses"] = new(2) + 1
    return t, k, x


@pytest.mark.parametrize("kind", ["statistics", "weights", "weights and losses"])
def test_threads_of_different_experts(lib, runner, kind):
    import torch
    written = ("counts", "probs", "losses") if kind == "statistics" else ("dlogits", "dbias")
    calls, keep, wants = (Call * len(EXPERTS))(), [], []
    for c, e in zip(calls, EXPERTS):
        t, k, x = tensors(lib, kind, e)
        stream = torch.cuda.Stream()
        c.T, c.E, c.k, c.kind, c.bytes, c.stream = t, e, k, int(kind != "statistics"), x["workspace"].numel(), stream.cuda_stream
        for name, v in x.items():
            setattr(c, name, v.data_ptr())
        keep.append((x, stream))
    torch.cuda.synchronize()

    def run(some, n, times):
        runner.run_calls(ctypes.cast(lib._lib.bq_moe_balance_loss, ctypes.c_void_p),
                         ctypes.cast(lib._lib.bq_moe_route_backward, ctypes.c_void_p), some, n, times)
        torch.cuda.synchronize()

    for i, (x, _) in enumerate(keep):                     # one after the other
        run(ctypes.byref(calls, i * ctypes.sizeof(Call)), 1, 1)
        wants.append({n: x[n].clone() for n in written})
        for n in written:
            x[n].zero_()
    torch.cuda.synchronize()
    if kind != "statistics":
        assert all(w["dlogits"].any() and w["dbias"].any() for w in wants)
    run(calls, len(EXPERTS), CALLS)
    assert [(c.errors, lib.status_string(c.status)) for c in calls] == [(0, "BQ_OK")] * len(EXPERTS)
    for (x, _), want in zip(keep, wants):
        assert all(torch.equal(x[n], want[n]) for n in written)

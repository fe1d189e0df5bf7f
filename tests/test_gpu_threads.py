"""Calls from several host threads."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import workloads
from tests._group_int4 import codes, gen, make_layer, scales, shape_of

pytestmark = pytest.mark.gpu


def calls(moe, dev):
    """One call of each kernel sequence, on tensors of its own: (name, function that returns its output)."""
    g = gen(1, dev)

    def x(T, H):
        return torch.randn((T, H), generator=g, device=dev).to(torch.bfloat16)

    N, K = 1024, 2048
    lin = moe.Int4Linear(codes(g, N, K // 2), scales(g, (N,), K, 64, "bf16"), 64)
    few_shape = shape_of(1024, 16, 2, 256, 256)
    few_layer = make_layer(few_shape, 64, "bf16", device=dev)
    shape = workloads.LayerShape(512, 16, 4, 256, 256, 1.0)
    layer = workloads.make_layer(shape, 390, 0, dev)
    for T in (1, 8, 16, 40, 300):
        a, o = x(T, K), torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        yield f"linear {T}", lambda a=a, o=o: lin(a, out=o)
    for T in (1, 4, 8):
        m, a = moe.MoEFewLayer(few_layer, few_shape, 64), x(T, 1024)
        yield f"few {T}", lambda m=m, a=a, o=torch.empty_like(a): m(a, out=o)
    for T in (3, 33, 400):
        m, a = moe.MoELayer(layer, shape, max_tokens=T), x(T, 512)
        yield f"layer {T}", lambda m=m, a=a, o=torch.empty_like(a): m(a, out=o)


def test_first_call_of_a_thread(cuda_device):
    """A host thread whose first CUDA work is the call itself, in a process that has made it before."""
    import int4_expert_ffn_sigmoid_b200 as moe
    for name, call in calls(moe, cuda_device):
        want, got = call().clone(), []
        torch.cuda.synchronize()

        def run():
            try:
                got.append(call())
            except Exception as e:  # noqa: BLE001
                got.append(e)

        t = threading.Thread(target=run)
        t.start()
        t.join()
        assert isinstance(got[0], torch.Tensor), (name, got[0])
        assert torch.equal(got[0], want), name


def run_at_once(times=4):
    """The calls, `times` each, every one from a thread and on a stream of its own, as a process's first launches."""
    import int4_expert_ffn_sigmoid_b200 as moe
    work = [c for _ in range(times) for c in calls(moe, torch.device("cuda:0"))]
    streams = [torch.cuda.Stream() for _ in work]
    got, start = [None] * len(work), threading.Barrier(len(work))
    torch.cuda.synchronize()

    def run(i):
        start.wait()
        try:
            with torch.cuda.stream(streams[i]):
                got[i] = work[i][1]()
        except Exception as e:  # noqa: BLE001
            got[i] = e

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (name, call), o in zip(work, got):
        assert isinstance(o, torch.Tensor), (name, o)
        first = o.clone()
        assert torch.equal(call(), first), name
    print("ok", len(work))


@pytest.mark.parametrize("again", range(3))
def test_first_calls_of_a_process_at_once(cuda_device, again):
    """What a launch asks once per device (SM count, cluster capacity, shared memory limits) reaches the other threads
    whole, whichever is first."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", "from tests.test_gpu_threads import run_at_once; run_at_once()"], cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr

"""Weights, scales and router constants that a PyTorch kernel writes directly ahead of a call, eagerly and captured:
such kernels do not let their dependents start early, so the call, which reads weights before it waits, sees them."""
import pytest
import torch

from tests._group_int4 import codes, gen, make_layer, scales, shape_of

pytestmark = pytest.mark.gpu


def replayed(step):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph.replay


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [1, 8, 40])
def test_linear(cuda_device, T, captured):
    import int4_expert_ffn_sigmoid_b200 as moe
    g = gen(T, cuda_device)
    N, K = 2304, 4096
    sets = [(codes(g, N, K // 2), scales(g, (N,), K, 64, "bf16")) for _ in range(3)]
    x = torch.randn((T, K), generator=g, device=cuda_device).to(torch.bfloat16)
    want = [moe.linear_forward(x, w, s, 64) for w, s in sets]
    src = [torch.empty_like(t) for t in sets[0]]
    lin = moe.Int4Linear(*[torch.empty_like(t) for t in sets[0]], 64)
    out = torch.empty_like(want[0])

    def step():
        lin(x, out=out)  # a call of ours ahead of the writers
        lin.w.copy_(src[0])
        lin.scales.copy_(src[1])
        lin(x, out=out)

    for t, v in zip(src, sets[0]):
        t.copy_(v)
    run = replayed(step) if captured else step
    for i in range(60):
        for t, v in zip(src, sets[i % 3]):
            t.copy_(v)
        run()
        assert torch.equal(out, want[i % 3]), i


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dims", [(512, 16, 2, 256, 256), (2048, 256, 8, 128, 128)])
def test_few(cuda_device, dims, captured):
    import int4_expert_ffn_sigmoid_b200 as moe
    shape = shape_of(*dims)
    layers = [make_layer(shape, 64, "bf16", seed=i, device=cuda_device) for i in range(3)]
    x = torch.randn((4, shape.H), generator=gen(4, cuda_device), device=cuda_device).to(torch.bfloat16)
    want = [moe.MoEFewLayer(L, shape, 64)(x) for L in layers]
    src, live = ({k: torch.empty_like(v) for k, v in layers[0].items()} for _ in range(2))
    for k, v in layers[0].items():
        src[k].copy_(v)
        live[k].copy_(v)
    m = moe.MoEFewLayer(live, shape, 64)
    out = torch.empty_like(want[0])
    order = sorted(live, key=lambda k: (k == "router_bias", k == "router_w", k))  # what is read first is written last

    def step():
        m(x, out=out)
        for k in order:
            live[k].copy_(src[k])
        m(x, out=out)

    run = replayed(step) if captured else step
    for i in range(60):
        for k, v in layers[i % 3].items():
            src[k].copy_(v)
        run()
        assert torch.equal(out, want[i % 3]), i

"""The same call gives the same bits, with the weights in L2 and not."""
import pytest
import torch

import workloads
from tests._group_int4 import codes, gen, make_layer, scales, shape_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 32])
def test_large_layer_from_cold_caches(cuda_device, T):
    """A weight stage is refilled only after its last reads: where it is not, a few elements of h of about one call
    in fifteen differ, when the weights come from HBM and the warps run apart."""
    import int4_expert_ffn_sigmoid_b200 as moe
    wl = workloads.WORKLOADS["large_layer"]
    layer = workloads.make_layer(wl.shape, wl.wid, 0, cuda_device, wl.bias_mode)
    x = workloads.make_x(wl.shape, T, wl.wid, device=cuda_device)
    m = moe.MoELayer(layer, wl.shape, max_tokens=T)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    first = m(x)
    for i in range(150):
        flush.fill_(i & 255)
        assert torch.equal(m(x), first), i


@pytest.mark.parametrize("T,N,K", [(4, 3001, 6144), (64, 4096, 4096), (300, 1024, 4096)])
def test_linear_from_cold_caches(cuda_device, T, N, K):
    import int4_expert_ffn_sigmoid_b200 as moe
    g = gen(T, cuda_device)
    x = torch.randn((T, K), generator=g, device=cuda_device).to(torch.bfloat16)
    lin = moe.Int4Linear(codes(g, N, K // 2), scales(g, (N,), K, 64, "bf16"), 64)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    first = lin(x)
    for i in range(60):
        flush.fill_(i)
        lin(x)  # and the second call beside the end of the first
        assert torch.equal(lin(x), first), i


@pytest.mark.parametrize("T,H,E,K", [(1, 1024, 64, 2), (8, 2560, 64, 8), (5, 3584, 14, 2)])
def test_few_from_cold_caches(cuda_device, T, H, E, K):
    import int4_expert_ffn_sigmoid_b200 as moe
    shape = shape_of(H, E, K, 512, 512)
    m = moe.MoEFewLayer(make_layer(shape, 64, "bf16", device=cuda_device), shape, 64)
    x = torch.randn((T, H), generator=gen(T, cuda_device), device=cuda_device).to(torch.bfloat16)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    first = m(x, residual=True)
    for i in range(60):
        flush.fill_(i)
        m(x)
        assert torch.equal(m(x, residual=True), first), i

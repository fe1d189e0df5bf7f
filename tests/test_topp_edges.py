"""Adaptive top-p of tokens whose score sum is zero or NaN: at least one pick is kept, and a NaN token's picks all are,
so that its output is NaN as it is without top-p."""
import numpy as np
import pytest
import torch

import oracle
from oracle import dense_masked
from tests._group_int4 import gen, make_layer, shape_of

TOPP = 0.7
BAD, LOW = 1, 3  # the tokens with a NaN and with scores that all underflow


def edge_tokens(T, H, device, value=1.0):
    """T tokens; BAD holds a NaN, LOW is the only one whose last column is not zero."""
    x = torch.randn((T, H), generator=gen(11, device), device=device).to(torch.bfloat16)
    x[:, H - 1] = 0
    x[BAD, 5] = float("nan")
    x[LOW] = 0
    x[LOW, H - 1] = value
    return x


def edge_router(L, depth):
    """Every expert's logit of token LOW is `depth`; the biases keep the picks apart."""
    L["router_w"] = L["router_w"].clone()
    L["router_w"][:, -1] = depth
    L["router_bias"] = torch.linspace(0.1, 0.2, L["router_w"].shape[0], device=L["router_w"].device)
    return L


def test_oracle_and_dense_form_keep_a_pick():
    g = gen(3, "cpu")
    E, H, K = 12, 16, 4
    L = edge_router({"router_w": torch.randn((E, H), generator=g)}, -1000.0)  # exp(1000) is infinite in 64 bits
    r = oracle.route(edge_tokens(5, H, "cpu"), L["router_w"], L["router_bias"], K, 2.0, TOPP)
    assert r["idx"][BAD].tolist() == [0, 1, 2, 3] and np.isnan(r["weights"][BAD]).all()
    assert r["idx"][LOW].tolist() == [8, -1, -1, -1]  # picks 11, 10, 9, 8 tie at score 0: the lowest expert is first
    assert np.isnan(r["weights"][LOW, 0]) and not r["weights"][LOW, 1:].any()
    for t in (0, 2, 4):
        assert r["idx"][t, 0] >= 0 and np.isfinite(r["weights"][t]).all()
    assert dense_masked.topp_keep(np.full(3, np.nan), np.array([4, 1, 2]), TOPP).tolist() == [True] * 3
    assert dense_masked.topp_keep(np.zeros(3), np.array([4, 1, 2]), TOPP).tolist() == [False, True, False]


def _edges(run, K):
    """run(topp) -> out, idx, weights."""
    out, idx, w = run(TOPP)
    assert bool((idx[BAD] >= 0).all()) and bool(torch.isnan(w[BAD]).all())
    assert not bool(torch.isfinite(out[BAD]).any())
    full = run(0.0)[1]
    assert idx[LOW].tolist() == [int(full[LOW].min())] + [-1] * (K - 1)
    assert bool(torch.isnan(w[LOW, 0])) and not bool(w[LOW, 1:].any())
    assert not bool(torch.isfinite(out[LOW]).any())
    keep = [t for t in range(out.shape[0]) if t not in (BAD, LOW)]
    assert bool(torch.isfinite(out[keep]).all()) and bool((idx[keep, 0] >= 0).all())
    return out, idx, w, keep


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T", [4, 7])
@pytest.mark.parametrize("H,E,K", [(256, 24, 6), (2048, 256, 8)])  # router in the layer kernel, and in front of it
def test_few_layer(cuda_device, H, E, K, T, residual):
    import int4_expert_ffn_sigmoid_b200 as moe
    shape = shape_of(H, E, K, 128, 0, 2.5)
    assert moe.few_kernel_launches(shape, T, 64) == (2 if H == 256 else 3)
    L = edge_router(make_layer(shape, 64, "bf16", device=cuda_device), -200.0)  # exp(200) is infinite in 32 bits
    x = edge_tokens(T, H, cuda_device)

    def run(topp, x=x):
        m = moe.MoEFewLayer(L, shape, 64, topp=topp)
        idx = torch.full((x.shape[0], K), -7, dtype=torch.int32, device=cuda_device)
        w = torch.full((x.shape[0], K), -7.0, device=cuda_device)
        return m(x, residual=residual, topk_idx=idx, topk_w=w), idx, w

    out, idx, w, keep = _edges(run, K)
    clean = x.clone()
    clean[[BAD, LOW]] = clean[0].clone()
    o, i, v = run(TOPP, clean)  # the other tokens do not notice
    assert torch.equal(idx[keep], i[keep]) and torch.equal(w[keep], v[keep])
    # the pass's touched experts are dealt out to warps, so the order of a row's f32 additions may change; both sums
    # are then rounded to bf16, half a step (2^-8) each
    a, b = out[keep].double(), o[keep].double()
    assert float(((a - b).norm(dim=1) / b.norm(dim=1)).max()) <= 2.0 ** -7


@pytest.mark.gpu
@pytest.mark.parametrize("T,flags", [(20, 0), (130, "MOE_FORCE_PREFILL"), (150, "MOE_FORCE_DECODE")])
def test_layer_paths(cuda_device, T, flags):
    import int4_expert_ffn_sigmoid_b200 as moe
    import workloads
    shape = workloads.LayerShape(1024, 64, 8, 256, 0, 2.5)
    f = getattr(moe, flags) if flags else 0
    L = edge_router(workloads.make_layer(shape, 377, 0, cuda_device), -200.0)
    x = edge_tokens(T, shape.H, cuda_device)

    def run(topp):
        idx = torch.full((T, shape.K), -7, dtype=torch.int32, device=cuda_device)
        w = torch.full((T, shape.K), -7.0, device=cuda_device)
        return moe.layer_forward(x, L, shape, flags=f | moe.MOE_DEBUG_CHECK, topk_idx=idx, topk_w=w, topp=topp), idx, w

    _edges(run, shape.K)

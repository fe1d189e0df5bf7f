"""The projection where each weight is kept in two bf16 parts: any call of up to eight tokens that does not stream, and
more tokens under MOE_FULL_WEIGHTS."""
import pytest
import torch

from tests._group_int4 import block_max, codes, gen, linear64, scales, weights64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import int4_expert_ffn_sigmoid_b200 as m
    return m


def bound(x, w, s, group, add=None, streamed=False):
    """A weight's two bf16 parts hold it to 2^-15: the scale's second part is off by half a step (2^-8) of at most 2^-8 of
    the scale, and so is the weight's; weight streaming holds an activation to 2^-15 of the largest of its
    256 columns, which is more.  Sums: as in linear_bound, an f32 chain of at most K / 16 + 64 additions, two products
    a weight here: K / 8 + 64."""
    W = weights64(w, s, group).abs()
    mag = x.double().abs() @ W.t()
    b = 2.0 ** -15 * (block_max(x, 256) @ W.t()) if streamed else 2.0 ** -15 * mag
    b = b + (x.shape[1] / 8 + 64) * 2.0 ** -23 * mag
    return b if add is None else b + 2.0 ** -23 * (mag + add.double().abs())


def fits(T, K):
    """Both int8 parts of T tokens' activations fit beside the rings."""
    return T <= 8 and 2 * T * (-(-K // 256) * 256 + 64) <= 113 * 1024


def check(out, x, w, s, group, add=None, streamed=False):
    want, b = linear64(x, w, s, group, add), bound(x, w, s, group, add, streamed)
    off = (out.double() - want).abs()
    assert bool((off <= b).all()), float((off / b).max())
    # independent errors of at most 2^-15 of a block's largest (under 2^-13 of its r.m.s.), or of 2^-15 of a weight
    assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -12


def make(T, N, K, group, stype, seed, dev):
    g = gen(seed, dev)
    x = torch.randn((T, K), generator=g, device=dev).to(torch.bfloat16)
    return (x, codes(g, N, K // 2), scales(g, (N,), K, group, stype),
            torch.randn((T, N), generator=g, device=dev).to(torch.bfloat16))


@pytest.mark.parametrize("stype,group", [("bf16", 128), ("f32", 32), ("f16", 64), ("f32", 0)])
@pytest.mark.parametrize("T,N,K", [(5, 129, 6144), (6, 2048, 6144), (7, 2368, 4128), (8, 512, 6144), (8, 48, 32768), (8, 2369, 8192),
                                   (1, 130, 32768), (2, 130, 32768), (3, 500, 20000), (5, 129, 12288)])
def test_few_tokens(moe, cuda_device, T, N, K, stype, group):
    """Long rows on few outputs, and activations that do not fit beside the streaming kernel's rings: one accuracy."""
    x, w, s, a = make(T, N, K, group, stype, T + N + K, cuda_device)
    lin = moe.Int4Linear(w, s, group)
    out = lin(x, add=a, flags=moe.MOE_OUT_F32)
    check(out, x, w, s, group, a, streamed=fits(T, K))
    assert torch.equal(lin(x, add=a), out.to(torch.bfloat16))
    assert torch.equal(lin(x, add=a, flags=moe.MOE_FULL_WEIGHTS), out.to(torch.bfloat16))  # it is the only form here


@pytest.mark.parametrize("stype,group", [("bf16", 128), ("f32", 32), ("f16", 64), ("bf16", 0)])
@pytest.mark.parametrize("T,N,K", [
    (9, 64, 128), (10, 1, 96), (17, 40, 8192), (20, 6200, 1184), (33, 1000, 992), (64, 1024, 1024), (65, 384, 736),
    (120, 2300, 4096), (128, 512, 512), (130, 257, 2048), (300, 1000, 416), (513, 130, 1184), (520, 4096, 6144),
])
def test_full_weights(moe, cuda_device, T, N, K, stype, group):
    x, w, s, a = make(T, N, K, group, stype, T + N + K, cuda_device)
    lin = moe.Int4Linear(w, s, group)
    f = moe.MOE_FULL_WEIGHTS
    out = lin(x, add=a, flags=f | moe.MOE_OUT_F32)
    check(out, x, w, s, group, a)
    assert torch.equal(lin(x, add=a, flags=f), out.to(torch.bfloat16))  # one rounding
    assert torch.equal(lin(x, add=a, flags=f | moe.MOE_OUT_F32), out)


@pytest.mark.parametrize("T", [8, 40])
def test_scales_of_every_size(moe, cuda_device, T):
    """Zero, negative, tiny and large scales (one range a row), every code; f32 scales that bf16 does not hold."""
    N, K, group = 2304, 4096, 64
    x, w, s, _ = make(T, N, K, group, "f32", 5, cuda_device)
    s[0::6] = 0
    s[1::6] *= -1
    s[2::6] *= 2.0 ** -90
    s[3::6] *= 2.0 ** 60
    s[4::6] = 1 + 2.0 ** -15
    w[5::6] = 0x88  # every code -8
    out = moe.linear_forward(x, w, s, group, flags=moe.MOE_OUT_F32 | moe.MOE_FULL_WEIGHTS)
    off, b = (out.double() - linear64(x, w, s, group)).abs(), bound(x, w, s, group)
    assert bool((off <= b).all()), float((off / b.clamp(min=1e-300)).max())
    assert bool((out[:, 0::6] == 0).all())


def test_captured_beside_the_rounded_form(moe, cuda_device):
    """Both forms and a few tokens in one graph, replayed on new inputs."""
    N, K, group = 700, 4096, 64
    x, w, s, a = make(48, N, K, group, "f16", 9, cuda_device)
    lin = moe.Int4Linear(w, s, group)
    f = moe.MOE_OUT_F32

    def run():
        return lin(x, flags=f | moe.MOE_FULL_WEIGHTS), lin(x, flags=f), lin(x[:8], flags=f)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        full, one, few = run()
    for seed in range(3):
        x.copy_(make(48, N, K, group, "f16", 90 + seed, cuda_device)[0])
        graph.replay()
        torch.cuda.synchronize()
        want = linear64(x, w, s, group)
        check(full, x, w, s, group)
        check(few, x[:8], w, s, group)
        assert 2.0 ** -12 < float((one.double() - want).norm() / want.norm()) < 2.0 ** -8.7  # weights in one part


def test_non_finite_rows(moe, cuda_device):
    """A token that holds NaN or an infinity gives no number anywhere; the others are untouched."""
    x, w, s, _ = make(20, 130, 512, 32, "bf16", 33, cuda_device)
    lin = moe.Int4Linear(w, s, 32)
    clean = lin(x, flags=moe.MOE_FULL_WEIGHTS)
    bad = x.clone()
    bad[0, 300] = float("nan")
    bad[19, 5] = float("inf")
    out = lin(bad, flags=moe.MOE_FULL_WEIGHTS)
    assert not bool(torch.isfinite(out[[0, 19]]).any())
    assert torch.equal(out[1:19], clean[1:19])

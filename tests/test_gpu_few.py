"""moe_few_forward on the GPU against the layer in 64 bits."""
import pytest
import torch

from tests._group_int4 import few64, gen, make_layer, route64, shape_of

pytestmark = pytest.mark.gpu

# Per-token relative L2 of the f32 output: activations and h are held to within 2^-15 of a block's largest value,
# about 2^-14 of the block's r.m.s. each; gate and up errors enter h once each (|silu'| <= 1.1) and h's own rounding
# follows.  Their root sum, 2^-14 * sqrt(1 + 1.1^2 + 1) < 2^-13, doubled for blocks with a larger peak.
F32_TOL = 2.0 ** -12


@pytest.fixture(scope="module")
def moe():
    import int4_expert_ffn_sigmoid_b200 as m
    return m


def tokens(T, shape, L, seed, device, topp=0.0):
    """T tokens whose routing decisions are not within rounding of falling the other way."""
    g, rows = gen(seed, device), []
    while len(rows) < T:
        x = torch.randn((1, shape.H), generator=g, device=device).to(torch.bfloat16)
        if route64(x, L, shape, topp)[1] > 1e-5:
            rows.append(x)
    return torch.cat(rows)


def check(moe, x, L, shape, group, residual=False, topp=0.0, max_tokens=None, **kw):
    T = x.shape[0]
    m = moe.MoEFewLayer(L, shape, group, max_tokens=max_tokens or T, topp=topp)
    idx = torch.full((T, shape.K), -7, dtype=torch.int32, device=x.device)
    wts = torch.full((T, shape.K), -7.0, device=x.device)
    out32 = m(x, residual=residual, flags=moe.MOE_OUT_F32 | moe.MOE_DEBUG_POISON, topk_idx=idx, topk_w=wts)
    out = m(x, residual=residual)
    picks, _ = route64(x, L, shape, topp)
    for t, (es, ws) in enumerate(picks):
        pad = shape.K - len(es)
        assert idx[t].tolist() == es + [-1] * pad
        assert wts[t].tolist() == pytest.approx(ws + [0.0] * pad, rel=1e-5)
    want = few64(x, L, shape, group, residual, topp)
    rel = (out32.double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(rel.max()) <= F32_TOL, rel
    assert torch.equal(out, out32.to(torch.bfloat16))  # one rounding
    assert torch.equal(out, m(x, residual=residual))  # and the same bits again
    return out


SHAPES = [
    # H, E, K, I, Is, scaling
    (128, 1, 1, 128, 0, 1.0), (128, 8, 2, 128, 128, 1.0), (256, 4, 4, 128, 256, 2.5), (384, 5, 3, 256, 128, 1.0),
    (640, 64, 8, 384, 0, 2.5), (1024, 64, 2, 512, 2048, 1.0), (1152, 33, 4, 896, 640, 1.0), (2048, 256, 8, 256, 512, 2.5),
]


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("T,group,stype", [(1, 32, "f32"), (3, 0, "f32"), (8, 128, "bf16"), (5, 64, "f16"), (4, 1024, "bf16")])
def test_matches_layer(moe, cuda_device, dims, T, group, stype):
    shape = shape_of(*dims)
    L = make_layer(shape, group, stype, seed=sum(dims[:5]), device=cuda_device)
    check(moe, tokens(T, shape, L, 7 + T, cuda_device), L, shape, group, residual=T % 2 == 1)


@pytest.mark.parametrize("T", [2, 6, 7, 9, 16, 21])
def test_token_counts(moe, cuda_device, T):
    """Odd passes, and more tokens than one pass serves."""
    shape = shape_of(512, 16, 3, 256, 384)
    L = make_layer(shape, 32, "bf16", device=cuda_device)
    x = tokens(T, shape, L, T, cuda_device)
    out = check(moe, x, L, shape, 32, residual=True, max_tokens=24)
    one = moe.MoEFewLayer(L, shape, 32)
    for t in (0, T - 1):  # a token's output does not depend on its company
        assert torch.equal(one(x[t:t + 1].contiguous(), residual=True)[0], out[t])


@pytest.mark.parametrize("topp", [0.3, 0.7, 0.95, 1.0])
def test_topp(moe, cuda_device, topp):
    shape = shape_of(256, 24, 6, 128, 128, 2.0)
    L = make_layer(shape, 64, "f16", seed=3, device=cuda_device)
    check(moe, tokens(8, shape, L, 5, cuda_device, topp), L, shape, 64, topp=topp)


def test_row_scales_agree_with_layer_forward(moe, cuda_device):
    """group = 0 reads the weights of layer_forward: same picks, outputs within both paths' errors."""
    import workloads
    shape = workloads.NANO
    L = workloads.make_layer(shape, 11, 0, cuda_device)
    x = tokens(8, shape, L, 2, cuda_device)
    idx, idx2 = (torch.empty((8, 2), dtype=torch.int32, device=cuda_device) for _ in range(2))
    a = moe.layer_forward(x, L, shape, flags=moe.MOE_OUT_F32, topk_idx=idx)
    b = moe.few_forward(x, L, shape, flags=moe.MOE_OUT_F32, topk_idx=idx2)
    assert torch.equal(idx, idx2)
    assert float(((a - b).norm(dim=1) / a.norm(dim=1)).max()) <= 2 * F32_TOL


def test_ties_and_nan_keys(moe, cuda_device):
    """Equal keys: the lower expert; a NaN key is the smallest."""
    shape = shape_of(128, 8, 3, 128, 0)
    L = make_layer(shape, 32, device=cuda_device)
    L["router_w"][:] = L["router_w"][0]
    L["router_bias"][:] = 0.25
    L["router_bias"][1] = float("nan")
    L["router_bias"][5] = 0.5
    x = torch.randn((2, 128), generator=gen(1, cuda_device), device=cuda_device).to(torch.bfloat16)
    idx = torch.empty((2, 3), dtype=torch.int32, device=cuda_device)
    out = moe.few_forward(x, L, shape, 32, flags=moe.MOE_OUT_F32, topk_idx=idx)
    assert idx.tolist() == [[5, 0, 2]] * 2
    want = few64(x, L, shape, 32, picks=idx)
    assert float(((out.double() - want).norm(dim=1) / want.norm(dim=1)).max()) <= F32_TOL
    L["router_bias"][:] = float("nan")  # nothing but NaN: still valid, distinct picks, lowest first
    moe.few_forward(x, L, shape, 32, topk_idx=idx)
    assert idx.tolist() == [[0, 1, 2]] * 2


def test_untouched_experts_are_not_read_into_the_result(moe, cuda_device):
    """NaN or infinite scales of an expert reach only the tokens that picked it."""
    shape = shape_of(512, 16, 2, 256, 256)
    L = make_layer(shape, 32, device=cuda_device)
    x = tokens(8, shape, L, 6, cuda_device)
    m = moe.MoEFewLayer(L, shape, 32)
    idx = torch.empty((8, 2), dtype=torch.int32, device=cuda_device)
    clean = m(x, topk_idx=idx)
    e = int(idx[3, 0])
    for name, v in (("s13", float("nan")), ("s2", float("inf")), ("s2", float("nan"))):
        keep = L[name][e].clone()
        L[name][e] = v
        out = m(x)
        L[name][e] = keep
        for t in range(8):
            if e in idx[t].tolist():
                assert not bool(torch.isfinite(out[t]).any())
            else:
                assert torch.equal(out[t], clean[t])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_token(moe, cuda_device, bad):
    shape = shape_of(256, 8, 2, 128, 128)
    L = make_layer(shape, 32, device=cuda_device)
    x = tokens(5, shape, L, 8, cuda_device)
    m = moe.MoEFewLayer(L, shape, 32)
    clean = m(x)
    x[2, 100] = bad
    out = m(x)
    assert not bool(torch.isfinite(out[2]).any())
    keep = [0, 1, 3, 4]
    assert torch.equal(out[keep], clean[keep])


def test_no_tokens(moe, cuda_device):
    shape = shape_of(128, 4, 1, 128, 0)
    L = make_layer(shape, 0, device=cuda_device)
    assert moe.few_forward(torch.empty((0, 128), dtype=torch.bfloat16, device=cuda_device), L, shape).shape == (0, 128)


def test_widest_layer(moe, cuda_device):
    """The largest hidden size, and experts whose codes lie past 2^32 bytes."""
    shape = shape_of(16384, 256, 2, 2048, 0)  # 256 x 33.5 MB of gate/up codes
    g = gen(4, cuda_device)
    L = make_layer(shape_of(16384, 256, 2, 128, 0), 128, "bf16", device=cuda_device)
    for name, rows, cols in (("w13", 4096, 16384), ("w2", 16384, 2048)):
        n = 256 * rows * cols // 2
        L[name] = torch.randint(-2 ** 63, 2 ** 63 - 1, (n // 8,), generator=g, device=cuda_device).view(torch.uint8).view(256, rows, cols // 2)
        L["s" + name[1:]] = (torch.rand((256, rows, cols // 128), generator=g, device=cuda_device) * 0.004 + 0.002).to(torch.bfloat16)
    L["router_bias"] += torch.linspace(0, 0.5, 256, device=cuda_device)  # the last experts are picked more often
    check(moe, tokens(5, shape, L, 1, cuda_device), L, shape, 128)


def test_streams_and_workspaces(moe, cuda_device):
    """Calls at the same time, each with its own workspace, and one workspace reused on one stream."""
    shape = shape_of(1024, 32, 4, 512, 512)
    L = make_layer(shape, 64, "bf16", device=cuda_device)
    m = moe.MoEFewLayer(L, shape, 64)
    xs = [tokens(t, shape, L, 40 + t, cuda_device) for t in (1, 4, 8)]
    want = [m(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    spaces = [m.new_workspace() for _ in xs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st, ws, o in zip(xs, streams, spaces, outs):
            m(x, out=o, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_decode_step_in_a_graph(moe, cuda_device):
    """A run as it is used: projection, MoE layer with residual, projection back with an add, twice, captured and
    replayed on new inputs."""
    shape = shape_of(1024, 16, 2, 512, 1024)
    L = make_layer(shape, 32, "bf16", device=cuda_device)
    g = gen(9, cuda_device)
    from tests._group_int4 import codes, linear64, scales
    wq, sq = codes(g, 1536, 512), scales(g, (1536,), 1024, 32, "bf16")
    wo, so = codes(g, 1024, 768), scales(g, (1024,), 1536, 32, "bf16")
    q, o = moe.Int4Linear(wq, sq, 32), moe.Int4Linear(wo, so, 32)
    m = moe.MoEFewLayer(L, shape, 32)
    x = tokens(3, shape, L, 3, cuda_device)
    seen = {}

    def step(v):
        for layer in range(2):
            seen["x%d" % layer] = v
            seen["q%d" % layer] = q(v)
            seen["o%d" % layer] = o(seen["q%d" % layer], add=v)
            v = seen["m%d" % layer] = m(seen["o%d" % layer], residual=True)
        return v

    step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x)
    for seed in range(3):
        x.copy_(tokens(3, shape, L, 50 + seed, cuda_device))
        graph.replay()
        torch.cuda.synchronize()
        for layer in range(2):  # each operator against 64 bits on what it was given: bf16 outputs, 2^-8 a value
            v = {k: seen[k + str(layer)].double() for k in "xqom"}
            for got, want in ((v["q"], linear64(v["x"], wq, sq, 32)), (v["o"], linear64(v["q"], wo, so, 32, v["x"]))):
                assert float((got - want).norm() / want.norm()) <= 2.0 ** -8
            if route64(v["o"], L, shape)[1] > 1e-5:
                want = few64(v["o"], L, shape, 32, residual=True)
                assert float((v["m"] - want).norm() / want.norm()) <= 2.0 ** -8


def test_binding_refusals(moe, cuda_device):
    shape = shape_of(256, 4, 2, 128, 128)
    L = make_layer(shape, 32, device=cuda_device)
    m = moe.MoEFewLayer(L, shape, 32, max_tokens=4)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=cuda_device)
    for bad in (x.float(), x[:, :128], x.cpu(), torch.zeros((5, 256), dtype=torch.bfloat16, device=cuda_device)):
        with pytest.raises(ValueError):
            m(bad)
    with pytest.raises(ValueError):
        m(x, topk_idx=torch.zeros((4, 2), dtype=torch.int64, device=cuda_device))
    with pytest.raises(moe.MoeError):
        m(x, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(moe.MoeError):
        m(x, out=x)
    with pytest.raises(moe.MoeError):
        m(x, flags=moe.MOE_FORCE_PREFILL)
    with pytest.raises(ValueError):
        moe.MoEFewLayer({**L, "s2": L["s2"].to(torch.bfloat16)}, shape, 32)
    with pytest.raises(ValueError):
        moe.MoEFewLayer(L, shape, 64)
    with pytest.raises(moe.MoeError):
        moe.MoEFewLayer(L, shape_of(256, 4, 2, 130, 128), 32)


@pytest.mark.parametrize("dims,T,group", [
    ((128, 64, 8, 8192, 8192, 1.0), 8, 32),    # the longest list of down units
    ((6144, 16, 8, 128, 128, 2.5), 8, 64),     # the most activations beside the rings
    ((7168, 8, 2, 128, 256, 1.0), 7, 128),     # a token more than fits: two passes
    ((6912, 8, 2, 128, 256, 1.0), 7, 128),
    ((16384, 8, 1, 128, 0, 1.0), 3, 32768),
])
def test_largest_shared_memory(moe, cuda_device, dims, T, group):
    shape = shape_of(*dims)
    L = make_layer(shape, group, "bf16", seed=1, device=cuda_device)
    assert moe.few_pass_tokens(shape, group) == (6 if shape.H == 7168 else T)
    check(moe, tokens(T, shape, L, 12, cuda_device), L, shape, group)


def test_split_router_passes(moe, cuda_device):
    """Router weights past the cluster's share: the logits kernel in front, in two passes, replayed."""
    shape = shape_of(2048, 256, 8, 128, 128)
    L = make_layer(shape, 128, "f32", device=cuda_device)
    assert moe.few_kernel_launches(shape, 8, 128) == 3 and moe.few_kernel_launches(shape, 13, 128) == 6
    assert moe.few_kernel_launches(shape_of(512, 256, 8, 128, 128), 8, 128) == 2
    x = tokens(13, shape, L, 31, cuda_device)
    out = check(moe, x, L, shape, 128, residual=True, max_tokens=13)
    m = moe.MoEFewLayer(L, shape, 128, max_tokens=13)
    got = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m(x, out=got, residual=True)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("E,H", [(3, 640), (100, 384), (256, 1024)])
def test_router_in_the_layer_kernel(moe, cuda_device, T, E, H):
    """Experts that do not divide among a cluster's CTAs, more than one round of warps, each count of columns."""
    shape = shape_of(H, E, min(E, 4), 128, 128)
    assert moe.few_kernel_launches(shape, T, 32) == 2
    L = make_layer(shape, 32, "f32", seed=E, device=cuda_device)
    check(moe, tokens(T, shape, L, 40 + T, cuda_device), L, shape, 32)


def test_router_placement_differs_by_pass(moe, cuda_device):
    """A full pass whose x does not fit beside the rings (logits kernel in front), then a short one where it does."""
    shape = shape_of(4096, 16, 2, 128, 0)
    assert moe.few_pass_tokens(shape, 128) == 8
    assert [moe.few_kernel_launches(shape, t, 128) for t in (2, 8, 10, 16)] == [2, 3, 5, 6]
    sizes = [moe.few_workspace_bytes(shape, t, 128) for t in range(1, 12)]
    assert sizes == sorted(sizes)
    L = make_layer(shape, 128, "bf16", device=cuda_device)
    check(moe, tokens(10, shape, L, 51, cuda_device), L, shape, 128, max_tokens=10)


@pytest.mark.parametrize("stype,group", [("bf16", 128), ("f32", 32)])
def test_tokens_that_share_a_column(moe, cuda_device, stype, group):
    """Tokens q and q + 4 with the same picks, with one pick in common, and with none."""
    shape = shape_of(256, 16, 2, 128, 128)
    L = make_layer(shape, group, stype, seed=3, device=cuda_device)
    x = tokens(8, shape, L, 61, cuda_device)
    for other in ([0, 1, 2, 3, 0, 1, 2, 3], [0, 1, 2, 3, 4, 1, 6, 3], [0, 0, 0, 0, 0, 0, 0, 0], list(range(8))):
        y = x[other].contiguous()
        out = check(moe, y, L, shape, group)
        for t, s in enumerate(other):  # equal tokens, equal rows
            assert torch.equal(out[t], out[other.index(s)])


@pytest.mark.parametrize("T", [1, 3, 8])
def test_every_word_of_the_picks_table_is_in_range(moe, cuda_device, T):
    """The table at the workspace's start (count, experts, token masks, slots): unused entries too name an expert and a
    slot, so that no mix of two tables leads out of the weights or the workspace."""
    shape = shape_of(256, 12, 3, 128, 128)
    L = make_layer(shape, 64, "bf16", device=cuda_device)
    m = moe.MoEFewLayer(L, shape, 64)
    x = tokens(T, shape, L, 71, cuda_device)
    idx = torch.empty((T, 3), dtype=torch.int32, device=cuda_device)
    m(x, topk_idx=idx)
    table = m.workspace[:4 * 257].cpu()
    words, slots = table.view(torch.int32), table[4 * 129:].view(torch.int8).view(64, 8)
    used = sorted(set(idx.flatten().tolist()))
    assert int(words[0]) == len(used) and words[1:1 + len(used)].tolist() == used
    assert bool(((words[1:65] >= 0) & (words[1:65] < 12)).all())
    assert bool((slots >= 0).all() and (slots < T * 3).all())
    for t in range(T):
        for k, e in enumerate(idx[t].tolist()):
            u = used.index(e)
            assert int(slots[u, t]) == t * 3 + k and (int(words[65 + u]) >> t) & 1

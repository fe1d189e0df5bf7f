"""moe_linear_forward on the GPU against the 64-bit product."""
import pytest
import torch

from tests._group_int4 import block_max, codes, gen, linear64, linear_bound, linear_rms, scales, weights64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import int4_expert_ffn_sigmoid_b200 as m
    return m


def check(out, x, w, s, group, add=None):
    want, b = linear64(x, w, s, group, add), linear_bound(x, w, s, group, add)
    if out.dtype == torch.bfloat16:  # one rounding: half a step, 2^-8 of the value
        b = b + 2.0 ** -8 * (want.abs() + b)
    off = (out.double() - want).abs()
    assert bool((off <= b + 1e-37).all()), float((off / (b + 1e-37)).max())


def make(T, N, K, group, stype, seed, add, dev):
    g = gen(seed, dev)
    x = torch.randn((T, K), generator=g, device=dev).to(torch.bfloat16)
    w, s = codes(g, N, K // 2), scales(g, (N,), K, group, stype)
    a = torch.randn((T, N), generator=g, device=dev).to(torch.bfloat16) if add else None
    return x, w, s, a


CASES = [
    # T, N, K, group, scales
    (1, 1, 32, 32, "f32"), (1, 1, 32, 0, "f32"), (1, 16, 64, 64, "bf16"), (2, 17, 96, 64, "f16"),
    (3, 7, 256, 32, "f32"), (4, 100, 288, 32, "bf16"), (5, 129, 512, 128, "f16"), (6, 40, 544, 256, "f32"),
    (7, 1000, 1120, 64, "bf16"), (8, 513, 1024, 32, "f32"), (8, 16, 8192, 512, "f16"), (1, 5001, 1120, 64, "f16"),
    (1, 2048, 2048, 0, "f32"), (2, 333, 4096, 1024, "bf16"), (1, 3, 32768, 128, "f32"), (8, 48, 32768, 32768, "f32"),
    (1, 1024, 1024, 128, "bf16"), (4, 6144, 2048, 32, "f32"), (3, 10240, 256, 32, "bf16"), (5, 31, 32, 128, "f32"),
    (9, 64, 128, 32, "f32"), (10, 1, 96, 32, "f16"), (16, 640, 2048, 128, "bf16"), (17, 129, 160, 64, "f32"),
    (31, 255, 1120, 64, "f16"), (33, 1000, 992, 32, "f32"), (64, 1024, 1024, 0, "f32"), (64, 130, 6144, 128, "bf16"),
    (65, 384, 736, 256, "f16"), (100, 77, 4096, 32, "f32"), (128, 512, 512, 64, "bf16"), (130, 257, 2048, 128, "f32"),
    (257, 200, 320, 32, "bf16"), (300, 1024, 1024, 128, "f16"), (513, 300, 96, 0, "f32"), (1025, 129, 256, 32, "f32"),
]


@pytest.mark.parametrize("T,N,K,group,stype", CASES)
def test_matches_product(moe, cuda_device, T, N, K, group, stype):
    x, w, s, a = make(T, N, K, group, stype, T * 131 + N * 7 + K, N % 2 == 0, cuda_device)
    lin = moe.Int4Linear(w, s, group)
    out32 = lin(x, add=a, flags=moe.MOE_OUT_F32)
    out = lin(x, add=a)
    check(out32, x, w, s, group, a)
    check(out, x, w, s, group, a)
    # the bf16 result is the f32 one, rounded once
    assert torch.equal(out, out32.to(torch.bfloat16))
    # and the same call gives the same bits
    assert torch.equal(out32, lin(x, add=a, flags=moe.MOE_OUT_F32))
    if N * T >= 4096:
        want = linear64(x, w, s, group, a)
        assert float((out32.double() - want).norm() / want.norm()) <= linear_rms(T, *w.shape)


@pytest.mark.parametrize("T", [1, 4, 8, 20, 150])
def test_strided_rows(moe, cuda_device, T):
    N, K, group = 200, 416, 32
    x, w, s, a = make(T, N, K, group, "bf16", 5, True, cuda_device)
    xs = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    xs[:, 16:16 + K] = x
    wide = torch.full((T, 3 * N + 1), 7.0, dtype=torch.bfloat16, device=cuda_device)
    base = wide.clone()
    aw = torch.full((T, N + 5), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    aw[:, 3:3 + N] = a
    lin = moe.Int4Linear(w, s, group)
    got = lin(xs[:, 16:16 + K], out=wide[:, N + 1:2 * N + 1], add=aw[:, 3:3 + N])
    check(got, x, w, s, group, a)
    base[:, N + 1:2 * N + 1] = got
    assert torch.equal(wide, base)  # nothing beside the columns was written
    # in place: the running sum is also the output
    run = a.clone()
    lin(x, out=run, add=run)
    assert torch.equal(run, got)


@pytest.mark.parametrize("T", [3, 40])
def test_guard_rows(moe, cuda_device, T):
    """Rows behind the last token and bytes before the first are left as they were."""
    N, K = 77, 160
    x, w, s, _ = make(T, N, K, 32, "f32", 9, False, cuda_device)
    big = torch.full((T + 4, N), 3.0, dtype=torch.bfloat16, device=cuda_device)
    moe.linear_forward(x, w, s, 32, out=big[2:2 + T])
    assert bool((big[:2] == 3).all()) and bool((big[2 + T:] == 3).all())
    check(big[2:2 + T], x, w, s, 32)


@pytest.mark.parametrize("T", [1, 8, 24])
def test_values(moe, cuda_device, T):
    """Zero, negative, tiny and large scales (one range a row); rows of zeros; activations of very different sizes."""
    N, K, group = 96, 512, 64
    x, w, s, _ = make(T, N, K, group, "f32", 21, False, cuda_device)
    s[0::6] = 0
    s[1::6] *= -1
    s[2::6] *= 1e-18
    s[3::6] *= 1e15
    w[4::6] = 0x88  # every code -8
    x[:, 7] *= 3000  # an outlier column
    x[0, 256:] = 0
    if T > 1:
        x[1] *= 1e-20
        x[2] *= 2.0 ** 60
        x[3] = 0
    out = moe.linear_forward(x, w, s, group, flags=moe.MOE_OUT_F32)
    check(out, x, w, s, group)
    assert bool((out[:, 0::6] == 0).all())
    if T > 1:
        assert bool((out[3] == 0).all())


@pytest.mark.parametrize("T", [2, 8, 30, 140])
def test_non_finite_rows(moe, cuda_device, T):
    """A token that holds NaN or an infinity gives no number anywhere; the others are untouched."""
    N, K, group = 130, 512, 32
    x, w, s, _ = make(T, N, K, group, "bf16", 33, False, cuda_device)
    lin = moe.Int4Linear(w, s, group)
    clean = lin(x)
    bad = x.clone()
    bad[0, 300] = float("nan")
    bad[T - 1, 5] = float("inf")
    out = lin(bad)
    assert bool((~torch.isfinite(out[0])).all()) and bool((~torch.isfinite(out[T - 1])).all())
    assert torch.equal(out[1:T - 1], clean[1:T - 1])


def test_no_tokens(moe, cuda_device):
    x, w, s, _ = make(0, 64, 64, 32, "f32", 1, False, cuda_device)
    assert moe.linear_forward(x, w, s, 32).shape == (0, 64)


def test_long_offsets(moe, cuda_device):
    """Codes and outputs past 2^32 bytes: rows at both ends and around the borders."""
    N, K, T = 300_000, 32768, 2
    g = gen(3, cuda_device)
    w = torch.randint(-2 ** 63, 2 ** 63 - 1, (N * K // 16,), generator=g, device=cuda_device).view(torch.uint8).view(N, K // 2)
    s = scales(g, (N,), K, 128, "bf16")
    x = torch.randn((T, K), generator=g, device=cuda_device).to(torch.bfloat16)
    out = moe.linear_forward(x, w, s, 128)
    edge = 2 ** 32 // (K // 2)  # the row that crosses 2^32 bytes
    rows = torch.tensor([0, 1, edge // 2 - 1, edge // 2, edge - 1, edge, edge + 1, N - 17, N - 2, N - 1], device=cuda_device)
    check(out[:, rows], x, w[rows], s[rows], 128)


@pytest.mark.parametrize("T", [1, 6, 48])
def test_two_calls_at_once(moe, cuda_device, T):
    N, K = 3001, 2048
    x, w, s, a = make(T, N, K, 128, "bf16", 4, True, cuda_device)
    lin = moe.Int4Linear(w, s, 128)
    want = lin(x, add=a)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o in zip(streams, outs):
            lin(x, out=o, add=a, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("T", [1, 8, 70])
def test_graph_replay(moe, cuda_device, T):
    N, K = 500, 1024
    x, w, s, _ = make(T, N, K, 32, "f16", 8, False, cuda_device)
    lin = moe.Int4Linear(w, s, 32)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=cuda_device)
    lin(x, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin(x, out=out)
    for seed in range(3):
        x.copy_(make(T, N, K, 32, "f16", 80 + seed, False, cuda_device)[0])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, w, s, 32)


def test_binding_refusals(moe, cuda_device):
    x, w, s, a = make(4, 64, 128, 32, "f32", 2, True, cuda_device)
    lin = moe.Int4Linear(w, s, 32)
    for bad in (x.float(), x[:, :96], x.cpu(), x[:1].expand(4, 128), x.t().contiguous().t()):
        with pytest.raises(ValueError):
            lin(bad)
    with pytest.raises(ValueError):
        lin(x, add=a[:2])
    with pytest.raises(ValueError):
        lin(x, out=torch.empty((4, 64), device=cuda_device))
    for args in ((w, s[:, :3], 32), (w, s.double(), 32), (w.cpu(), s, 32), (w, s, 64), (w[:, ::2], s, 32)):
        with pytest.raises(ValueError):
            moe.Int4Linear(*args)
    with pytest.raises(moe.MoeError):
        moe.Int4Linear(w, scales(gen(0, cuda_device), (64,), 128, 48), 48)  # not a power of two
    with pytest.raises(moe.MoeError):
        lin(x, out=x[:, :64])  # overlaps x


FIRST_CALL = """
import torch
import int4_expert_ffn_sigmoid_b200 as moe
from tests._group_int4 import codes, gen, make_layer, scales, shape_of
dev = torch.device("cuda:0")
g = gen(1, dev)
cases = [(1, 320, 1024), (6, 320, 1024), (40, 320, 1024), (300, 320, 1024)]
lins = [(moe.Int4Linear(codes(g, N, K // 2), scales(g, (N,), K, 32), 32), torch.randn((T, K), device=dev).bfloat16())
        for T, N, K in cases]
shape = shape_of(1024, 8, 2, 128, 128)
few = moe.MoEFewLayer(make_layer(shape, 32, device=dev), shape, 32)
v = torch.randn((2, 1024), device=dev).bfloat16()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = [l(x) for l, x in lins] + [few(v)]
graph.replay()
torch.cuda.synchronize()
for o, w in zip(outs, [l(x) for l, x in lins] + [few(v)]):
    assert torch.equal(o, w)
print("same")
"""


def test_first_call_inside_a_capture(cuda_device):
    """A process whose first calls are captured: nothing is set up outside."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_side_stream_tensors(moe, cuda_device):
    """Inputs made and outputs used on a stream of their own."""
    st = torch.cuda.Stream()
    x, w, s, a = make(5, 640, 512, 64, "bf16", 3, True, cuda_device)
    lin = moe.Int4Linear(w, s, 64)
    want = lin(x, add=a)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(50):
            y = x.clone()
            got = lin(y, add=a)
            del y
    st.synchronize()
    assert torch.equal(got, want)
    got = lin(x, add=a, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("stype,group", [("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("T,N,K", [
    # narrow to wide tiles of tokens, their columns in one CTA or shared out; the last tile of each seldom full
    (17, 128, 128), (17, 40, 8192), (300, 1000, 416), (20, 6200, 1184), (513, 130, 1184), (256, 130, 2048),
    (300, 2300, 416), (300, 1000, 1184), (40, 4100, 2048), (170, 500, 4096), (513, 2300, 416), (90, 6200, 4096),
    (120, 2300, 4096), (513, 4100, 416), (520, 4096, 6144),
])
def test_tiles(moe, cuda_device, T, N, K, stype, group):
    x, w, s, a = make(T, N, K, group, stype, T + N, True, cuda_device)
    out = moe.Int4Linear(w, s, group)(x, add=a, flags=moe.MOE_OUT_F32)
    check(out, x, w, s, group, a)
    want = linear64(x, w, s, group, a)
    assert float((out.double() - want).norm() / want.norm()) <= linear_rms(T, *w.shape)


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("N", [128, 130, 1003])
def test_wide_stores(moe, cuda_device, T, N):
    """Rows on 8- and 16-byte borders, with a last piece of rows that is not whole; f32 and bf16 outputs."""
    K, group = 1024, 128
    x, w, s, a = make(T, N, K, group, "bf16", 6, True, cuda_device)
    lin = moe.Int4Linear(w, s, group)
    wide = (N + 7) // 4 * 4
    aw = torch.full((T, wide), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    aw[:, :N] = a
    for flags, dtype in ((0, torch.bfloat16), (moe.MOE_OUT_F32, torch.float32)):
        for at in (0, 1):  # on a border, and beside it
            buf = torch.full((T * wide + 8,), 7.0, dtype=dtype, device=cuda_device)
            out = buf[at:at + T * wide].view(T, wide)[:, :N]
            lin(x, out=out, add=aw[:, :N], flags=flags)
            check(out, x, w, s, group, a)
            assert bool((buf[at:at + T * wide].view(T, wide)[:, N:] == 7).all())
            assert bool((buf[:at] == 7).all()) and bool((buf[at + T * wide:] == 7).all())


@pytest.mark.parametrize("stype,group", [("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("T", [1, 4, 8, 24])
def test_smallest_activations(moe, cuda_device, T, stype, group):
    """Blocks of 256 columns around 2^-113, below which activations are held to 2^-128 and no longer to 2^-15 of the
    block's largest; the scales bring the sums back into f32's normal range."""
    N, K = 96, 1536
    x, w, s, _ = make(T, N, K, group, stype, 41, False, cuda_device)
    s *= 2.0 ** 80
    g = gen(42, cuda_device)
    for b, e in enumerate((-112, -113, -114, -120, -126, -130)):  # magnitudes in [2^(e-1), 2^e)
        m = torch.randint(128, 256, (T, 256), generator=g, device=cuda_device).double() * 2.0 ** (e - 8)
        m *= torch.randint(0, 2, (T, 256), generator=g, device=cuda_device) * 2 - 1
        x[:, 256 * b:256 * (b + 1)] = m.to(torch.bfloat16)
    assert float(x[:, -256:].abs().max()) <= 2.0 ** -130 and float(x[:, -256:].abs().min()) > 0
    out = moe.linear_forward(x, w, s, group, flags=moe.MOE_OUT_F32)
    W = weights64(w, s, group).abs()
    mag = x.double().abs() @ W.t()
    held = (2.0 ** -15 * block_max(x, 256)).clamp(min=2.0 ** -128)
    b = held @ W.t() + (K / 16 + 64) * 2.0 ** -23 * mag
    if T > 8:  # x as it is, subnormal values among it; each weight rounded to bf16
        b = (2.0 ** -8 + 2.0 ** -16) * mag + (K / 16 + 64) * 2.0 ** -23 * mag
    off = (out.double() - linear64(x, w, s, group)).abs()
    assert bool((off <= b).all()), float((off / b).max())
    # a block below 2^-113 counts: alone, it gives more than its bound
    alone = x.clone()
    alone[:, :512], alone[:, 768:] = 0, 0
    want = linear64(alone, w, s, group)
    got = moe.linear_forward(alone, w, s, group, flags=moe.MOE_OUT_F32).double()
    assert float((got - want).norm() / want.norm()) <= (2.0 ** -12 if T <= 8 else 2.0 ** -8)

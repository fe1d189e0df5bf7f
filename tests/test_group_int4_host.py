"""Argument checks of the group-scaled int4 operators: every refusal comes before any CUDA call (fake pointers)."""
import ctypes
import os
import subprocess

import pytest
import torch

from tests._group_int4 import shape_of

FAKE = 1 << 24
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_int4.h")
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._load_build_module().build()
    import int4_expert_ffn_sigmoid_b200 as m
    return m


def linear(moe, T=0, N=64, K=128, group=32, stype=0, flags=0, ldx=0, ldo=0, lda=0, x=FAKE, w=2 * FAKE, s=3 * FAKE,
           add=None, out=4 * FAKE, size=None):
    c = moe.moe_linear_cfg_t(struct_size=ctypes.sizeof(moe.moe_linear_cfg_t) if size is None else size, N=N, K=K,
                             group=group, scale_type=stype, flags=flags, ldx=ldx, ldo=ldo, lda=lda)
    return moe.lib.moe_linear_forward(vp(x), vp(w), vp(s), vp(add), vp(out), T, ctypes.byref(c), None)


def test_linear_refusals(moe):
    INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert linear(moe) == 0  # T = 0: nothing to do
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(N=0), dict(K=0), dict(stype=3), dict(stype=-1), dict(flags=1),
               dict(flags=1 << 12), dict(size=8), dict(x=0), dict(w=0), dict(s=0), dict(out=0), dict(x=FAKE + 8),
               dict(w=FAKE + 8), dict(s=FAKE + 4), dict(out=4 * FAKE + 1), dict(add=4 * FAKE + 1), dict(ldx=120),
               dict(ldo=63), dict(lda=63), dict(ldx=-128), dict(ldx=1 << 41), dict(out=4 * FAKE + 2, flags=16)):
        assert linear(moe, **kw) == INV, kw
    for kw in (dict(group=16), dict(group=48), dict(group=-32), dict(group=65536), dict(K=48), dict(K=32800),
               dict(N=(1 << 20) + 1), dict(ldx=132)):
        assert linear(moe, **kw) == UNS, kw
    # overlaps: out with x, w, scales or a different add
    assert linear(moe, T=4, out=FAKE + 16) == INV
    assert linear(moe, T=4, out=2 * FAKE) == INV
    assert linear(moe, T=4, out=3 * FAKE) == INV
    assert linear(moe, T=4, add=4 * FAKE + 2) == INV
    assert linear(moe, T=4, add=4 * FAKE, flags=moe.MOE_OUT_F32) == INV
    assert linear(moe, T=4, add=4 * FAKE, lda=128) == INV
    assert moe.lib.moe_linear_forward(None, None, None, None, None, 0, None, None) == INV


def test_linear_launches(moe):
    assert moe.linear_kernel_launches(64, 128, 0, 32) == 0
    assert moe.linear_kernel_launches(64, 128, 1, 32) == 1
    assert moe.linear_kernel_launches(64, 100, 1, 32) == 0
    assert moe.linear_kernel_launches(64, 128, 500, 0) >= 1


def few(moe, shape=None, T=0, group=32, flags=0, x=FAKE, out=4 * FAKE, ws=8 * FAKE, ws_bytes=1 << 40, null=None,
        patch=None, wpatch=None):
    shape = shape or shape_of(256, 8, 2, 128, 128)
    c = moe.make_few_cfg(shape, group, 0, flags)
    c.workspace, c.workspace_bytes = ws, ws_bytes
    if patch:
        patch(c)
    w = moe.moe_few_weights_t(**{n: 2 * FAKE for n, _ in moe.moe_few_weights_t._fields_})
    if null:
        setattr(w, null, None)
    if wpatch:
        wpatch(w)
    return moe.lib.moe_few_forward(vp(x), ctypes.byref(w), vp(out), T, ctypes.byref(c), None)


def test_few_refusals(moe):
    INV, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
    assert few(moe) == 0
    for n, _ in moe.moe_few_weights_t._fields_:
        assert few(moe, null=n) == INV, n
    assert few(moe, shape_of(256, 8, 2, 128, 0), null="sh_w2") == 0
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(x=0), dict(out=0), dict(x=FAKE + 8), dict(out=FAKE + 8),
               dict(ws=8 * FAKE + 16), dict(flags=moe.MOE_FORCE_DECODE), dict(flags=1 << 12), dict(flags=moe.MOE_TRACE),
               dict(T=4, out=FAKE), dict(patch=lambda c: setattr(c, "struct_size", 4)),
               dict(patch=lambda c: setattr(c, "scale_type", 5)), dict(patch=lambda c: setattr(c, "topp", -1.0)),
               dict(patch=lambda c: setattr(c, "topp", float("nan"))),
               dict(patch=lambda c: setattr(c, "routed_scaling", 0.0)),
               dict(patch=lambda c: setattr(c, "topk_idx_out", FAKE + 4)),
               dict(wpatch=lambda w: setattr(w, "s13", FAKE + 8)), dict(shape=shape_of(256, 2, 3, 128, 0))):
        assert few(moe, **kw) == INV, kw
    for s in (shape_of(200, 8, 2, 128, 0), shape_of(16512, 8, 2, 128, 0), shape_of(256, 300, 2, 128, 0),
              shape_of(256, 16, 9, 128, 0), shape_of(256, 8, 2, 100, 0), shape_of(256, 8, 2, 128, 100)):
        assert few(moe, s) == UNS
        assert moe.few_workspace_bytes(s, 4, 32) == 0 and moe.few_pass_tokens(s, 32) == 0
    assert few(moe, group=33) == UNS
    assert few(moe, T=2, ws=0) == WS and few(moe, T=2, ws_bytes=64) == WS
    assert moe.lib.moe_few_forward(None, None, None, 0, None, None) == INV


def test_few_sizes(moe):
    s = shape_of(1024, 64, 2, 512, 2048)
    p = moe.few_pass_tokens(s, 32)
    assert p >= 1 and moe.few_workspace_bytes(s, 0, 32) > 0
    sizes = [moe.few_workspace_bytes(s, t, 32) for t in range(1, 40)]
    assert sizes == sorted(sizes) and sizes[p - 1] == sizes[-1]  # passes reuse one workspace
    one = moe.few_kernel_launches(s, 1, 32)
    assert one >= 1 and moe.few_kernel_launches(s, 0, 32) == 0
    assert moe.few_kernel_launches(s, p, 32) == one and moe.few_kernel_launches(s, p + 1, 32) == 2 * one


def test_struct_layouts(moe, tmp_path):
    src = tmp_path / "layout.c"
    fields = [("moe_linear_cfg_t", ("group", "flags", "ldx", "lda")),
              ("moe_few_cfg_t", ("routed_scaling", "topp", "group", "flags", "workspace", "topk_w_out")),
              ("moe_few_weights_t", ("w13", "sh_s2"))]
    body = "".join(f'printf("%zu ", sizeof({t}));' + "".join(f'printf("%zu ", offsetof({t}, {f}));' for f in fs)
                   for t, fs in fields)
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "moe_int4.h"\nint main(void){{{body} return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    want = []
    for t, fs in fields:
        cls = getattr(moe, t)
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fs]
    assert got == want


def test_binding_refuses_host_tensors(moe):
    with pytest.raises(ValueError):
        moe.Int4Linear(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 1)), 32)
    with pytest.raises(ValueError):
        moe.Int4Linear(torch.zeros(16, dtype=torch.uint8), torch.zeros((4, 1)), 32)


def test_few_refuses_overlaps(moe):
    """out, the workspace and the pick outputs meet nothing else that the call reads or writes."""
    INV = moe.MOE_ERR_INVALID_ARG
    shape = shape_of(256, 8, 2, 128, 128)
    reads = [n for n, _ in moe.moe_few_weights_t._fields_]
    at = {n: (20 + i) << 20 for i, n in enumerate(reads)}  # every tensor a MB of its own

    def call(out=0, ws=1 << 20, idx=2 << 20, w=3 << 20, x=4 << 20, flags=0, T=8):
        def spread(p):
            for n, a in at.items():
                setattr(p, n, a)

        def picks(c):
            c.topk_idx_out, c.topk_w_out = idx, w
        return few(moe, shape, T, out=out, ws=ws, x=x, flags=flags, patch=picks, wpatch=spread)

    ws_bytes = moe.few_workspace_bytes(shape, 8, 32)
    sizes = {"router_w": 8 * 256 * 4, "router_bias": 8 * 4, "w13": 8 * 256 * 128, "s13": 8 * 256 * 8 * 4,
             "w2": 8 * 256 * 64, "s2": 8 * 256 * 4 * 4, "sh_w13": 256 * 128, "sh_s13": 256 * 8 * 4, "sh_w2": 256 * 64,
             "sh_s2": 256 * 4 * 4}
    assert set(sizes) == set(reads)
    for n, size in sizes.items():
        first, last = at[n], at[n] + size - 16
        assert call(out=first) == INV and call(out=last) == INV and call(out=first - 16) == INV, n
        assert call(out=1 << 20, ws=first) == INV, n
        assert call(out=64 << 20, idx=first) == INV and call(out=64 << 20, w=last) == INV, n
    out = 64 << 20
    assert call(out=out, ws=out) == INV and call(out=out, ws=out - ws_bytes // 256 * 256 + 256) == INV
    assert call(out=out, idx=out + 8 * 256 * 2 - 16) == INV and call(out=out, flags=moe.MOE_OUT_F32, w=out + 8 * 256 * 2) == INV
    assert call(out=out, idx=3 << 20, w=3 << 20) == INV and call(out=out, ws=4 << 20) == INV and call(out=out, idx=4 << 20) == INV
    assert call(out=4 << 20, T=0) == 0  # nothing is read or written


def test_full_weights_flag(moe):
    import re
    with open(HEADER) as f:
        bit = re.search(r"#define MOE_FULL_WEIGHTS \(1u << (\d+)\)", f.read())
    assert moe.MOE_FULL_WEIGHTS == 1 << int(bit.group(1))
    f = moe.MOE_FULL_WEIGHTS
    for flags in (f, f | moe.MOE_OUT_F32, moe.MOE_TEST_STALL, f | moe.MOE_TEST_STALL):
        assert linear(moe, flags=flags) == 0  # T = 0: nothing to do
    assert linear(moe, flags=f | moe.MOE_ADD_RESIDUAL) == moe.MOE_ERR_INVALID_ARG
    assert few(moe, flags=f) == moe.MOE_ERR_INVALID_ARG  # always streams
    assert few(moe, flags=moe.MOE_TEST_STALL) == moe.MOE_ERR_INVALID_ARG

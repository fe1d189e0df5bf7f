"""B200 (sm_100a) forward pass of one int4 expert-FFN MoE layer with a
sigmoid+bias router: the Python binding of ``libmoe_int4.so``.

This module only marshals arguments: every step of the layer (router,
selection, bucketing, expert FFNs, shared expert, combine) runs in the
library's CUDA kernels.  torch provides device memory and streams.  There is
no fallback: if the library is missing, importing the binding raises.

The C ABI is declared in ``include/moe_int4.h``; the names here mirror it.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "MoeError", "moe_cfg_t", "moe_shared_weights_t", "lib", "EXPORTED_SYMBOLS",
    "MOE_ADD_RESIDUAL", "MOE_DEBUG_CHECK", "MOE_FORCE_DECODE", "MOE_FORCE_PREFILL", "MOE_OUT_F32",
    "MOE_TEST_STALL", "MOE_LOOKAHEAD", "MOE_TEST_BAD_INDEX", "MOE_TRACE", "MOE_DEBUG_POISON", "MOE_STACK_FUSED",
    "MOE_WEIGHTS_INT8", "weight_flags",
    "MOE_DEVSTAT_TIMEOUT", "MOE_DEVSTAT_BAD_EXPERT", "device_status", "stack_trace",
    "moe_stack_weights_t", "stack_workspace_bytes", "stack_path", "stack_forward", "stack_layers",
    "MOE_PATH_FUSED_STACK", "MOE_PATH_PER_LAYER",
    "workspace_bytes", "workspace_bytes_upto", "layer_forward", "MoELayer", "decode_max_tokens", "kernel_launches", "layer_path",
    "MOE_PATH_SMALL_BATCH", "MOE_PATH_TENSOR_CORE", "MOE_PATH_LARGE_STREAMING", "LIB_PATH",
    "moe_linear_cfg_t", "moe_few_cfg_t", "moe_few_weights_t", "MOE_SCALE_F32", "MOE_SCALE_BF16", "MOE_SCALE_F16",
    "MOE_FULL_WEIGHTS",
    "linear_forward", "linear_kernel_launches", "Int4Linear",
    "few_forward", "few_workspace_bytes", "few_pass_tokens", "few_kernel_launches", "MoEFewLayer",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_int4.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_CHECK = 5

MOE_ADD_RESIDUAL = 1 << 0
MOE_DEBUG_CHECK = 1 << 1
MOE_FORCE_DECODE = 1 << 2
MOE_FORCE_PREFILL = 1 << 3
MOE_OUT_F32 = 1 << 4
MOE_LOOKAHEAD = 1 << 5
MOE_TEST_STALL = 1 << 6
MOE_TEST_BAD_INDEX = 1 << 7
MOE_TRACE = 1 << 8
MOE_DEBUG_POISON = 1 << 9
MOE_STACK_FUSED = 1 << 10
MOE_WEIGHTS_INT8 = 1 << 11
MOE_FULL_WEIGHTS = 1 << 13
TRACE_SLOTS = 16  # MOE_TRACE stamps per (CTA, layer)
# device status word (the first 4 bytes of the workspace)
MOE_DEVSTAT_BAD_EXPERT = 1 << 0
MOE_DEVSTAT_BAD_SLOT = 1 << 1
MOE_DEVSTAT_BAD_COUNT = 1 << 2
MOE_DEVSTAT_BAD_TASK = 1 << 3
MOE_DEVSTAT_TIMEOUT = 1 << 4
# kernel sequences (moe_layer_path)
MOE_PATH_SMALL_BATCH = 1
MOE_PATH_TENSOR_CORE = 2
MOE_PATH_LARGE_STREAMING = 3
MOE_PATH_FUSED_STACK = 4
MOE_PATH_PER_LAYER = 5

# scale types of the group-scaled int4 operators
MOE_SCALE_F32, MOE_SCALE_BF16, MOE_SCALE_F16 = range(3)

MOE_STAGE_ROUTE, MOE_STAGE_GATE_UP, MOE_STAGE_DOWN, MOE_STAGE_COMBINE = range(4)
MOE_NUM_STAGES = 4
STAGE_NAMES = ("route", "gate_up", "down", "combine")

# Every function declared in include/moe_int4.h.
EXPORTED_SYMBOLS = ("moe_layer_workspace_bytes", "moe_layer_forward", "moe_status_str",
                    "moe_abi_version", "moe_decode_max_tokens", "moe_layer_forward_static_ws",
                    "moe_layer_kernel_launches", "moe_layer_path", "moe_layer_workspace_bytes_upto",
                    "moe_stack_workspace_bytes", "moe_stack_path", "moe_stack_forward", "moe_stack_trace_offset",
                    "moe_linear_forward", "moe_linear_kernel_launches", "moe_few_workspace_bytes",
                    "moe_few_pass_tokens", "moe_few_kernel_launches", "moe_few_forward")

# Scratch capacity of moe_layer_forward_static_ws (the entry point for callers
# that cannot allocate device memory).
MOE_STATIC_WORKSPACE_BYTES = 32 << 20


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str = "moe_layer_forward"):
        self.status = status
        super().__init__(f"{what} failed: {status_str(status)} ({status})")


class moe_cfg_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("Is", ctypes.c_int32),
                ("routed_scaling", ctypes.c_float), ("flags", ctypes.c_uint32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("topk_idx_out", ctypes.c_void_p), ("topk_w_out", ctypes.c_void_p),
                ("stage_events", ctypes.c_void_p), ("topp", ctypes.c_float)]


class moe_shared_weights_t(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("s13", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p)]


class moe_stack_weights_t(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("w13", ctypes.c_void_p), ("s13", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("shared", moe_shared_weights_t)]


class moe_linear_cfg_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("group", ctypes.c_int32), ("scale_type", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("ldx", ctypes.c_int64), ("ldo", ctypes.c_int64), ("lda", ctypes.c_int64)]


class moe_few_cfg_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("Is", ctypes.c_int32),
                ("routed_scaling", ctypes.c_float), ("topp", ctypes.c_float), ("group", ctypes.c_int32),
                ("scale_type", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("topk_idx_out", ctypes.c_void_p), ("topk_w_out", ctypes.c_void_p)]


class moe_few_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("router_w", "router_bias", "w13", "s13", "w2", "s2",
                                               "sh_w13", "sh_s13", "sh_w2", "sh_s2")]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python int4_expert_ffn_sigmoid_b200/_build.py`")
    L = ctypes.CDLL(LIB_PATH)
    vp = ctypes.c_void_p
    L.moe_layer_workspace_bytes.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32]
    L.moe_layer_workspace_bytes.restype = ctypes.c_size_t
    L.moe_layer_workspace_bytes_upto.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32]
    L.moe_layer_workspace_bytes_upto.restype = ctypes.c_size_t
    L.moe_layer_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(moe_shared_weights_t),
                                    vp, ctypes.c_int32, ctypes.POINTER(moe_cfg_t), vp]
    L.moe_layer_forward.restype = ctypes.c_int
    L.moe_layer_forward_static_ws.argtypes = L.moe_layer_forward.argtypes
    L.moe_layer_forward_static_ws.restype = ctypes.c_int
    L.moe_status_str.argtypes = [ctypes.c_int]
    L.moe_status_str.restype = ctypes.c_char_p
    L.moe_abi_version.argtypes = []
    L.moe_abi_version.restype = ctypes.c_int
    L.moe_decode_max_tokens.argtypes = []
    L.moe_decode_max_tokens.restype = ctypes.c_int32
    L.moe_layer_kernel_launches.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32]
    L.moe_layer_kernel_launches.restype = ctypes.c_int32
    L.moe_layer_path.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32]
    L.moe_layer_path.restype = ctypes.c_int32
    L.moe_stack_workspace_bytes.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32, ctypes.c_int32]
    L.moe_stack_workspace_bytes.restype = ctypes.c_size_t
    L.moe_stack_path.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32, ctypes.c_int32]
    L.moe_stack_path.restype = ctypes.c_int32
    L.moe_stack_forward.argtypes = [vp, ctypes.POINTER(moe_stack_weights_t), ctypes.c_int32, vp, ctypes.c_int32,
                                    ctypes.POINTER(moe_cfg_t), vp]
    L.moe_stack_forward.restype = ctypes.c_int
    L.moe_stack_trace_offset.argtypes = [ctypes.POINTER(moe_cfg_t), ctypes.c_int32, ctypes.c_int32]
    L.moe_stack_trace_offset.restype = ctypes.c_size_t
    lin, few = ctypes.POINTER(moe_linear_cfg_t), ctypes.POINTER(moe_few_cfg_t)
    L.moe_linear_forward.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int32, lin, vp]
    L.moe_linear_forward.restype = ctypes.c_int
    L.moe_linear_kernel_launches.argtypes = [lin, ctypes.c_int32]
    L.moe_linear_kernel_launches.restype = ctypes.c_int32
    L.moe_few_workspace_bytes.argtypes = [few, ctypes.c_int32]
    L.moe_few_workspace_bytes.restype = ctypes.c_size_t
    L.moe_few_pass_tokens.argtypes = [few]
    L.moe_few_pass_tokens.restype = ctypes.c_int32
    L.moe_few_kernel_launches.argtypes = [few, ctypes.c_int32]
    L.moe_few_kernel_launches.restype = ctypes.c_int32
    L.moe_few_forward.argtypes = [vp, ctypes.POINTER(moe_few_weights_t), vp, ctypes.c_int32, few, vp]
    L.moe_few_forward.restype = ctypes.c_int
    if L.moe_abi_version() != 2:
        raise ImportError("libmoe_int4.so ABI version mismatch")
    return L


lib = _load()


def status_str(status: int) -> str:
    return lib.moe_status_str(int(status)).decode()


def decode_max_tokens() -> int:
    return int(lib.moe_decode_max_tokens())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_cfg(shape, flags: int = 0, workspace: Optional[torch.Tensor] = None,
             topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
             stage_events=None, topp: float = 0.0) -> moe_cfg_t:
    c = moe_cfg_t()
    c.topp = float(topp)
    c.struct_size = ctypes.sizeof(moe_cfg_t)
    c.H, c.E, c.K, c.I, c.Is = shape.H, shape.E, shape.K, shape.I, shape.Is
    c.routed_scaling = float(shape.routed_scaling)
    c.flags = int(flags)
    if workspace is not None:
        c.workspace = workspace.data_ptr()
        c.workspace_bytes = workspace.numel() * workspace.element_size()
    c.topk_idx_out = None if topk_idx is None else topk_idx.data_ptr()
    c.topk_w_out = None if topk_w is None else topk_w.data_ptr()
    if stage_events is not None:
        if len(stage_events) != 2 * MOE_NUM_STAGES:
            raise ValueError(f"stage_events needs {2 * MOE_NUM_STAGES} events")
        arr = (ctypes.c_void_p * len(stage_events))(*[int(e.cuda_event) for e in stage_events])
        c._events_keepalive = arr
        c.stage_events = ctypes.cast(arr, ctypes.c_void_p).value
    return c


def kernel_launches(shape, T: int, flags: int = 0) -> int:
    """Kernels one layer_forward call launches for T tokens (0: invalid)."""
    c = make_cfg(shape, flags)
    return int(lib.moe_layer_kernel_launches(ctypes.byref(c), int(T)))


def layer_path(shape, T: int, flags: int = 0) -> int:
    """MOE_PATH_* of a layer_forward call for T tokens (0: invalid)."""
    c = make_cfg(shape, flags)
    return int(lib.moe_layer_path(ctypes.byref(c), int(T)))


def workspace_bytes(shape, T: int, flags: int = 0) -> int:
    c = make_cfg(shape, flags)
    return int(lib.moe_layer_workspace_bytes(ctypes.byref(c), int(T)))


def workspace_bytes_upto(shape, T: int, flags: int = 0) -> int:
    c = make_cfg(shape, flags)
    return int(lib.moe_layer_workspace_bytes_upto(ctypes.byref(c), int(T)))


def new_workspace(shape, T: int, device, flags: int = 0) -> torch.Tensor:
    """A workspace for any call of up to T tokens under `flags`."""
    n = workspace_bytes_upto(shape, T, flags)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_layer_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _check_dev(name, t, dtype, shape=None):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def weight_flags(layer: dict, shape) -> int:
    """MOE_WEIGHTS_INT8 when ``layer``'s expert codes are one byte per element
    (w13 rows of H bytes), 0 for packed int4 (H/2 bytes)."""
    n = layer["w13"].shape[-1]
    if n == shape.H:
        return MOE_WEIGHTS_INT8
    if 2 * n == shape.H:
        return 0
    raise ValueError(f"w13 rows of {n} bytes fit neither int4 nor int8 codes of H={shape.H}")


def layer_forward(x: torch.Tensor, layer: dict, shape, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, flags: int = 0,
                  topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None, stage_events=None, topp: float = 0.0) -> torch.Tensor:
    """Call ``moe_layer_forward`` on torch tensors (see include/moe_int4.h).

    ``layer`` holds router_w, router_bias, w13, s13, w2, s2 and, when
    shape.Is > 0, sh_w13, sh_s13, sh_w2, sh_s2 (the layout of
    ``workloads.make_layer``).  With int8 expert weights (one byte per element)
    ``flags`` must hold MOE_WEIGHTS_INT8.  Returns ``out`` (bf16 [T, H]).  ``stage_events``:
    optional sequence of 2*MOE_NUM_STAGES ``torch.cuda.Event`` already recorded
    once (so that they exist); the library records them around each stage."""
    T = x.shape[0]
    H, E, I, Is = shape.H, shape.E, shape.I, shape.Is
    per = 1 if flags & MOE_WEIGHTS_INT8 else 2  # code elements per byte
    _check_dev("x", x, torch.bfloat16, (T, H))
    _check_dev("router_w", layer["router_w"], torch.float32, (E, H))
    _check_dev("router_bias", layer["router_bias"], torch.float32, (E,))
    _check_dev("w13", layer["w13"], torch.uint8, (E, 2 * I, H // per))
    _check_dev("s13", layer["s13"], torch.float32, (E, 2 * I))
    _check_dev("w2", layer["w2"], torch.uint8, (E, H, I // per))
    _check_dev("s2", layer["s2"], torch.float32, (E, H))
    sh = moe_shared_weights_t()
    if Is > 0:
        _check_dev("sh_w13", layer["sh_w13"], torch.uint8, (2 * Is, H // per))
        _check_dev("sh_s13", layer["sh_s13"], torch.float32, (2 * Is,))
        _check_dev("sh_w2", layer["sh_w2"], torch.uint8, (H, Is // per))
        _check_dev("sh_s2", layer["sh_s2"], torch.float32, (H,))
        sh.w13, sh.s13 = layer["sh_w13"].data_ptr(), layer["sh_s13"].data_ptr()
        sh.w2, sh.s2 = layer["sh_w2"].data_ptr(), layer["sh_s2"].data_ptr()
    odt = torch.float32 if flags & MOE_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((T, H), dtype=odt, device=x.device)
    _check_dev("out", out, odt, (T, H))
    if workspace is None:
        workspace = new_workspace(shape, T, x.device, flags)
    if topk_idx is not None:
        _check_dev("topk_idx", topk_idx, torch.int32, (T, shape.K))
    if topk_w is not None:
        _check_dev("topk_w", topk_w, torch.float32, (T, shape.K))
    cfg = make_cfg(shape, flags, workspace, topk_idx, topk_w, stage_events, topp)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    st = lib.moe_layer_forward(_ptr(x), _ptr(layer["router_w"]), _ptr(layer["router_bias"]),
                               _ptr(layer["w13"]), _ptr(layer["s13"]), _ptr(layer["w2"]),
                               _ptr(layer["s2"]), ctypes.byref(sh), _ptr(out), int(T),
                               ctypes.byref(cfg), ctypes.c_void_p(s.cuda_stream))
    if st != MOE_OK:
        raise MoeError(st)
    return out


STACK_KEYS = ("router_w", "router_bias", "w13", "s13", "w2", "s2", "sh_w13", "sh_s13", "sh_w2", "sh_s2")


def stack_layers(layers) -> dict:
    """Stacks per-layer weight dicts (``workloads.make_layer``'s layout) along a
    new leading layer dimension: the layout moe_stack_forward reads."""
    keys = [k for k in STACK_KEYS if k in layers[0]]
    return {k: torch.stack([l[k] for l in layers]).contiguous() for k in keys}


def stack_workspace_bytes(shape, T: int, L: int, flags: int = 0) -> int:
    c = make_cfg(shape, flags)
    return int(lib.moe_stack_workspace_bytes(ctypes.byref(c), int(T), int(L)))


def stack_path(shape, T: int, L: int, flags: int = 0) -> int:
    """MOE_PATH_FUSED_STACK or MOE_PATH_PER_LAYER of a stack_forward call (0: invalid)."""
    c = make_cfg(shape, flags)
    return int(lib.moe_stack_path(ctypes.byref(c), int(T), int(L)))


def stack_forward(x: torch.Tensor, stacked: dict, shape, outs: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, flags: int = 0,
                  topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None, topp: float = 0.0) -> torch.Tensor:
    """Call ``moe_stack_forward`` on torch tensors: ``stacked`` holds the
    weights of L layers stacked along dimension 0 (see ``stack_layers``).
    Returns ``outs`` (bf16 [L, T, H]; outs[l] is layer l's output).
    ``topk_idx`` / ``topk_w``: optional [L, T, K]."""
    T = x.shape[0]
    H, E, K, I, Is = shape.H, shape.E, shape.K, shape.I, shape.Is
    L = stacked["router_w"].shape[0]
    per = 1 if flags & MOE_WEIGHTS_INT8 else 2  # code elements per byte
    _check_dev("x", x, torch.bfloat16, (T, H))
    _check_dev("router_w", stacked["router_w"], torch.float32, (L, E, H))
    _check_dev("router_bias", stacked["router_bias"], torch.float32, (L, E))
    _check_dev("w13", stacked["w13"], torch.uint8, (L, E, 2 * I, H // per))
    _check_dev("s13", stacked["s13"], torch.float32, (L, E, 2 * I))
    _check_dev("w2", stacked["w2"], torch.uint8, (L, E, H, I // per))
    _check_dev("s2", stacked["s2"], torch.float32, (L, E, H))
    w = moe_stack_weights_t()
    w.router_w, w.router_bias = stacked["router_w"].data_ptr(), stacked["router_bias"].data_ptr()
    w.w13, w.s13 = stacked["w13"].data_ptr(), stacked["s13"].data_ptr()
    w.w2, w.s2 = stacked["w2"].data_ptr(), stacked["s2"].data_ptr()
    if Is > 0:
        _check_dev("sh_w13", stacked["sh_w13"], torch.uint8, (L, 2 * Is, H // per))
        _check_dev("sh_s13", stacked["sh_s13"], torch.float32, (L, 2 * Is))
        _check_dev("sh_w2", stacked["sh_w2"], torch.uint8, (L, H, Is // per))
        _check_dev("sh_s2", stacked["sh_s2"], torch.float32, (L, H))
        w.shared.w13, w.shared.s13 = stacked["sh_w13"].data_ptr(), stacked["sh_s13"].data_ptr()
        w.shared.w2, w.shared.s2 = stacked["sh_w2"].data_ptr(), stacked["sh_s2"].data_ptr()
    if outs is None:
        outs = torch.empty((L, T, H), dtype=torch.bfloat16, device=x.device)
    _check_dev("outs", outs, torch.bfloat16, (L, T, H))
    if workspace is None:
        n = stack_workspace_bytes(shape, T, L, flags)
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, "moe_stack_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    if topk_idx is not None:
        _check_dev("topk_idx", topk_idx, torch.int32, (L, T, K))
    if topk_w is not None:
        _check_dev("topk_w", topk_w, torch.float32, (L, T, K))
    cfg = make_cfg(shape, flags, workspace, topk_idx, topk_w, topp=topp)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    st = lib.moe_stack_forward(_ptr(x), ctypes.byref(w), int(L), _ptr(outs), int(T), ctypes.byref(cfg),
                               ctypes.c_void_p(s.cuda_stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_stack_forward")
    return outs


def stack_trace(workspace: torch.Tensor, shape, T: int, L: int, flags: int, grid: int) -> torch.Tensor:
    """The MOE_TRACE stamps of the last fused call on ``workspace``: int64
    [grid, L + 1, 16] nanosecond timer values, 0 where a CTA took no stamp
    (see moe_stack_trace_offset).  Synchronises the stream."""
    c = make_cfg(shape, flags | MOE_TRACE)
    off = int(lib.moe_stack_trace_offset(ctypes.byref(c), int(T), int(L)))
    if off == 0:
        raise ValueError("this call does not trace (not the fused kernel, or no MOE_TRACE)")
    n = grid * (L + 1) * TRACE_SLOTS
    return workspace[off:off + 8 * n].view(torch.int64).view(grid, L + 1, TRACE_SLOTS).cpu()


def device_status(workspace: torch.Tensor) -> int:
    """The device status word (MOE_DEVSTAT_* bits) that the last call on
    ``workspace`` left in its first 4 bytes (synchronises the stream)."""
    return int(workspace[:4].view(torch.int32).item()) & 0xFFFFFFFF


class MoELayer:
    """One layer's device weights plus a workspace sized for every call of up
    to ``max_tokens`` tokens under any per-call flags (the kernel sequence,
    and so the workspace, depends on MOE_FORCE_DECODE / MOE_FORCE_PREFILL).
    The code width of the expert weights (int4 or int8) is read from their
    shapes and its flag added to every call."""

    def __init__(self, layer: dict, shape, max_tokens: int, device=None):
        self.layer = layer
        self.shape = shape
        self.device = torch.device(device) if device is not None else layer["w13"].device
        self.max_tokens = int(max_tokens)
        self.weight_flags = weight_flags(layer, shape)
        n = max(workspace_bytes_upto(shape, self.max_tokens, f | self.weight_flags)
                for f in (0, MOE_FORCE_DECODE, MOE_FORCE_PREFILL))
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, "moe_layer_workspace_bytes")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, residual: bool = False,
                 flags: int = 0, topk_idx=None, topk_w=None, stage_events=None) -> torch.Tensor:
        if x.shape[0] > self.max_tokens:
            raise ValueError(f"T={x.shape[0]} exceeds max_tokens={self.max_tokens}")
        f = flags | self.weight_flags | (MOE_ADD_RESIDUAL if residual else 0)
        return layer_forward(x, self.layer, self.shape, out=out, workspace=self.workspace, flags=f,
                             topk_idx=topk_idx, topk_w=topk_w, stage_events=stage_events)


# ---------------------------------------------------------------------------
# Int4 weights with group scales (include/moe_int4.h)
# ---------------------------------------------------------------------------
_SCALE_TYPES = {torch.float32: MOE_SCALE_F32, torch.bfloat16: MOE_SCALE_BF16, torch.float16: MOE_SCALE_F16}


def _scale_type(name: str, scales: torch.Tensor) -> int:
    if scales.dtype not in _SCALE_TYPES:
        raise ValueError(f"{name}: expected float32, bfloat16 or float16 scales, got {scales.dtype}")
    return _SCALE_TYPES[scales.dtype]


def _scale_shape(rows, cols: int, group: int) -> tuple:
    """Shape of the scales of a matrix [*rows, cols]: [*rows, ceil(cols / group)], or [*rows] for group 0."""
    return (*rows, -(-cols // group)) if group else tuple(rows)


def _raw_stream(device: torch.device, stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _rows_of(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """The elements between rows of a 2-D tensor whose rows are contiguous (0: their length)."""
    if t.device != device or t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: expected a {dtype} tensor of shape {shape} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return 0
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: expected contiguous rows, got strides {t.stride()}")
    if shape[0] > 1:
        if t.stride(0) < shape[1]:
            raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
        return t.stride(0)
    return 0


class Int4Linear:
    """A dense projection with int4 weights and group scales (``moe_linear_forward``).

    ``w``: uint8 [N, K/2] packed codes; ``scales``: float32, bfloat16 or float16 [N, ceil(K/group)]
    ([N] with ``group`` = 0, one scale a row).  Calls may run at the same time, on any stream of the
    weights' device.  Weights are read before the kernel ahead on the stream has ended: PyTorch operations may
    write them there, kernels that start their dependents early (this library's among them) may not."""

    def __init__(self, w: torch.Tensor, scales: torch.Tensor, group: int = 128):
        if w.dim() != 2:
            raise ValueError(f"w: expected [N, K/2] codes, got shape {tuple(w.shape)}")
        self.N, self.K, self.group = w.shape[0], 2 * w.shape[1], int(group)
        if self.group < 0:
            raise ValueError(f"group: {group}")
        _check_dev("w", w, torch.uint8)
        _check_dev("scales", scales, scales.dtype, _scale_shape((self.N,), self.K, self.group))
        if scales.device != w.device:
            raise ValueError(f"w is on {w.device}, scales on {scales.device}")
        self.w, self.scales, self.device = w, scales, w.device
        self._w, self._s = w.data_ptr(), scales.data_ptr()
        self.cfg = moe_linear_cfg_t(struct_size=ctypes.sizeof(moe_linear_cfg_t), N=self.N, K=self.K, group=self.group,
                                    scale_type=_scale_type("scales", scales))
        self._cref, self._index = ctypes.byref(self.cfg), self.device.index
        if lib.moe_linear_kernel_launches(ctypes.byref(self.cfg), 1) == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, "moe_linear_forward")

    def __call__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                 flags: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """out[t] = W x[t] (+ add[t]).  x: bfloat16 [T, K], add: bfloat16 [T, N], out: bfloat16 (float32 under
        MOE_OUT_F32) [T, N]; each may have rows further apart than their length.  ``out`` may be ``add``.  Above eight
        tokens the weights are rounded to bf16 unless ``flags`` holds MOE_FULL_WEIGHTS."""
        shape, cref, ap = x.shape, self._cref, None
        T = shape[0] if shape else -1
        # the common call, without a look at each tensor's strides
        if not (flags == 0 and out is None and stream is None and x.dtype is torch.bfloat16 and x.get_device() == self._index
                and x.is_contiguous() and shape == (T, self.K)):
            return self._general(x, out, add, flags, stream)
        if add is not None:
            if not (add.dtype is torch.bfloat16 and add.get_device() == self._index and add.is_contiguous()
                    and add.shape == (T, self.N)):
                return self._general(x, out, add, flags, stream)
            ap = add.data_ptr()
        if torch._C._cuda_getDevice() != self._index:
            return self._general(x, out, add, flags, stream)
        out = x.new_empty(T, self.N)
        if T == 0:
            return out
        st = lib.moe_linear_forward(x.data_ptr(), self._w, self._s, ap, out.data_ptr(), T, cref,
                                    torch._C._cuda_getCurrentRawStream(self._index))
        if st != MOE_OK:
            raise MoeError(st, "moe_linear_forward")
        return out

    def _general(self, x, out, add, flags, stream):
        if x.dim() != 2:
            raise ValueError(f"x: expected [T, {self.K}], got shape {tuple(x.shape)}")
        T, device = x.shape[0], self.device
        odt = torch.float32 if flags & MOE_OUT_F32 else torch.bfloat16
        ldx, ldo, lda, ap = _rows_of("x", x, torch.bfloat16, (T, self.K), device), 0, 0, None
        if out is None:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                out = x.new_empty((T, self.N), dtype=odt)
        else:
            ldo = _rows_of("out", out, odt, (T, self.N), device)
        if add is not None:
            lda = _rows_of("add", add, torch.bfloat16, (T, self.N), device)
            ap = add.data_ptr()
        if T == 0:
            return out
        c = moe_linear_cfg_t.from_buffer_copy(self.cfg)
        c.ldx, c.ldo, c.lda, c.flags = ldx, ldo, lda, flags
        with torch.cuda.device(device):
            st = lib.moe_linear_forward(x.data_ptr(), self._w, self._s, ap, out.data_ptr(), T, ctypes.byref(c),
                                        _raw_stream(device, stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_linear_forward")
        return out


def linear_forward(x: torch.Tensor, w: torch.Tensor, scales: torch.Tensor, group: int = 128,
                   out: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None, flags: int = 0,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One call of ``Int4Linear(w, scales, group)``."""
    return Int4Linear(w, scales, group)(x, out=out, add=add, flags=flags, stream=stream)


def linear_kernel_launches(N: int, K: int, T: int, group: int = 128, scale_type: int = MOE_SCALE_F32) -> int:
    """Kernels one linear call launches for T tokens (0: T = 0, or an unsupported shape)."""
    c = moe_linear_cfg_t(struct_size=ctypes.sizeof(moe_linear_cfg_t), N=N, K=K, group=group, scale_type=scale_type)
    return int(lib.moe_linear_kernel_launches(ctypes.byref(c), int(T)))


def make_few_cfg(shape, group: int, scale_type: int = MOE_SCALE_F32, flags: int = 0, topp: float = 0.0) -> moe_few_cfg_t:
    return moe_few_cfg_t(struct_size=ctypes.sizeof(moe_few_cfg_t), H=shape.H, E=shape.E, K=shape.K, I=shape.I,
                         Is=shape.Is, routed_scaling=float(shape.routed_scaling), topp=float(topp), group=int(group),
                         scale_type=int(scale_type), flags=int(flags))


def few_workspace_bytes(shape, T: int, group: int = 0) -> int:
    """Workspace of a few-token layer call for up to T tokens (0: an unsupported shape)."""
    return int(lib.moe_few_workspace_bytes(ctypes.byref(make_few_cfg(shape, group)), int(T)))


def few_pass_tokens(shape, group: int = 0) -> int:
    """Tokens that one pass of the few-token layer's kernels serves (0: an unsupported shape)."""
    return int(lib.moe_few_pass_tokens(ctypes.byref(make_few_cfg(shape, group))))


def few_kernel_launches(shape, T: int, group: int = 0) -> int:
    """Kernels one few-token layer call launches for T tokens (0: T = 0, or an unsupported shape)."""
    return int(lib.moe_few_kernel_launches(ctypes.byref(make_few_cfg(shape, group)), int(T)))


class MoEFewLayer:
    """A whole MoE layer for a few tokens (``moe_few_forward``) with group-scaled int4 weights.

    ``layer``: router_w, router_bias, w13, s13, w2, s2 and, when shape.Is > 0, sh_w13, sh_s13, sh_w2, sh_s2, as in
    ``layer_forward`` but with scales [..., rows, ceil(cols/group)] of one type (float32, bfloat16 or float16);
    ``group`` = 0 takes ``layer_forward``'s own scales [..., rows].  Holds a workspace for calls of up to
    ``max_tokens`` tokens: its calls are ordered on one stream; give each stream that may run at the same time (each
    captured graph among them) a ``workspace`` of its own (``new_workspace``).  What ``Int4Linear`` says of its
    weights holds for the layer's too."""

    def __init__(self, layer: dict, shape, group: int = 0, max_tokens: int = 8, topp: float = 0.0):
        H, E, I, Is = shape.H, shape.E, shape.I, shape.Is
        self.layer, self.shape, self.group, self.max_tokens = layer, shape, int(group), int(max_tokens)
        self.device = layer["w13"].device
        sdt = layer["s13"].dtype
        mats = [("w13", (E, 2 * I), H), ("w2", (E, H), I)]
        if Is > 0:
            mats += [("sh_w13", (2 * Is,), H), ("sh_w2", (H,), Is)]
        self.cfg = make_few_cfg(shape, self.group, _scale_type("s13", layer["s13"]), topp=topp)
        n = int(lib.moe_few_workspace_bytes(ctypes.byref(self.cfg), self.max_tokens))
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, "moe_few_workspace_bytes")
        _check_dev("router_w", layer["router_w"], torch.float32, (E, H))
        _check_dev("router_bias", layer["router_bias"], torch.float32, (E,))
        keys = ["router_w", "router_bias"]
        for name, rows, cols in mats:
            sname = name.replace("w", "s")
            _check_dev(name, layer[name], torch.uint8, (*rows, cols // 2))
            _check_dev(sname, layer[sname], sdt, _scale_shape(rows, cols, self.group))
            keys += [name, sname]
        if any(layer[k].device != self.device for k in keys):
            raise ValueError(f"the layer's tensors are not all on {self.device}")
        self._tensors = [layer[k] for k in keys]  # their addresses are kept
        self.weights = moe_few_weights_t(**{k: layer[k].data_ptr() for k in keys})
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.cfg.workspace, self.cfg.workspace_bytes = self.workspace.data_ptr(), n
        self._add = moe_few_cfg_t.from_buffer_copy(self.cfg)
        self._add.flags = MOE_ADD_RESIDUAL
        self._crefs, self._wref, self._index = ((ctypes.byref(self.cfg), ctypes.byref(self._add)),
                                                ctypes.byref(self.weights), self.device.index)

    def new_workspace(self) -> torch.Tensor:
        return torch.empty_like(self.workspace)

    def _check(self, name, t, dtype, shape):
        if t.device != self.device or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")

    def __call__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, residual: bool = False, flags: int = 0,
                 topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """The layer's output for x (bfloat16 [T, H]); bfloat16 [T, H], float32 under MOE_OUT_F32."""
        if x.dim() != 2:
            raise ValueError(f"x: expected [T, {self.shape.H}], got shape {tuple(x.shape)}")
        T = x.shape[0]
        # the common call, without a configuration of its own
        if (flags == 0 and out is None and topk_idx is None and topk_w is None and workspace is None and stream is None
                and x.dtype is torch.bfloat16 and x.get_device() == self._index and x.is_contiguous()
                and x.shape == (T, self.shape.H) and 0 < T <= self.max_tokens and torch._C._cuda_getDevice() == self._index):
            out = x.new_empty(T, self.shape.H)
            st = lib.moe_few_forward(x.data_ptr(), self._wref, out.data_ptr(), T, self._crefs[bool(residual)],
                                     torch._C._cuda_getCurrentRawStream(self._index))
            if st != MOE_OK:
                raise MoeError(st, "moe_few_forward")
            return out
        shape = self.shape
        if T > self.max_tokens:
            raise ValueError(f"T={T} exceeds max_tokens={self.max_tokens}")
        f = flags | (MOE_ADD_RESIDUAL if residual else 0)
        odt = torch.float32 if f & MOE_OUT_F32 else torch.bfloat16
        self._check("x", x, torch.bfloat16, (T, shape.H))
        if out is None:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                out = x.new_empty((T, shape.H), dtype=odt)
        self._check("out", out, odt, (T, shape.H))
        if topk_idx is not None:
            self._check("topk_idx", topk_idx, torch.int32, (T, shape.K))
        if topk_w is not None:
            self._check("topk_w", topk_w, torch.float32, (T, shape.K))
        ws = self.workspace if workspace is None else workspace
        if workspace is not None:
            self._check("workspace", ws, torch.uint8, ws.shape)
        if T == 0:
            return out
        c = moe_few_cfg_t.from_buffer_copy(self.cfg)
        c.flags = f
        c.workspace, c.workspace_bytes = ws.data_ptr(), ws.numel()
        c.topk_idx_out = None if topk_idx is None else topk_idx.data_ptr()
        c.topk_w_out = None if topk_w is None else topk_w.data_ptr()
        with torch.cuda.device(self.device):
            st = lib.moe_few_forward(x.data_ptr(), self._wref, out.data_ptr(), T, ctypes.byref(c),
                                     _raw_stream(self.device, stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_few_forward")
        return out


def few_forward(x: torch.Tensor, layer: dict, shape, group: int = 0, out: Optional[torch.Tensor] = None,
                flags: int = 0, topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None, topp: float = 0.0) -> torch.Tensor:
    """One call of ``MoEFewLayer``, with a workspace of its own."""
    with torch.cuda.stream(stream):  # the workspace belongs to the stream that uses it
        m = MoEFewLayer(layer, shape, group, max_tokens=max(1, x.shape[0]), topp=topp)
    return m(x, out=out, flags=flags, topk_idx=topk_idx, topk_w=topk_w, stream=stream)

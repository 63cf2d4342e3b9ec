"""Thin ctypes binding of libmoe (include/moe.h).

Argument marshalling only: every step of the forward runs in the CUDA
kernels of ``libmoe.so``.  torch is used for device memory and streams.
There is no fallback: if the library is missing, every call raises.

The functions keep the C names without the ``moe_`` prefix:

* :func:`ffn_forward`   - moe_ffn_forward (router, permutation, grouped GEMMs,
  combine), on caller-provided torch tensors;
* :func:`route`         - moe_route (router only);
* :func:`add_rmsnorm`, :func:`quantize_fp8`, :func:`select_experts`,
  :func:`route_groups`, :func:`gemm_fp8`, :func:`experts_forward_fp8`,
  :func:`experts_workspace_size_fp8` - the layer in 8 bits;
* :func:`workspace_size`, :func:`device_status`, :func:`profile_enable`,
  :func:`profile_read`, :func:`status_string`, :func:`abi_version`.

:class:`MoEBlock` mirrors the interface of mojolearn.MoEBlock (forward,
load_state_dict, router_logits_, selected_experts_, routing_weights_) on
top of these calls; :class:`MoEBlockFP8` is the block in 8 bits.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_ACT = 2
MOE_ERR_DTYPE = 3
MOE_ERR_SHAPE = 4
MOE_ERR_ALIGNMENT = 5
MOE_ERR_WORKSPACE = 6
MOE_ERR_CUDA = 7
MOE_ERR_TIMEOUT = 8
MOE_ERR_DEVICE = 9

ACT_SILU_GATED = 0
ACT_RELU = 1
ACT_NAMES = {"silu_gated": ACT_SILU_GATED, "silu": ACT_SILU_GATED, "relu": ACT_RELU}

F32 = 0
BF16 = 1
F64 = 2
NUM_STAGES = 6

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
GROUP_MAX = 0
GROUP_TOP2 = 1
GROUP_NAMES = {"max": GROUP_MAX, "top2": GROUP_TOP2}
QUANT_BLOCK = 128
SCORE_NAMES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}

_lock = threading.Lock()
_lib = None


class RouteOpts(ctypes.Structure):
    """moe_route_opts_t (include/moe.h)."""
    _fields_ = [("score", ctypes.c_int), ("selection_bias", ctypes.c_void_p),
                ("dynamic_threshold", ctypes.c_float), ("capacity_factor", ctypes.c_float),
                ("seq_len", ctypes.c_int64), ("slot_kept", ctypes.c_void_p),
                ("balance", ctypes.c_void_p)]


class GroupOpts(ctypes.Structure):
    """moe_group_opts_t (include/moe.h)."""
    _fields_ = [("score", ctypes.c_int), ("selection_bias", ctypes.c_void_p),
                ("groups", ctypes.c_int), ("top_groups", ctypes.c_int),
                ("group_score", ctypes.c_int), ("scale", ctypes.c_float)]


class MoEError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"libmoe status {status} ({status_string(status)}): {detail}")


def lib() -> ctypes.CDLL:
    """Loads libmoe.so (once).  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing; build it with `python -m mixture_experts_ffn_09_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.moe_ffn_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32, i32]
        L.moe_ffn_workspace_size.restype = sz
        L.moe_ffn_forward.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i64, i64, i64,
                                      i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_ffn_forward.restype = i32
        L.moe_ffn_forward_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i64,
                                              i64, i64, i32, vp, vp, vp, vp, vp]
        L.moe_ffn_forward_noalloc.restype = i32
        L.moe_ffn_forward_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i64, i64,
                                         i64, i32, vp, vp, vp, vp, vp, sz,
                                         ctypes.POINTER(RouteOpts), vp]
        L.moe_ffn_forward_ex.restype = i32
        L.moe_route_ex.argtypes = [vp, vp, vp, i64, i64, i32, i32, i32, i32, vp, vp, vp,
                                   ctypes.POINTER(RouteOpts), vp]
        L.moe_route_ex.restype = i32
        L.moe_route.argtypes = [vp, vp, vp, i64, i64, i32, i32, i32, i32, vp, vp, vp, vp]
        L.moe_route.restype = i32
        f32 = ctypes.c_float
        L.moe_add_rmsnorm.argtypes = [vp, vp, vp, f32, i64, i64, i32, vp, vp, vp, vp, vp]
        L.moe_add_rmsnorm.restype = i32
        L.moe_quantize_fp8.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, vp]
        L.moe_quantize_fp8.restype = i32
        L.moe_select_experts.argtypes = [vp, i64, i32, i32, i32, ctypes.POINTER(GroupOpts), vp, vp, vp]
        L.moe_select_experts.restype = i32
        L.moe_route_groups.argtypes = [vp, vp, vp, i64, i64, i32, i32, i32, i32,
                                       ctypes.POINTER(GroupOpts), vp, vp, vp, vp]
        L.moe_route_groups.restype = i32
        L.moe_gemm_fp8.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, i32, vp]
        L.moe_gemm_fp8.restype = i32
        L.moe_experts_workspace_size_fp8.argtypes = [i64, i64, i64, i32, i32]
        L.moe_experts_workspace_size_fp8.restype = sz
        L.moe_experts_forward_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32,
                                              i32, vp, sz, vp]
        L.moe_experts_forward_fp8.restype = i32
        L.moe_status_string.argtypes = [i32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = i32
        L.moe_device_status.argtypes = [vp]
        L.moe_device_status.restype = i32
        L.moe_device_error_peek.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.moe_device_error_peek.restype = i32
        L.moe_kernel_launches.argtypes = []
        L.moe_kernel_launches.restype = ctypes.c_ulonglong
        L.moe_error_sites.argtypes = [ctypes.c_uint]
        L.moe_error_sites.restype = ctypes.c_char_p
        L.moe_profile_enable.argtypes = [i32]
        L.moe_profile_enable.restype = i32
        L.moe_profile_read.argtypes = [ctypes.POINTER(ctypes.c_float), i32]
        L.moe_profile_read.restype = i32
        L.moe_debug_bounded_wait.argtypes = [i32, vp]
        L.moe_debug_bounded_wait.restype = i32
        L.moe_set_pdl.argtypes = [i32]
        L.moe_set_pdl.restype = i32
        L.moe_set_debug_sync.argtypes = [i32]
        L.moe_set_debug_sync.restype = i32
        L.moe_set_fused_gather.argtypes = [i32]
        L.moe_set_fused_gather.restype = i32
        L.moe_set_gemm_mode.argtypes = [i32]
        L.moe_set_gemm_mode.restype = i32
        L.moe_set_small_cluster.argtypes = [i32]
        L.moe_set_small_cluster.restype = i32
        L.moe_stage_name.argtypes = [i32]
        L.moe_stage_name.restype = ctypes.c_char_p
        _lib = L
        return L


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def last_error() -> str:
    return lib().moe_last_error().decode()


def abi_version() -> int:
    return int(lib().moe_abi_version())


def _check(status: int) -> None:
    if status != MOE_OK:
        raise MoEError(status, last_error())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype is torch.float32:
        return F32
    if t.dtype is torch.bfloat16:
        return BF16
    if t.dtype is torch.float64:
        return F64
    return -1


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _act_code(act) -> int:
    if isinstance(act, str):
        if act not in ACT_NAMES:
            return 99
        return ACT_NAMES[act]
    return int(act)


def workspace_size(T: int, D: int, F: int, E: int, K: int, dtype: int, act=ACT_SILU_GATED) -> int:
    return int(lib().moe_ffn_workspace_size(T, D, F, E, K, dtype, _act_code(act)))


def _expect(t, shape, name, dtype=None, required=True):
    """Shape / dtype / device / contiguity checks of one tensor argument."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if isinstance(t, int):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def ffn_forward(x, router, gate_up_proj, down_proj, E: int, K: int, norm_topk_prob: bool, act,
                out, selected_experts=None, routing_weights=None, router_bias=None, b1=None,
                b2=None, router_logits=None, workspace=None, stream=None) -> None:
    """moe_ffn_forward on torch tensors.  x (..., D); out like x."""
    import torch
    D = int(x.shape[-1])
    T = int(x.numel() // D) if D else 0
    F = int(down_proj.shape[-1])
    dt = _dtype_code(x)
    a = _act_code(act)
    if dt in (F32, BF16) and a in (ACT_SILU_GATED, ACT_RELU) and 1 <= K <= E and T > 0:
        wdt = x.dtype
        gu_rows = 2 * F if a == ACT_SILU_GATED else F
        _expect(x, tuple(x.shape), "x", wdt)
        _expect(router, (E, D), "router", wdt)
        _expect(gate_up_proj, (E, gu_rows, D), "gate_up_proj", wdt)
        _expect(down_proj, (E, D, F), "down_proj", wdt)
        _expect(out, tuple(x.shape), "out", wdt)
        _expect(selected_experts, (T, K), "selected_experts", torch.int64, False)
        _expect(routing_weights, (T, K), "routing_weights", torch.float32, False)
        _expect(router_bias, (E,), "router_bias", torch.float32, False)
        _expect(b1, (E, F), "b1", torch.float32, False)
        _expect(b2, (E, D), "b2", torch.float32, False)
        _expect(router_logits, (T, E), "router_logits", torch.float32, False)
    ws_bytes = 0
    if workspace is not None and not isinstance(workspace, int):
        ws_bytes = workspace.numel() * workspace.element_size()
    elif isinstance(workspace, int):
        raise ValueError("pass the workspace as a tensor")
    st = lib().moe_ffn_forward(
        _ptr(x), _ptr(router), _ptr(gate_up_proj), _ptr(down_proj), E, K, int(bool(norm_topk_prob)),
        a, _ptr(out), _ptr(selected_experts), _ptr(routing_weights), T, D, F, dt,
        _ptr(router_bias), _ptr(b1), _ptr(b2), _ptr(router_logits), _ptr(workspace), ws_bytes,
        _stream(stream))
    _check(st)


def ffn_forward_noalloc(x, router, gate_up_proj, down_proj, E: int, K: int, norm_topk_prob: bool,
                        act, out, selected_experts=None, routing_weights=None, router_bias=None,
                        b1=None, b2=None, router_logits=None, stream=None) -> None:
    """moe_ffn_forward_noalloc: the same forward without a workspace, for
    callers that cannot allocate device memory when they run the layer (the
    library's static scratch of noalloc_scratch_bytes() is used instead)."""
    import torch
    D = int(x.shape[-1])
    T = int(x.numel() // D) if D else 0
    F = int(down_proj.shape[-1])
    dt = _dtype_code(x)
    a = _act_code(act)
    if dt in (F32, BF16) and a in (ACT_SILU_GATED, ACT_RELU) and 1 <= K <= E and T > 0:
        wdt = x.dtype
        gu_rows = 2 * F if a == ACT_SILU_GATED else F
        _expect(x, tuple(x.shape), "x", wdt)
        _expect(router, (E, D), "router", wdt)
        _expect(gate_up_proj, (E, gu_rows, D), "gate_up_proj", wdt)
        _expect(down_proj, (E, D, F), "down_proj", wdt)
        _expect(out, tuple(x.shape), "out", wdt)
        _expect(selected_experts, (T, K), "selected_experts", torch.int64, False)
        _expect(routing_weights, (T, K), "routing_weights", torch.float32, False)
        _expect(router_bias, (E,), "router_bias", torch.float32, False)
        _expect(b1, (E, F), "b1", torch.float32, False)
        _expect(b2, (E, D), "b2", torch.float32, False)
        _expect(router_logits, (T, E), "router_logits", torch.float32, False)
    st = lib().moe_ffn_forward_noalloc(
        _ptr(x), _ptr(router), _ptr(gate_up_proj), _ptr(down_proj), E, K, int(bool(norm_topk_prob)),
        a, _ptr(out), _ptr(selected_experts), _ptr(routing_weights), T, D, F, dt,
        _ptr(router_bias), _ptr(b1), _ptr(b2), _ptr(router_logits), _stream(stream))
    _check(st)


def noalloc_scratch_bytes() -> int:
    """Size of the static scratch behind ffn_forward_noalloc: the value of
    MOE_NOALLOC_SCRATCH_BYTES in include/moe.h (32 MiB).  A CPU test pins it
    against the library: sizes up to it pass the size check, one byte more
    of workspace is refused."""
    return 32 << 20


def _opts(score="softmax", selection_bias=None, dynamic_threshold=0.0, capacity_factor=0.0,
          seq_len=0, slot_kept=None, balance=None) -> RouteOpts:
    sc = SCORE_NAMES.get(score, score) if isinstance(score, str) else int(score)
    if isinstance(sc, str):
        sc = 99
    return RouteOpts(int(sc), _ptr(selection_bias), float(dynamic_threshold),
                     float(capacity_factor), int(seq_len), _ptr(slot_kept), _ptr(balance))


def ffn_forward_ex(x, router, gate_up_proj, down_proj, E: int, K: int, norm_topk_prob: bool, act,
                   out, selected_experts=None, routing_weights=None, router_bias=None, b1=None,
                   b2=None, router_logits=None, workspace=None, stream=None, **opts) -> None:
    """moe_ffn_forward_ex: the forward with routing options (score,
    selection_bias, dynamic_threshold, capacity_factor, seq_len, slot_kept,
    balance - see include/moe.h)."""
    import torch
    D = int(x.shape[-1])
    T = int(x.numel() // D) if D else 0
    F = int(down_proj.shape[-1])
    dt = _dtype_code(x)
    a = _act_code(act)
    if dt in (F32, BF16) and a in (ACT_SILU_GATED, ACT_RELU) and 1 <= K <= E and T > 0:
        wdt = x.dtype
        gu_rows = 2 * F if a == ACT_SILU_GATED else F
        _expect(x, tuple(x.shape), "x", wdt)
        _expect(router, (E, D), "router", wdt)
        _expect(gate_up_proj, (E, gu_rows, D), "gate_up_proj", wdt)
        _expect(down_proj, (E, D, F), "down_proj", wdt)
        _expect(out, tuple(x.shape), "out", wdt)
        _expect(selected_experts, (T, K), "selected_experts", torch.int64, False)
        _expect(routing_weights, (T, K), "routing_weights", torch.float32, False)
        _expect(router_bias, (E,), "router_bias", torch.float32, False)
        _expect(b1, (E, F), "b1", torch.float32, False)
        _expect(b2, (E, D), "b2", torch.float32, False)
        _expect(router_logits, (T, E), "router_logits", torch.float32, False)
        _expect(opts.get("selection_bias"), (E,), "selection_bias", torch.float32, False)
        _expect(opts.get("slot_kept"), (T, K), "slot_kept", torch.uint8, False)
        _expect(opts.get("balance"), (4,), "balance", torch.float32, False)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    o = _opts(**opts)
    st = lib().moe_ffn_forward_ex(
        _ptr(x), _ptr(router), _ptr(gate_up_proj), _ptr(down_proj), E, K, int(bool(norm_topk_prob)),
        a, _ptr(out), _ptr(selected_experts), _ptr(routing_weights), T, D, F, dt,
        _ptr(router_bias), _ptr(b1), _ptr(b2), _ptr(router_logits), _ptr(workspace), ws_bytes,
        ctypes.byref(o), _stream(stream))
    _check(st)


def route_ex(x, router, K: int, norm_topk_prob: bool, selected_experts, routing_weights,
             router_bias=None, router_logits=None, stream=None, **opts) -> None:
    """moe_route_ex: the router with options (not capacity or balance)."""
    import torch
    D = int(x.shape[-1])
    T = int(x.numel() // D) if D else 0
    E = int(router.shape[0])
    dt = _dtype_code(x)
    if dt in (F32, BF16) and 1 <= K <= E and T > 0:
        _expect(x, tuple(x.shape), "x", x.dtype)
        _expect(router, (E, D), "router", x.dtype)
        _expect(selected_experts, (T, K), "selected_experts", torch.int64)
        _expect(routing_weights, (T, K), "routing_weights", torch.float32)
        _expect(router_bias, (E,), "router_bias", torch.float32, False)
        _expect(router_logits, (T, E), "router_logits", torch.float32, False)
        _expect(opts.get("selection_bias"), (E,), "selection_bias", torch.float32, False)
        _expect(opts.get("slot_kept"), (T, K), "slot_kept", torch.uint8, False)
    o = _opts(**opts)
    st = lib().moe_route_ex(_ptr(x), _ptr(router), _ptr(router_bias), T, D, E, K,
                            int(bool(norm_topk_prob)), dt, _ptr(router_logits),
                            _ptr(selected_experts), _ptr(routing_weights), ctypes.byref(o),
                            _stream(stream))
    _check(st)


def route(x, router, K: int, norm_topk_prob: bool, selected_experts, routing_weights,
          router_bias=None, router_logits=None, stream=None) -> None:
    """moe_route on torch tensors."""
    import torch
    D = int(x.shape[-1])
    T = int(x.numel() // D) if D else 0
    E = int(router.shape[0])
    dt = _dtype_code(x)
    if dt in (F32, BF16) and 1 <= K <= E and T > 0:
        _expect(x, tuple(x.shape), "x", x.dtype)
        _expect(router, (E, D), "router", x.dtype)
        _expect(selected_experts, (T, K), "selected_experts", torch.int64)
        _expect(routing_weights, (T, K), "routing_weights", torch.float32)
        _expect(router_bias, (E,), "router_bias", torch.float32, False)
        _expect(router_logits, (T, E), "router_logits", torch.float32, False)
    st = lib().moe_route(_ptr(x), _ptr(router), _ptr(router_bias), T, D, E, K,
                         int(bool(norm_topk_prob)), dt, _ptr(router_logits),
                         _ptr(selected_experts), _ptr(routing_weights), _stream(stream))
    _check(st)


def _blocks(n: int) -> int:
    return -(-n // QUANT_BLOCK)


def _rows(shape) -> int:
    return math.prod(shape[:-1]) if len(shape) != 2 else shape[0]


# The 8-bit calls take microseconds on the GPU at decode sizes, so their
# binding is kept short: torch and the library are looked up once, and an
# argument that is as it should be costs one comparison of each kind.
_torch = None


def _fast():
    """(torch, library, current device), loading the first two when needed."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch, _lib or lib(), _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else -1


def _raw_stream(stream, dev: int):
    """The cudaStream_t of a stream argument (None: the current stream of device dev)."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else _stream(None)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _want(t, shape, dtype, name, dev, required=True):
    """Checks one tensor and returns its address (0 for None)."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return 0
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev >= 0:
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")


def add_rmsnorm(x, weight, eps: float, residual=None, sum_out=None, out=None, out8=None,
                scales=None, stream=None) -> None:
    """moe_add_rmsnorm on torch tensors.  x (..., D); weight (D,); residual,
    sum_out, out like x; out8 float8_e4m3fn like x; scales float32
    (rows, ceil(D / 128))."""
    torch, L, dev = _fast()
    shape, dtype = x.shape, x.dtype
    D = shape[-1]
    T = _rows(x.shape)
    dt = _dtype_code(x)
    ok = dt in (F32, BF16) and T > 0       # else the library says what is wrong
    px, pw, pr, ps, po, p8, pc = (
        _want(x, shape, dtype, "x", dev), _want(weight, (D,), dtype, "weight", dev),
        _want(residual, shape, dtype, "residual", dev, False),
        _want(sum_out, shape, dtype, "sum_out", dev, False), _want(out, shape, dtype, "out", dev, False),
        _want(out8, shape, torch.float8_e4m3fn, "out8", dev, False),
        _want(scales, (T, _blocks(D)), torch.float32, "scales", dev, False)) if ok else (None,) * 7
    _check(L.moe_add_rmsnorm(px, pr, pw, eps, T, D, dt, ps, po, p8, pc, _raw_stream(stream, dev)))


def quantize_fp8(x, out8, scales, block_rows: int = 1, stream=None) -> None:
    """moe_quantize_fp8 on torch tensors.  x (..., rows, cols), out8
    float8_e4m3fn like x, scales float32: (..., rows, ceil(cols / 128)) with
    block_rows 1, (..., ceil(rows / 128), ceil(cols / 128)) with 128.  Give a
    gate_up weight (E, 2F, D) as its view (E, 2, F, D)."""
    torch, L, dev = _fast()
    if x.dim() < 2:
        raise ValueError("x needs at least two dimensions (rows, cols)")
    rows, cols = x.shape[-2], x.shape[-1]
    dt = _dtype_code(x)
    px = p8 = pc = None
    if dt in (F32, BF16) and x.numel() > 0 and block_rows in (1, QUANT_BLOCK):
        px = _want(x, x.shape, x.dtype, "x", dev)
        p8 = _want(out8, x.shape, torch.float8_e4m3fn, "out8", dev)
        pc = _want(scales, (*x.shape[:-2], rows if block_rows == 1 else _blocks(rows), _blocks(cols)),
                   torch.float32, "scales", dev)
    mats = x.numel() // (rows * cols) if rows * cols else 0
    _check(L.moe_quantize_fp8(px, dt, mats, rows, cols, block_rows, p8, pc, _raw_stream(stream, dev)))


def _group_opts(score, selection_bias, groups, top_groups, group_score, scale, E, dev) -> GroupOpts:
    sc = SCORE_NAMES.get(score, 99) if isinstance(score, str) else int(score)
    gs = GROUP_NAMES.get(group_score, 99) if isinstance(group_score, str) else int(group_score)
    bias = _want(selection_bias, (E,), _torch.float32, "selection_bias", dev, False)
    return GroupOpts(sc, bias or None, groups, top_groups, gs, scale)


def select_experts(logits, K: int, norm_topk_prob: bool, selected_experts, routing_weights,
                   score="softmax", selection_bias=None, groups: int = 1, top_groups: int = 0,
                   group_score="max", scale: float = 1.0, stream=None) -> None:
    """moe_select_experts on torch tensors: logits (..., E) float32,
    selected_experts int64 and routing_weights float32 of K per row."""
    torch, L, dev = _fast()
    E = logits.shape[-1]
    T = _rows(logits.shape)
    pl = ps = pw = None
    if T > 0 and K >= 1:
        pl = _want(logits, logits.shape, torch.float32, "logits", dev)
        ps = _want(selected_experts, (T, K), torch.int64, "selected_experts", dev)
        pw = _want(routing_weights, (T, K), torch.float32, "routing_weights", dev)
    o = _group_opts(score, selection_bias, groups, top_groups, group_score, scale, E, dev)
    _check(L.moe_select_experts(pl, T, E, K, 1 if norm_topk_prob else 0, ctypes.byref(o), ps, pw,
                                _raw_stream(stream, dev)))


def route_groups(x, router, K: int, norm_topk_prob: bool, router_logits, selected_experts,
                 routing_weights, router_bias=None, score="softmax", selection_bias=None,
                 groups: int = 1, top_groups: int = 0, group_score="max", scale: float = 1.0,
                 stream=None) -> None:
    """moe_route_groups on torch tensors: the router's product, then
    :func:`select_experts`; router_logits (T, E) float32 is written."""
    torch, L, dev = _fast()
    D = x.shape[-1]
    T = _rows(x.shape)
    E = router.shape[0]
    dt = _dtype_code(x)
    px = pr = pb = pl = ps = pw = None
    if dt in (F32, BF16) and T > 0 and K >= 1:
        px = _want(x, x.shape, x.dtype, "x", dev)
        pr = _want(router, (E, D), x.dtype, "router", dev)
        pb = _want(router_bias, (E,), torch.float32, "router_bias", dev, False) or None
        pl = _want(router_logits, (T, E), torch.float32, "router_logits", dev)
        ps = _want(selected_experts, (T, K), torch.int64, "selected_experts", dev)
        pw = _want(routing_weights, (T, K), torch.float32, "routing_weights", dev)
    o = _group_opts(score, selection_bias, groups, top_groups, group_score, scale, E, dev)
    _check(L.moe_route_groups(px, pr, pb, T, D, E, K, 1 if norm_topk_prob else 0, dt, ctypes.byref(o),
                              pl, ps, pw, _raw_stream(stream, dev)))


def gemm_fp8(a, a_scales, w, w_scales, out, offsets=None, stream=None) -> None:
    """moe_gemm_fp8 on torch tensors: a (M, K), w (E, N, K) or (N, K)
    float8_e4m3fn; scales float32; offsets (E + 1,) int32; out (M, N)
    bfloat16 or float32."""
    torch, L, dev = _fast()
    if a.dim() != 2 or w.dim() not in (2, 3):
        raise ValueError("a must be (M, K), w (E, N, K) or (N, K)")
    M, K = a.shape
    ws = w.shape
    N = ws[-2]
    E = ws[0] if len(ws) == 3 else 1
    dt = _dtype_code(out)
    pa = pc = pw = pv = pf = po = None
    if dt in (F32, BF16) and M > 0 and N > 0 and K > 0 and E > 0:
        f8, f32 = torch.float8_e4m3fn, torch.float32
        kb = _blocks(K)
        pa = _want(a, (M, K), f8, "a", dev)
        pc = _want(a_scales, (M, kb), f32, "a_scales", dev)
        pw = _want(w, (*ws[:-1], K), f8, "w", dev)
        pv = _want(w_scales, (*ws[:-2], _blocks(N), kb), f32, "w_scales", dev)
        pf = _want(offsets, (E + 1,), torch.int32, "offsets", dev, False) or None
        po = _want(out, (M, N), out.dtype, "out", dev)
    _check(L.moe_gemm_fp8(pa, pc, pw, pv, pf, E, M, N, K, po, dt, _raw_stream(stream, dev)))


def experts_workspace_size_fp8(T: int, D: int, F: int, E: int, K: int) -> int:
    return int(lib().moe_experts_workspace_size_fp8(T, D, F, E, K))


def experts_forward_fp8(x, x_scales, selected_experts, routing_weights, gate_up_proj, gate_up_scales,
                        down_proj, down_scales, out, workspace=None, stream=None) -> None:
    """moe_experts_forward_fp8 on torch tensors: x (..., D), gate_up_proj
    (E, 2F, D) and down_proj (E, D, F) float8_e4m3fn; x_scales
    (T, ceil(D / 128)), gate_up_scales (E, 2, ceil(F / 128), ceil(D / 128)),
    down_scales (E, ceil(D / 128), ceil(F / 128)) float32; selected_experts
    (T, K) int64, routing_weights (T, K) float32; out bfloat16 like x."""
    torch, L, dev = _fast()
    D = x.shape[-1]
    T = _rows(x.shape)
    E, F = down_proj.shape[0], down_proj.shape[-1]
    K = selected_experts.shape[-1]
    ptrs, ws_bytes, pws = (None,) * 9, 0, None
    if T > 0 and E > 0 and F > 0 and K > 0:
        f8, f32 = torch.float8_e4m3fn, torch.float32
        db, fb = _blocks(D), _blocks(F)
        ptrs = (_want(x, x.shape, f8, "x", dev), _want(x_scales, (T, db), f32, "x_scales", dev),
                _want(selected_experts, (T, K), torch.int64, "selected_experts", dev),
                _want(routing_weights, (T, K), f32, "routing_weights", dev),
                _want(gate_up_proj, (E, 2 * F, D), f8, "gate_up_proj", dev),
                _want(gate_up_scales, (E, 2, fb, db), f32, "gate_up_scales", dev),
                _want(down_proj, (E, D, F), f8, "down_proj", dev),
                _want(down_scales, (E, db, fb), f32, "down_scales", dev),
                _want(out, x.shape, torch.bfloat16, "out", dev))
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        pws = _want(workspace, workspace.shape, workspace.dtype, "workspace", dev)
    _check(L.moe_experts_forward_fp8(*ptrs, T, D, F, E, K, pws, ws_bytes, _raw_stream(stream, dev)))


GEMM_AUTO, GEMM_1SM, GEMM_2SM = 0, 1, 2


def set_gemm_mode(mode: int) -> int:
    """Selects the bf16 grouped GEMM (GEMM_AUTO, GEMM_1SM, GEMM_2SM);
    returns the previous mode."""
    prev = int(lib().moe_set_gemm_mode(int(mode)))
    if prev < 0:
        raise ValueError(f"unknown GEMM mode {mode}")
    return prev


def set_tail_swap(max_rows: int) -> int:
    """An expert's last CTA-pair tile of at most max_rows rows (0..128)
    runs with swapped operands; 0 turns it off.  Returns the previous value."""
    prev = int(lib().moe_set_tail_swap(int(max_rows)))
    if prev < 0:
        raise ValueError(f"tail swap rows out of range: {max_rows}")
    return prev


SMALL_CLUSTER_AUTO = 0


def set_small_cluster(ctas: int) -> int:
    """Cluster size of the one-kernel float32 small layer: SMALL_CLUSTER_AUTO
    (16 where possible, else 8), 8 or 16.  Returns the previous value."""
    prev = int(lib().moe_set_small_cluster(int(ctas)))
    if prev < 0:
        raise ValueError(f"small-layer cluster size must be 0, 8 or 16, not {ctas}")
    return prev


def set_pdl(on: bool) -> bool:
    """Programmatic dependent launch between a forward's kernels (default
    off; see moe_set_pdl in include/moe.h); returns the previous setting."""
    return bool(lib().moe_set_pdl(int(bool(on))))


FUSED_GATHER_OFF, FUSED_GATHER_ON, FUSED_GATHER_AUTO = 0, 1, 2


def set_fused_gather(mode) -> int:
    """Selects whether the bf16 gate_up GEMM gathers its rows from x itself
    (TMA gather4) or reads an expert-sorted copy: False/"off", True/"on" or
    "auto" (the default; see moe_set_fused_gather in include/moe.h), or the
    FUSED_GATHER_* value.  Returns the previous value (an int)."""
    if isinstance(mode, str):
        mode = {"off": FUSED_GATHER_OFF, "on": FUSED_GATHER_ON, "auto": FUSED_GATHER_AUTO}[mode]
    elif isinstance(mode, bool):
        mode = FUSED_GATHER_ON if mode else FUSED_GATHER_OFF
    prev = int(lib().moe_set_fused_gather(int(mode)))
    if prev < 0:
        raise ValueError(f"fused gather mode must be 0, 1 or 2, not {mode}")
    return prev


def device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status."""
    return int(lib().moe_device_status(_stream(stream)))


def set_debug_sync(timeout_ms: int) -> int:
    """With timeout_ms > 0 every forward waits, bounded, after each kernel
    and fails naming the first kernel that did not finish; returns the
    previous setting."""
    return int(lib().moe_set_debug_sync(int(timeout_ms)))


def device_error_peek() -> int:
    """The device error word, read without waiting for any stream and
    without clearing it (for watchdogs)."""
    w = ctypes.c_uint(0)
    _check(lib().moe_device_error_peek(ctypes.byref(w)))
    return int(w.value)


def kernel_launches() -> int:
    """Kernels this library has launched in the process so far."""
    return int(lib().moe_kernel_launches())


def error_sites(word: int) -> str:
    """Names of the kernel roles whose bounded waits set bits in ``word``."""
    return lib().moe_error_sites(ctypes.c_uint(word)).decode()


def debug_bounded_wait(timeout_ms: int, stream=None) -> None:
    """Launches the failure-detection probe (a bounded wait that must time
    out); read the outcome with device_status()."""
    _check(lib().moe_debug_bounded_wait(int(timeout_ms), _stream(stream)))


def profile_enable(on: bool = True) -> None:
    _check(lib().moe_profile_enable(int(bool(on))))


def profile_read() -> tuple[dict, int]:
    """Per-stage milliseconds summed since enable/last read, and the number
    of forward calls they cover."""
    buf = (ctypes.c_float * NUM_STAGES)()
    calls = int(lib().moe_profile_read(buf, NUM_STAGES))
    names = [lib().moe_stage_name(i).decode() for i in range(NUM_STAGES)]
    return {n: float(buf[i]) for i, n in enumerate(names)}, calls


class MoEBlock:
    """Sparse MoE feed-forward block with mojolearn.MoEBlock's interface.

    Weights are device tensors in the Hugging Face layout: router (E, D),
    gate_up_proj (E, 2F, D), down_proj (E, D, F) (or W1 (E, F, D), W2
    (E, D, F) plus biases for the ReLU expert).  ``forward`` runs
    moe_ffn_forward and keeps ``router_logits_``, ``selected_experts_``
    (int64) and ``routing_weights_`` of the last call."""

    def __init__(self, router, gate_up_proj, down_proj, top_k: int = 2,
                 norm_topk_prob: bool = True, hidden_act: str = "silu", router_bias=None,
                 b1=None, b2=None):
        if hidden_act not in ACT_NAMES:
            raise NotImplementedError(f"hidden_act {hidden_act!r}")
        E = int(router.shape[0])
        if not (1 <= int(top_k) <= E):
            raise ValueError(f"top_k={top_k} outside [1, {E}]")
        self.router, self.gate_up_proj, self.down_proj = router, gate_up_proj, down_proj
        self.router_bias, self.b1, self.b2 = router_bias, b1, b2
        self.top_k = int(top_k)
        self.norm_topk_prob = bool(norm_topk_prob)
        self.act = ACT_NAMES[hidden_act]
        self._ws = None
        self.router_logits_ = self.selected_experts_ = self.routing_weights_ = None

    @property
    def num_experts(self) -> int:
        return int(self.router.shape[0])

    def load_state_dict(self, sd: dict) -> "MoEBlock":
        for k in ("router", "gate_up_proj", "down_proj"):
            cur = getattr(self, k)
            if tuple(sd[k].shape) != tuple(cur.shape):
                raise ValueError(f"{k}: shape {tuple(sd[k].shape)} != {tuple(cur.shape)}")
        for k in ("router", "gate_up_proj", "down_proj"):
            getattr(self, k).copy_(sd[k])
        return self

    def forward(self, x, stream=None):
        import torch
        if x.dtype == torch.float64:
            raise TypeError("float64 input is not supported")
        D = int(x.shape[-1])
        T = x.numel() // D
        E, K = self.num_experts, self.top_k
        F = int(self.down_proj.shape[-1])
        need = workspace_size(T, D, F, E, K, _dtype_code(x), self.act)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
        out = torch.empty_like(x)
        self.router_logits_ = torch.empty(T, E, dtype=torch.float32, device=x.device)
        self.selected_experts_ = torch.empty(T, K, dtype=torch.int64, device=x.device)
        self.routing_weights_ = torch.empty(T, K, dtype=torch.float32, device=x.device)
        ffn_forward(x, self.router, self.gate_up_proj, self.down_proj, E, K, self.norm_topk_prob,
                    self.act, out, self.selected_experts_, self.routing_weights_,
                    self.router_bias, self.b1, self.b2, self.router_logits_, self._ws, stream)
        return out

    __call__ = forward


class MoEBlockFP8:
    """The SiLU-gated block with 8-bit experts: optional residual RMS norm,
    routing with groups, experts in the block format (include/moe.h).

    Made from bf16 or float32 weights in the Hugging Face layout, which it
    quantises once: router (E, D) stays in its type, gate_up_proj (E, 2F, D)
    and down_proj (E, D, F) become e4m3 with block scales.  With norm_weight
    (D,) the input is normed first; ``forward(x, residual)`` then returns the
    block's output, and ``residual_`` holds x + residual.  The output is bf16,
    whatever the type of x (bf16 or float32, the router's).  Routing options are
    those of :func:`select_experts`.  Keeps ``router_logits_``,
    ``selected_experts_`` and ``routing_weights_`` of the last call.

    Calls may overlap on several streams and in several threads: every call
    takes its buffers, the workspace too, from the allocator's pool of its
    stream (of the graph, while one is captured), and none is kept for the next
    call.  The attributes are set as a call returns, so with several threads
    they are those of any of them."""

    def __init__(self, router, gate_up_proj, down_proj, top_k: int = 2, norm_topk_prob: bool = True,
                 norm_weight=None, eps: float = 1e-6, router_bias=None, **routing):
        import torch
        E, F2, D = (int(n) for n in gate_up_proj.shape)
        F = F2 // 2
        if not 1 <= int(top_k) <= E:
            raise ValueError(f"top_k={top_k} outside [1, {E}]")
        if tuple(down_proj.shape) != (E, D, F) or F2 != 2 * F:
            raise ValueError(f"down_proj has shape {tuple(down_proj.shape)}, expected {(E, D, F2 / 2)}")
        self.router, self.router_bias = router, router_bias
        self.norm_weight, self.eps = norm_weight, float(eps)
        self.top_k, self.norm_topk_prob, self.routing = int(top_k), bool(norm_topk_prob), routing
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=gate_up_proj.device)  # noqa: E731
        f8, f32 = torch.float8_e4m3fn, torch.float32
        self.gate_up_proj, self.down_proj = new((E, 2 * F, D), f8), new((E, D, F), f8)
        self.gate_up_scales = new((E, 2, _blocks(F), _blocks(D)), f32)
        self.down_scales = new((E, _blocks(D), _blocks(F)), f32)
        quantize_fp8(gate_up_proj.view(E, 2, F, D), self.gate_up_proj.view(E, 2, F, D),
                     self.gate_up_scales, QUANT_BLOCK)
        quantize_fp8(down_proj, self.down_proj, self.down_scales, QUANT_BLOCK)
        # calls may come on any stream: the weights are in place on return
        if gate_up_proj.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
        self.residual_ = self.router_logits_ = self.selected_experts_ = self.routing_weights_ = None

    @property
    def num_experts(self) -> int:
        return int(self.router.shape[0])

    def forward(self, x, residual=None, stream=None):
        import torch
        if residual is not None and self.norm_weight is None:
            raise ValueError("a residual needs norm_weight")
        if stream is not None:                 # buffers of that stream's pool
            with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
                return self.forward(x, residual)
        E, F, D = int(self.down_proj.shape[0]), int(self.down_proj.shape[-1]), int(x.shape[-1])
        T, K = _rows(x.shape), self.top_k
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=x.device)  # noqa: E731
        x8, xs = new(x.shape, torch.float8_e4m3fn), new((T, _blocks(D)), torch.float32)
        total = x if self.norm_weight is not None else None
        if self.norm_weight is not None:
            if residual is not None:
                total = torch.empty_like(x)
            y = torch.empty_like(x)
            add_rmsnorm(x, self.norm_weight, self.eps, residual, total if residual is not None else None, y, x8, xs)
            x = y
        else:
            quantize_fp8(x.view(T, D), x8.view(T, D), xs, 1)
        logits, selected = new((T, E), torch.float32), new((T, K), torch.int64)
        weights = new((T, K), torch.float32)
        route_groups(x, self.router, K, self.norm_topk_prob, logits, selected, weights, self.router_bias,
                     **self.routing)
        ws = new(max(experts_workspace_size_fp8(T, D, F, E, K), 1), torch.uint8)
        out = new(x.shape, torch.bfloat16)
        experts_forward_fp8(x8, xs, selected, weights, self.gate_up_proj, self.gate_up_scales, self.down_proj,
                            self.down_scales, out, ws)
        # only now: another thread may be inside a call of its own
        self.residual_, self.router_logits_ = total, logits
        self.selected_experts_, self.routing_weights_ = selected, weights
        return out

    __call__ = forward

"""ctypes binding of libq4lin.so (argument marshalling only).

Every step of the layer runs in the library's CUDA kernels; this module only
turns torch tensors into pointers and sizes and raises on a nonzero status.
If the library has not been built it raises: there is no other path.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libq4lin.so")

OK = 0
STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED_SHAPE", 3: "MISALIGNED", 4: "WORKSPACE",
          5: "DEVICE", 6: "CUDA", 7: "TIMEOUT"}
ROUTE_AUTO, ROUTE_GEMV, ROUTE_TC_SPLITK, ROUTE_TC, ROUTE_TC_FP16, ROUTE_STREAM_MMA = 0, 1, 2, 3, 4, 5
ROUTE_NAMES = {ROUTE_AUTO: "auto", ROUTE_GEMV: "gemv", ROUTE_TC_SPLITK: "tc_splitk", ROUTE_TC: "tc",
               ROUTE_TC_FP16: "tc_fp16", ROUTE_STREAM_MMA: "stream_mma"}

QTYPES = {"q4g64": 0, "q5g64": 1, "q6g64": 2, "w8g32": 3}

EXPORTS = ("q4lin_workspace_bytes", "q4lin_linear", "q4lin_linear_route", "q4lin_linear_qtype",
           "q4lin_linear_fp16_static", "q4lin_qtype_kernel_launches", "q4lin_linear_add",
           "q4lin_route_workspace_bytes", "q4lin_select_route", "q4lin_tile_plan", "q4lin_kernel_launches",
           "q4lin_status_string",
           "q4lin_device_status", "q4lin_clear_device_status", "q4lin_last_error_detail",
           "q4lin_hbm_read_probe", "q4lin_diag_wait_expiry", "q4lin_linear_swiglu", "q4lin_linear_pair",
           "q4lin_qtype_workspace_bytes", "q4lin_host_workspace_bytes", "q4lin_linear_host", "q4lin_fused_route", "q4lin_qtype_route", "q4lin_version",
           "q4lin_lora_workspace_bytes", "q4lin_lora_route", "q4lin_linear_lora", "q4lin_moe_router",
           "q4lin_moe_workspace_bytes", "q4lin_moe_experts", "q4lin_moe", "q4lin_qk_norm_rope",
           "q4lin_prompt_attention", "q4lin_kv4_page_bytes", "q4lin_kv4_append", "q4lin_kv4_read",
           "q4lin_kv4_workspace_bytes", "q4lin_kv4_attention", "q4lin_token_logprobs")

_lib = None


class Q4LinError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        detail = last_error_detail()
        super().__init__(f"q4lin: {what}{STATUS.get(status, status)}: {status_string(status)}"
                         + (f" [{detail}]" if detail else ""))


def last_error_detail() -> str:
    return load().q4lin_last_error_detail().decode(errors="replace")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library (once).  Raises if it is missing: build it first."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} not found: build it with `python -m weight_only_bit_q4_gb300.build`")
    lib = ctypes.CDLL(p)
    i64, sz, vp = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    lib.q4lin_workspace_bytes.argtypes = [i64, i64, i64]
    lib.q4lin_workspace_bytes.restype = sz
    lib.q4lin_route_workspace_bytes.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.q4lin_route_workspace_bytes.restype = sz
    lib.q4lin_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
    lib.q4lin_linear.restype = ctypes.c_int
    lib.q4lin_linear_route.argtypes = [ctypes.c_int, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    lib.q4lin_linear_qtype.argtypes = [ctypes.c_int, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    lib.q4lin_linear_qtype.restype = ctypes.c_int
    lib.q4lin_linear_fp16_static.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.q4lin_linear_fp16_static.restype = ctypes.c_int
    lib.q4lin_linear_route.restype = ctypes.c_int
    lib.q4lin_select_route.argtypes = [i64, i64, i64]
    lib.q4lin_select_route.restype = ctypes.c_int
    lib.q4lin_tile_plan.argtypes = [ctypes.c_int, i64, i64, i64, ctypes.POINTER(ctypes.c_int),
                                    ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int64),
                                    ctypes.POINTER(ctypes.c_int)]
    lib.q4lin_tile_plan.restype = ctypes.c_int
    lib.q4lin_kernel_launches.argtypes = [i64, i64, i64]
    lib.q4lin_kernel_launches.restype = ctypes.c_int
    lib.q4lin_linear_add.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.q4lin_linear_add.restype = ctypes.c_int
    lib.q4lin_qtype_kernel_launches.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.q4lin_qtype_kernel_launches.restype = ctypes.c_int
    lib.q4lin_status_string.argtypes = [ctypes.c_int]
    lib.q4lin_status_string.restype = ctypes.c_char_p
    lib.q4lin_device_status.argtypes = []
    lib.q4lin_device_status.restype = ctypes.c_int
    lib.q4lin_clear_device_status.argtypes = []
    lib.q4lin_clear_device_status.restype = ctypes.c_int
    lib.q4lin_last_error_detail.argtypes = []
    lib.q4lin_last_error_detail.restype = ctypes.c_char_p
    lib.q4lin_hbm_read_probe.argtypes = [vp, sz, vp, ctypes.c_int, vp]
    lib.q4lin_hbm_read_probe.restype = ctypes.c_int
    lib.q4lin_diag_wait_expiry.argtypes = [ctypes.c_uint32, vp, vp]
    lib.q4lin_diag_wait_expiry.restype = ctypes.c_int
    lib.q4lin_qtype_workspace_bytes.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.q4lin_qtype_workspace_bytes.restype = sz
    lib.q4lin_linear_swiglu.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.q4lin_linear_swiglu.restype = ctypes.c_int
    lib.q4lin_linear_pair.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp]
    lib.q4lin_linear_pair.restype = ctypes.c_int
    lib.q4lin_host_workspace_bytes.argtypes = [i64, i64, i64]
    lib.q4lin_host_workspace_bytes.restype = sz
    lib.q4lin_linear_host.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
    lib.q4lin_linear_host.restype = ctypes.c_int
    lib.q4lin_qtype_route.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.q4lin_qtype_route.restype = ctypes.c_int
    lib.q4lin_fused_route.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.q4lin_fused_route.restype = ctypes.c_int
    ci, cf = ctypes.c_int, ctypes.c_float
    lib.q4lin_lora_workspace_bytes.argtypes = [i64] * 5
    lib.q4lin_lora_workspace_bytes.restype = sz
    lib.q4lin_lora_route.argtypes = [i64] * 4
    lib.q4lin_lora_route.restype = ci
    lib.q4lin_linear_lora.argtypes = [vp] * 9 + [i64] * 5 + [vp, vp]
    lib.q4lin_linear_lora.restype = ci
    lib.q4lin_moe_router.argtypes = [vp] * 5 + [i64] * 3 + [ci, ci, vp]
    lib.q4lin_moe_router.restype = ci
    lib.q4lin_moe_workspace_bytes.argtypes = [i64] * 4 + [ci]
    lib.q4lin_moe_workspace_bytes.restype = sz
    lib.q4lin_moe_experts.argtypes = [vp] * 8 + [i64] * 4 + [ci, vp, vp]
    lib.q4lin_moe_experts.restype = ci
    lib.q4lin_moe.argtypes = [vp] * 10 + [i64] * 4 + [ci, ci, vp, vp]
    lib.q4lin_moe.restype = ci
    lib.q4lin_qk_norm_rope.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64] + [i64] * 6 + [cf, ci, vp]
    lib.q4lin_qk_norm_rope.restype = ci
    lib.q4lin_prompt_attention.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i64] + [i64] * 5 + [cf, vp]
    lib.q4lin_prompt_attention.restype = ci
    lib.q4lin_kv4_page_bytes.argtypes = [i64]
    lib.q4lin_kv4_page_bytes.restype = sz
    lib.q4lin_kv4_append.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp] + [i64] * 6 + [vp]
    lib.q4lin_kv4_append.restype = ci
    lib.q4lin_kv4_read.argtypes = [vp, vp, vp, vp, vp, i64, vp, i64] + [i64] * 6 + [vp]
    lib.q4lin_kv4_read.restype = ci
    lib.q4lin_kv4_workspace_bytes.argtypes = [i64] * 6
    lib.q4lin_kv4_workspace_bytes.restype = sz
    lib.q4lin_kv4_attention.argtypes = [vp, i64, vp, vp, vp, vp, i64] + [i64] * 7 + [cf, vp, vp]
    lib.q4lin_kv4_attention.restype = ci
    lib.q4lin_token_logprobs.argtypes = [vp, ci, i64, vp, vp, vp, vp, vp] + [i64] * 3 + [ci, vp]
    lib.q4lin_token_logprobs.restype = ci
    lib.q4lin_version.argtypes = []
    lib.q4lin_version.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().q4lin_status_string(int(status)).decode()


def version() -> str:
    return load().q4lin_version().decode()


def workspace_bytes(N: int, K: int, T: int, route: int = ROUTE_AUTO) -> int:
    if route == ROUTE_AUTO:
        return int(load().q4lin_workspace_bytes(N, K, T))
    return int(load().q4lin_route_workspace_bytes(route, N, K, T))


def select_route(N: int, K: int, T: int) -> int:
    return int(load().q4lin_select_route(N, K, T))


def tile_plan(N: int, K: int, T: int, route: int = ROUTE_AUTO) -> tuple:
    """(token-tile width, split-K cluster size) of the tensor-core route's main launch; (0, 1) for the GEMV."""
    p = tile_plan_full(N, K, T, route)
    return p["n"], p["split_k"]


def tile_plan_full(N: int, K: int, T: int, route: int = ROUTE_AUTO) -> dict:
    """The whole tensor-core plan: tile width, main-launch split, main-launch tiles, tail split (0 = none)."""
    bn, sk, mt, ts = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int64(0), ctypes.c_int(0)
    st = load().q4lin_tile_plan(route, N, K, T, ctypes.byref(bn), ctypes.byref(sk), ctypes.byref(mt),
                                ctypes.byref(ts))
    if st != OK:
        raise Q4LinError(st, "tile plan: ")
    return {"n": int(bn.value), "split_k": int(sk.value), "main_tiles": int(mt.value), "tail_split_k": int(ts.value)}


def kernel_launches(N: int, K: int, T: int, qtype: str = "q4g64") -> int:
    """Kernels one call launches (q4lin_linear, or q4lin_linear_qtype for another format)."""
    if qtype == "q4g64":
        return int(load().q4lin_kernel_launches(N, K, T))
    return int(load().q4lin_qtype_kernel_launches(QTYPES[qtype], N, K, T))


_IMPLEMENTED = (ROUTE_GEMV, ROUTE_TC_SPLITK, ROUTE_TC, ROUTE_TC_FP16, ROUTE_STREAM_MMA)


def implemented_routes():
    """Routes the library can run (the others return INVALID_ARG)."""
    return _IMPLEMENTED


def device_status() -> int:
    return int(load().q4lin_device_status())


def clear_device_status() -> int:
    return int(load().q4lin_clear_device_status())


_torch = None


def _t():
    """torch, imported at the first call (the binding itself loads without it)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _new(shape, dtype, device, stream, output=True):
    """A tensor that a call makes for itself.

    For a ``stream`` other than the current one it is that stream's: torch's allocator hands a
    freed block out again at once on the stream it belongs to, so scratch of the current stream,
    freed when the call returns, would be written over while the kernels on ``stream`` still use
    it.  An output goes on to the caller and is marked as used on the current stream too.
    """
    torch = _t()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if output:
        t.record_stream(current)
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def linear_raw(wq_ptr, scales_ptr, x_ptr, y_ptr, N, K, T, ws_ptr=None, stream=None,
               route: int = ROUTE_AUTO) -> int:
    """Pointer-level call; returns the status code (no exception)."""
    lib = load()
    if route == ROUTE_AUTO:
        return int(lib.q4lin_linear(wq_ptr, scales_ptr, x_ptr, y_ptr, N, K, T, ws_ptr, stream))
    return int(lib.q4lin_linear_route(route, wq_ptr, scales_ptr, x_ptr, y_ptr, N, K, T, ws_ptr, stream))


def linear(wq, scales, x, y=None, workspace=None, stream=None, route: int = ROUTE_AUTO):
    """Y[T, N] (bf16) = dequant(wq, scales) applied to X[T, K] (bf16) on the GPU.

    wq: uint8 [N, Kp/2]; scales: fp16 (or int16/uint16 bit patterns) [N, Kp/64],
    Kp = K rounded up to 128 (the planes' stored width; columns k >= K are
    padding); x: bf16 [T, K]; all CUDA, contiguous.  ``y`` (bf16 [T, N]) and
    ``workspace`` (uint8, >= workspace_bytes) are allocated here with torch if
    not given.  Runs on ``stream`` (a torch.cuda.Stream) or the current stream.
    As everywhere in this module, what is allocated here belongs to the stream of
    the call; tensors that are passed in must be ready on it and live until it is
    past the call.
    """
    import torch

    T, K = x.shape
    N = wq.shape[0]
    Kp = (K + 127) // 128 * 128
    if tuple(wq.shape) != (N, Kp // 2) or tuple(scales.shape) != (N, Kp // 64):
        raise ValueError(f"shape mismatch: wq {tuple(wq.shape)} scales {tuple(scales.shape)} x {tuple(x.shape)}")
    for name, t in (("wq", wq), ("scales", scales), ("x", x)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if wq.dtype != torch.uint8 or x.dtype != torch.bfloat16 or scales.element_size() != 2:
        raise ValueError("dtypes: wq uint8, scales fp16 bits, x bf16")
    if y is None:
        y = _new((T, N), torch.bfloat16, x.device, stream)
    elif y.shape != (T, N) or y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise ValueError("y must be a contiguous bf16 [T, N] tensor")
    need = workspace_bytes(N, K, T, route)
    if need and workspace is None:
        workspace = _new(need, torch.uint8, x.device, stream, output=False)
    s = (stream or torch.cuda.current_stream(x.device)).cuda_stream
    st = linear_raw(_ptr(wq), _ptr(scales), _ptr(x), _ptr(y), N, K, T,
                    _ptr(workspace) if need else None, ctypes.c_void_p(s), route)
    if st != OK:
        raise Q4LinError(st)
    return y


FUSED_OPS = {"add": 1, "swiglu": 2, "pair": 3}


def qtype_route(qtype: str, N: int, K: int, T: int) -> int:
    """Route q4lin_linear_qtype takes for this format and shape."""
    return int(load().q4lin_qtype_route(QTYPES[qtype], N, K, T))


def fused_route(op: str, N: int, K: int, T: int) -> int:
    """Route of a fused operation ("add", "swiglu", "pair"; N = F for swiglu, rows per weight for pair)."""
    return int(load().q4lin_fused_route(FUSED_OPS[op], N, K, T))


def host_workspace_bytes(N: int, K: int, T: int) -> int:
    return int(load().q4lin_host_workspace_bytes(N, K, T))


def linear_host(wq, scales, x_host, y_host=None, workspace=None, stream=None):
    """q4lin_linear_host: X and Y in page-locked host memory, the weights on the GPU.

    x_host: pinned CPU bf16 [T, K] (or int16 bit patterns); ``y_host`` (pinned CPU bf16
    [T, N]) and ``workspace`` (CUDA uint8, >= host_workspace_bytes) are allocated here if
    not given.  The call is stream-ordered: y_host holds the result once ``stream`` (a
    torch.cuda.Stream, default the current one) has passed it.
    """
    import torch

    T, K = x_host.shape
    N = wq.shape[0]
    Kp = (K + 127) // 128 * 128
    if tuple(wq.shape) != (N, Kp // 2) or tuple(scales.shape) != (N, Kp // 64):
        raise ValueError(f"shape mismatch: wq {tuple(wq.shape)} scales {tuple(scales.shape)} x {tuple(x_host.shape)}")
    for name, t in (("wq", wq), ("scales", scales)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if x_host.is_cuda or not x_host.is_contiguous() or x_host.element_size() != 2:
        raise ValueError("x_host must be a contiguous 2-byte CPU tensor (pinned)")
    if y_host is None:
        y_host = torch.empty((T, N), dtype=torch.bfloat16).pin_memory()
    elif y_host.is_cuda or tuple(y_host.shape) != (T, N) or y_host.element_size() != 2 or not y_host.is_contiguous():
        raise ValueError("y_host must be a contiguous 2-byte CPU [T, N] tensor (pinned)")
    if workspace is None:
        workspace = _new(max(host_workspace_bytes(N, K, T), 256), torch.uint8, wq.device, stream, output=False)
    s = (stream or torch.cuda.current_stream(wq.device)).cuda_stream
    st = int(load().q4lin_linear_host(_ptr(wq), _ptr(scales), _ptr(x_host), _ptr(y_host), N, K, T,
                                      _ptr(workspace), ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st)
    return y_host


def linear_add(wq, scales, x, r, y=None, stream=None):
    """LinearAdd: Y = W . X + R (bf16 [T, N]); ``y`` may be ``r`` itself for an in-place add."""
    import torch

    T, K = x.shape
    N = wq.shape[0]
    Kp = (K + 127) // 128 * 128
    if tuple(wq.shape) != (N, Kp // 2) or tuple(scales.shape) != (N, Kp // 64) or tuple(r.shape) != (T, N):
        raise ValueError(f"shape mismatch: wq {tuple(wq.shape)} scales {tuple(scales.shape)} x {tuple(x.shape)} "
                         f"r {tuple(r.shape)}")
    for name, t in (("wq", wq), ("scales", scales), ("x", x), ("r", r)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if y is None:
        y = _new((T, N), torch.bfloat16, x.device, stream)
    s = (stream or torch.cuda.current_stream(x.device)).cuda_stream
    st = int(load().q4lin_linear_add(_ptr(wq), _ptr(scales), _ptr(x), _ptr(r), _ptr(y), N, K, T, ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st)
    return y


def linear_qtype(qtype: str, planes, scales, x, y=None, stream=None):
    """Y[T, N] (bf16) for a sibling weight format ("q4g64", "q5g64", "q6g64", "w8g32").

    planes: (codes,) for q4g64 / w8g32, (low codes, high bits) for q5g64 / q6g64;
    planes and scales stored for Kp = K rounded up to 128 columns (see q4lin.h);
    all CUDA, contiguous.  Workspace (W8 beyond the decode GEMV) is allocated here.
    """
    import torch

    qt = QTYPES[qtype]
    T, K = x.shape
    Kp = (K + 127) // 128 * 128
    codes = planes[0]
    N = codes.shape[0]
    code_cols = Kp if qtype == "w8g32" else Kp // 2
    group = 32 if qtype == "w8g32" else 64
    bits = {"q5g64": 1, "q6g64": 2}.get(qtype, 0)
    if tuple(codes.shape) != (N, code_cols) or tuple(scales.shape) != (N, Kp // group):
        raise ValueError(f"shape mismatch: codes {tuple(codes.shape)} scales {tuple(scales.shape)} x {tuple(x.shape)}")
    high = planes[1] if bits else None
    if bits and tuple(high.shape) != (N, Kp * bits // 8):
        raise ValueError(f"shape mismatch: high {tuple(high.shape)}")
    for name, t in (("codes", codes), ("scales", scales), ("x", x)) + ((("high", high),) if bits else ()):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if y is None:
        y = _new((T, N), torch.bfloat16, x.device, stream)
    need = int(load().q4lin_qtype_workspace_bytes(qt, N, K, T))
    ws = _new(need, torch.uint8, x.device, stream, output=False) if need else None
    s = (stream or torch.cuda.current_stream(x.device)).cuda_stream
    st = int(load().q4lin_linear_qtype(qt, _ptr(codes), _ptr(high) if bits else None, _ptr(scales), _ptr(x),
                                       _ptr(y), N, K, T, _ptr(ws), ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st)
    return y


def hbm_read_probe(buf, sink, blocks: int = 0, stream=None) -> None:
    """Enqueue one pass of the HBM read probe over ``buf`` (a CUDA tensor, 16-byte
    aligned, size a multiple of 16 bytes); ``sink`` is an int32 CUDA tensor with at
    least ``blocks`` (default four per SM) elements."""
    import torch

    s = (stream or torch.cuda.current_stream(buf.device)).cuda_stream
    st = int(load().q4lin_hbm_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), int(blocks),
                                         ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st, "hbm read probe: ")


def diag_wait_expiry(limit: int, out, stream=None) -> None:
    """Enqueue the wait-expiry check (see q4lin.h); ``out`` is an int32 CUDA tensor."""
    import torch

    s = (stream or torch.cuda.current_stream(out.device)).cuda_stream
    st = int(load().q4lin_diag_wait_expiry(int(limit), _ptr(out), ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st, "wait expiry check: ")


def _check_planes(wq, scales, K, what):
    Kp = (K + 127) // 128 * 128
    if wq.shape[1] != Kp // 2 or tuple(scales.shape) != (wq.shape[0], Kp // 64):
        raise ValueError(f"{what}: shape mismatch wq {tuple(wq.shape)} scales {tuple(scales.shape)} K {K}")
    for name, t in (("wq", wq), ("scales", scales)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be a contiguous CUDA tensor")


def linear_swiglu(wq, scales, x, y=None, stream=None):
    """LinearSwiGLU: Y[T, F] = silu(W[:F] . X) * (W[F:] . X) for a packed weight of 2F rows."""
    import torch

    T, K = x.shape
    n2 = wq.shape[0]
    if n2 % 2:
        raise ValueError("the gate/up weight has an even number of rows")
    F = n2 // 2
    _check_planes(wq, scales, K, "linear_swiglu")
    if y is None:
        y = _new((T, F), torch.bfloat16, x.device, stream)
    s = (stream or torch.cuda.current_stream(x.device)).cuda_stream
    st = int(load().q4lin_linear_swiglu(_ptr(wq), _ptr(scales), _ptr(x), _ptr(y), F, K, T, ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st)
    return y


def linear_pair(wq_a, scales_a, wq_b, scales_b, x, y_a=None, y_b=None, stream=None):
    """LinearPair: (W_a . X, W_b . X) in one call; returns (Y_a [T, N_a], Y_b [T, N_b])."""
    import torch

    T, K = x.shape
    _check_planes(wq_a, scales_a, K, "linear_pair a")
    _check_planes(wq_b, scales_b, K, "linear_pair b")
    Na, Nb = wq_a.shape[0], wq_b.shape[0]
    if y_a is None:
        y_a = _new((T, Na), torch.bfloat16, x.device, stream)
    if y_b is None:
        y_b = _new((T, Nb), torch.bfloat16, x.device, stream)
    s = (stream or torch.cuda.current_stream(x.device)).cuda_stream
    st = int(load().q4lin_linear_pair(_ptr(wq_a), _ptr(scales_a), _ptr(wq_b), _ptr(scales_b), _ptr(x), _ptr(y_a),
                                      _ptr(y_b), Na, Nb, K, T, ctypes.c_void_p(s)))
    if st != OK:
        raise Q4LinError(st)
    return y_a, y_b


# ---------------------------------------------------------------- operators around the projections
# These are called once or more per token of a decode step, where the host's time per call
# counts: each tensor is checked once, with attribute reads only, and pointers go to the
# library as plain integers.

def _stream_ptr(stream, device):
    if stream is not None:
        return stream.cuda_stream
    return _t()._C._cuda_getCurrentRawStream(device.index)


def _need(name, t, dtype, shape):
    """A contiguous CUDA tensor of this dtype and shape; returns its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor {dtype} {tuple(shape)}; got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _need_bits16(name, t, shape):
    """fp16 scales, or their bit patterns in a 2-byte integer type."""
    if t.element_size() != 2 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-byte CUDA tensor {tuple(shape)}; got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _scratch(workspace, need, device, stream):
    """(address, the tensor that keeps it alive) of at least ``need`` workspace bytes."""
    if need == 0:
        return None, None
    if workspace is None:
        workspace = _new(need, _t().uint8, device, stream, output=False)
    elif not workspace.is_cuda or not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes")
    return workspace.data_ptr(), workspace


def lora_workspace_bytes(N: int, K: int, T: int, L: int, R: int) -> int:
    """Workspace bytes of linear_lora for N x K weights, T tokens, L adapters of rank up to R."""
    return int(load().q4lin_lora_workspace_bytes(N, K, T, L, R))


def lora_route(N: int, K: int, T: int, R: int) -> int:
    """Route linear_lora takes (as select_route), -1 for sizes it refuses."""
    return int(load().q4lin_lora_route(N, K, T, R))


def linear_lora(wq, scales, x, lora_a, lora_b, adapter_ids, adapter_scales=None, ranks=None, y=None, workspace=None,
                stream=None):
    """Y[T, N] = W X + scale_a B_a (A_a X), token by token with the adapter a = adapter_ids[t].

    wq, scales, x as ``linear``; lora_a bf16 [L, R, K]; lora_b bf16 [L, N, R]; adapter_ids
    int32 [T] (outside [0, L): no adapter); adapter_scales fp32 [L] or None; ranks int32 [L]
    or None (the first ranks[a] rows of A_a and columns of B_a are used); R a multiple of 8
    up to 256.  ``y`` (bf16 [T, N]) and ``workspace`` (uint8, >= lora_workspace_bytes) are
    allocated here if not given.
    """
    torch = _t()
    bf16 = torch.bfloat16
    T, K = x.shape
    L, R, _ = lora_a.shape
    N = wq.shape[0]
    Kp = (K + 127) // 128 * 128
    lib = load()
    dev = x.device
    if y is None:
        y = _new((T, N), bf16, dev, stream)
    ws, ws_keep = _scratch(workspace, lib.q4lin_lora_workspace_bytes(N, K, T, L, R), dev, stream)
    st = lib.q4lin_linear_lora(
        _need("wq", wq, torch.uint8, (N, Kp // 2)), _need_bits16("scales", scales, (N, Kp // 64)), _need("x", x, bf16, (T, K)),
        _need("lora_a", lora_a, bf16, (L, R, K)), _need("lora_b", lora_b, bf16, (L, N, R)),
        _need("adapter_ids", adapter_ids, torch.int32, (T,)),
        None if adapter_scales is None else _need("adapter_scales", adapter_scales, torch.float32, (L,)),
        None if ranks is None else _need("ranks", ranks, torch.int32, (L,)), _need("y", y, bf16, (T, N)),
        N, K, T, L, R, ws, _stream_ptr(stream, dev))
    if st != OK:
        raise Q4LinError(st)
    return y


def moe_workspace_bytes(T: int, H: int, F: int, E: int, top_k: int) -> int:
    """Workspace bytes of moe / moe_experts."""
    return int(load().q4lin_moe_workspace_bytes(T, H, F, E, top_k))


def moe_router(x, w_router, top_k: int, bias=None, renormalize: bool = True, ids=None, weights=None, stream=None):
    """The top_k experts of every token and their softmax weights: (ids int32 [T, top_k], weights fp32 [T, top_k]).

    x bf16 [T, H]; w_router bf16 [E, H]; bias fp32 [E] added to the logits (-inf: the expert is
    never chosen) or None.  Where fewer than top_k experts can be chosen, id -1 with weight 0.
    """
    torch = _t()
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    if ids is None:
        ids = _new((T, top_k), torch.int32, dev, stream)
    if weights is None:
        weights = _new((T, top_k), torch.float32, dev, stream)
    st = load().q4lin_moe_router(
        _need("x", x, torch.bfloat16, (T, H)), _need("w_router", w_router, torch.bfloat16, (E, H)),
        None if bias is None else _need("bias", bias, torch.float32, (E,)), _need("ids", ids, torch.int32, (T, top_k)),
        _need("weights", weights, torch.float32, (T, top_k)), T, H, E, top_k, 1 if renormalize else 0,
        _stream_ptr(stream, dev))
    if st != OK:
        raise Q4LinError(st)
    return ids, weights


def _expert_planes(wq_gate_up, scales_gate_up, wq_down, scales_down, H):
    """Checked addresses of the experts' planes, E and F."""
    torch = _t()
    E, F2 = wq_gate_up.shape[:2]
    if F2 % 2:
        raise ValueError("wq_gate_up holds an even number of rows per expert: gate rows, then up rows")
    F = F2 // 2
    Hp, Fp = (H + 127) // 128 * 128, (F + 127) // 128 * 128
    return (_need("wq_gate_up", wq_gate_up, torch.uint8, (E, F2, Hp // 2)),
            _need_bits16("scales_gate_up", scales_gate_up, (E, F2, Hp // 64)),
            _need("wq_down", wq_down, torch.uint8, (E, H, Fp // 2)),
            _need_bits16("scales_down", scales_down, (E, H, Fp // 64)), E, F)


def moe_experts(x, ids, weights, wq_gate_up, scales_gate_up, wq_down, scales_down, y=None, workspace=None, stream=None):
    """Y[T, H] = sum_j weights[t, j] W_down,e (silu(W_gate,e x) * (W_up,e x)), e = ids[t, j].

    x bf16 [T, H]; ids int32 and weights fp32 [T, top_k] (an id outside [0, E): that choice adds
    nothing); wq_gate_up uint8 [E, 2F, Hp/2] (gate rows, then up rows), wq_down uint8 [E, H, Fp/2]
    with their fp16 scales per 64 columns (Hp, Fp: H, F rounded up to 128).
    """
    torch = _t()
    T, H = x.shape
    k = ids.shape[1]
    gu, gus, dn, dns, E, F = _expert_planes(wq_gate_up, scales_gate_up, wq_down, scales_down, H)
    lib = load()
    if y is None:
        y = _new((T, H), torch.bfloat16, x.device, stream)
    ws, ws_keep = _scratch(workspace, lib.q4lin_moe_workspace_bytes(T, H, F, E, k), x.device, stream)
    st = lib.q4lin_moe_experts(
        _need("x", x, torch.bfloat16, (T, H)), _need("ids", ids, torch.int32, (T, k)),
        _need("weights", weights, torch.float32, (T, k)), gu, gus, dn, dns, _need("y", y, torch.bfloat16, (T, H)),
        T, H, F, E, k, ws, _stream_ptr(stream, x.device))
    if st != OK:
        raise Q4LinError(st)
    return y


def moe(x, w_router, wq_gate_up, scales_gate_up, wq_down, scales_down, top_k: int, bias=None, renormalize: bool = True,
        y=None, ids=None, weights=None, workspace=None, stream=None):
    """The whole mixture-of-experts layer, ``moe_router`` then ``moe_experts`` in one call: (y, ids, weights)."""
    torch = _t()
    T, H = x.shape
    dev = x.device
    gu, gus, dn, dns, E, F = _expert_planes(wq_gate_up, scales_gate_up, wq_down, scales_down, H)
    lib = load()
    if y is None:
        y = _new((T, H), torch.bfloat16, dev, stream)
    if ids is None:
        ids = _new((T, top_k), torch.int32, dev, stream)
    if weights is None:
        weights = _new((T, top_k), torch.float32, dev, stream)
    ws, ws_keep = _scratch(workspace, lib.q4lin_moe_workspace_bytes(T, H, F, E, top_k), dev, stream)
    st = lib.q4lin_moe(
        _need("x", x, torch.bfloat16, (T, H)), _need("w_router", w_router, torch.bfloat16, (E, H)),
        None if bias is None else _need("bias", bias, torch.float32, (E,)), gu, gus, dn, dns,
        _need("ids", ids, torch.int32, (T, top_k)), _need("weights", weights, torch.float32, (T, top_k)),
        _need("y", y, torch.bfloat16, (T, H)), T, H, F, E, top_k, 1 if renormalize else 0, ws, _stream_ptr(stream, dev))
    if st != OK:
        raise Q4LinError(st)
    return y, ids, weights


def _rows(name, t, D, bf16):
    """Address, row stride and heads of bf16 rows [T, heads * D] or [T, heads, D], contiguous within a row."""
    if t.dtype is not bf16 or not t.is_cuda:
        raise ValueError(f"{name} must be a bf16 CUDA tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        n = shape[1]
        if D == 0 or n % D or stride[1] != 1:
            raise ValueError(f"{name} must be [T, heads * {D}] or [T, heads, {D}] with contiguous rows")
        return t.data_ptr(), stride[0] if shape[0] > 1 else n, n // D
    if len(shape) != 3 or shape[2] != D or stride[2] != 1 or (shape[1] > 1 and stride[1] != D):
        raise ValueError(f"{name}: the heads of a row must lie side by side, {D} values each")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * D, shape[1]


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                 k_out=None, stream=None):
    """RMS norm of every query and key head, then the rotation by the token's position: (q_out, k_out).

    q bf16 [T, Hq * D] (or [T, Hq, D]) and k likewise, rows of any stride (slices of a packed
    projection output); q_weight, k_weight bf16 [D]; cos_sin fp32 [P, rot] (rot / 2 cosines, then
    sines); positions int32 [T] (outside [0, P): the token's outputs are not written).  ``q_out``
    and ``k_out`` may be q and k (in place); allocated here if not given.
    """
    torch = _t()
    D = q_weight.shape[0]
    T = q.shape[0]
    P, rot = cos_sin.shape
    if q_out is None:
        q_out = _new(q.shape, q.dtype, q.device, stream)
    if k_out is None:
        k_out = _new(k.shape, k.dtype, k.device, stream)
    bf16 = torch.bfloat16
    qp, ldq, hq = _rows("q", q, D, bf16)
    kp, ldk, hk = _rows("k", k, D, bf16)
    qo, ldqo, hqo = _rows("q_out", q_out, D, bf16)
    ko, ldko, hko = _rows("k_out", k_out, D, bf16)
    if (hqo, hko) != (hq, hk) or k.shape[0] != T or q_out.shape[0] != T or k_out.shape[0] != T:
        raise ValueError("q, k and their outputs must have the same tokens and heads")
    st = load().q4lin_qk_norm_rope(
        qp, ldq, kp, ldk, _need("q_weight", q_weight, bf16, (D,)), _need("k_weight", k_weight, bf16, (D,)),
        _need("cos_sin", cos_sin, torch.float32, (P, rot)), _need("positions", positions, torch.int32, (T,)), qo, ldqo, ko,
        ldko, T, hq, hk, D, rot, P, eps, 1 if interleaved else 0, _stream_ptr(stream, q.device))
    if st != OK:
        raise Q4LinError(st)
    return q_out, k_out


# ---------------------------------------------------------------- attention, its 4-bit cache, and the logits' answers

KV_PAGE = 64   # tokens of a cache page
_PAGE_BYTES = {}


def _page_bytes(D):
    if D not in _PAGE_BYTES:
        _PAGE_BYTES[D] = int(load().q4lin_kv4_page_bytes(D))
    return _PAGE_BYTES[D]


def _run(index, fn, *args):
    """The library works on the current device: device ``index`` becomes it for the call if it is another."""
    if _torch._C._cuda_getDevice() == index:
        st = fn(*args)
    else:
        with _torch.cuda.device(index):
            st = fn(*args)
    if st != OK:
        raise Q4LinError(st)


def _same_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on one device; got {t.device} beside cuda:{index}")


def _raw_stream(stream, index):
    return _torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _out(t, name, shape, dtype, device, stream):
    """(address, tensor) of an output: the one given, checked, or a new one."""
    if t is None:
        t = _new(shape, dtype, device, stream)
        return t.data_ptr(), t
    return _need(name, t, dtype, shape), t


def prompt_attention(q, k, v, cu_seqlens, scale: float | None = None, out=None, stream=None):
    """Causal attention of packed prompts, each token over its own sequence up to itself: out [T, Hq, D].

    q bf16 [T, Hq, D]; k, v bf16 [T, Hk, D] (or [T, Hk * D]), Hq a multiple of Hk, D a multiple of 8 up to
    128, rows of any stride (slices of a packed projection output); cu_seqlens int32 [S + 1] on the GPU:
    sequence s is rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (rows outside all of them are not
    written).  ``scale`` is D ** -0.5 if not given.
    """
    torch = _t()
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    T, hq, D = q.shape
    if out is None:
        out = _new((T, hq, D), torch.bfloat16, q.device, stream)
    bf16 = torch.bfloat16
    qp, ldq, _ = _rows("q", q, D, bf16)
    kp, ldk, hk = _rows("k", k, D, bf16)
    vp, ldv, hv = _rows("v", v, D, bf16)
    op, ldo, ho = _rows("out", out, D, bf16)
    if k.shape[0] != T or v.shape[0] != T or out.shape[0] != T or hk != hv or ho != hq:
        raise ValueError("q, k, v and out must have the same tokens; k and v, and q and out the same heads")
    S = cu_seqlens.shape[0] - 1
    if S < 0:
        raise ValueError("cu_seqlens holds one value more than there are sequences")
    dev = q.get_device()
    _same_device(dev, k, v, cu_seqlens, out)
    _run(dev, load().q4lin_prompt_attention, qp, ldq, kp, ldk, vp, ldv,
         _need("cu_seqlens", cu_seqlens, torch.int32, (S + 1,)), op, ldo, T, S, hq, hk, D,
         D ** -0.5 if scale is None and D else scale or 0.0, _raw_stream(stream, dev))
    return out


def kv4_page_bytes(D: int) -> int:
    """Bytes that a page of the cache (KV_PAGE tokens) holds per head of D values; 0 for sizes it does not take."""
    return _page_bytes(D)


def _cache(cache, page_table, D):
    """Checked addresses and sizes of a cache uint8 [pages, Hk, page bytes] and its page table int32 [S, max_pages]."""
    torch = _t()
    if cache.dim() != 3 or page_table.dim() != 2:
        raise ValueError("cache must be [pages, Hk, page bytes] and page_table [S, max_pages]")
    P, hk, _ = cache.shape
    S, M = page_table.shape
    nb = _page_bytes(D)
    if nb == 0:
        raise ValueError(f"the cache takes heads of 64, 96 or 128 values, not {D}")
    return (_need("cache", cache, torch.uint8, (P, hk, nb)), _need("page_table", page_table, torch.int32, (S, M)), P, hk, S, M)


def kv4_append(k, v, cache, page_table, positions, rows=None, stream=None):
    """Keys and values of T tokens into the 4-bit cache (in place); returns the cache.

    k, v bf16 [T, Hk, D], rows of any stride; cache uint8 [pages, Hk, kv4_page_bytes(D)]; page_table
    int32 [S, max_pages]: the page of each KV_PAGE tokens of a sequence; token t is token positions[t] (int32)
    of sequence rows[t] (int32; None: of sequence t).  Tokens whose row, position or page is out of
    range are left out; the places written to must differ.
    """
    torch = _t()
    if k.dim() != 3:
        raise ValueError("k must be [T, Hk, D]")
    T, hk, D = k.shape
    dev = k.get_device()
    cp, tp, P, hc, S, M = _cache(cache, page_table, D)
    kp, ldk, _ = _rows("k", k, D, torch.bfloat16)
    vp, ldv, hv = _rows("v", v, D, torch.bfloat16)
    if hc != hk or hv != hk or v.shape[0] != T:
        raise ValueError("k, v and the cache must have the same heads, k and v the same tokens")
    if rows is None and T > S:
        raise ValueError("without rows token t belongs to sequence t: more tokens than sequences")
    _same_device(dev, v, cache, page_table, positions, rows)
    _run(dev, load().q4lin_kv4_append, kp, ldk, vp, ldv, cp, tp,
         None if rows is None else _need("rows", rows, torch.int32, (T,)), _need("positions", positions, torch.int32, (T,)),
         T, S, M, P, hk, D, _raw_stream(stream, dev))
    return cache


def kv4_read(cache, page_table, positions, D: int, rows=None, k=None, v=None, stream=None):
    """What the cache holds for T tokens: (k, v) bf16 [T, Hk, D].  Arguments as ``kv4_append``; the rows of
    tokens that are out of range are left as they are (zeros where k and v are made here)."""
    torch = _t()
    T = positions.shape[0]
    dev = cache.get_device()
    cp, tp, P, hk, S, M = _cache(cache, page_table, D)

    def fresh():
        t = _new((T, hk, D), torch.bfloat16, cache.device, stream)
        with torch.cuda.stream(stream):
            return t.zero_()

    k = fresh() if k is None else k
    v = fresh() if v is None else v
    kp, ldk, h1 = _rows("k", k, D, torch.bfloat16)
    vp, ldv, h2 = _rows("v", v, D, torch.bfloat16)
    if h1 != hk or h2 != hk or k.shape[0] != T or v.shape[0] != T:
        raise ValueError("k and v must have the cache's heads and a row per token")
    if rows is None and T > S:
        raise ValueError("without rows token t belongs to sequence t: more tokens than sequences")
    _same_device(dev, page_table, positions, rows, k, v)
    _run(dev, load().q4lin_kv4_read, cp, tp, None if rows is None else _need("rows", rows, torch.int32, (T,)),
         _need("positions", positions, torch.int32, (T,)), kp, ldk, vp, ldv, T, S, M, P, hk, D, _raw_stream(stream, dev))
    return k, v


_KV_NEED = {}   # (device, S, q_len, Hq, Hk, D, max_pages): workspace bytes


def kv4_workspace_bytes(S: int, q_len: int, Hq: int, Hk: int, D: int, max_pages: int, device: int | None = None) -> int:
    """Workspace bytes of kv4_attention on a device (its index; None: the current one)."""
    sizes = (S, q_len, Hq, Hk, D, max_pages)
    if device is None:
        return int(load().q4lin_kv4_workspace_bytes(*sizes))
    key = (device, *sizes)
    if key not in _KV_NEED:
        if len(_KV_NEED) > 4096:
            _KV_NEED.clear()
        with _t().cuda.device(device):   # (the library answers for the current device)
            _KV_NEED[key] = int(load().q4lin_kv4_workspace_bytes(*sizes))
    return _KV_NEED[key]


def kv4_attention(q, cache, page_table, lengths, scale: float | None = None, out=None, workspace=None, stream=None):
    """Attention of each sequence's newest tokens over the 4-bit cache: out [S * q_len, Hq, D].

    q bf16 [S * q_len, Hq, D], rows of any stride: row s * q_len + i is the token that sees the first
    lengths[s] - (q_len - 1 - i) tokens of sequence s (none: zeros); lengths int32 [S]; cache and
    page_table as ``kv4_append``.  ``scale`` is D ** -0.5 if not given; ``workspace`` (uint8, >=
    kv4_workspace_bytes) is allocated here if not given.
    """
    torch = _t()
    if q.dim() != 3:
        raise ValueError("q must be [S * q_len, Hq, D]")
    T, hq, D = q.shape
    cp, tp, P, hk, S, M = _cache(cache, page_table, D)
    n = T // S if S else 0
    if n * S != T:
        raise ValueError("q must hold the same number of tokens for every sequence")
    if out is None:
        out = _new((T, hq, D), torch.bfloat16, q.device, stream)
    qp, ldq, _ = _rows("q", q, D, torch.bfloat16)
    op, ldo, ho = _rows("out", out, D, torch.bfloat16)
    if ho != hq or out.shape[0] != T:
        raise ValueError("out must have q's tokens and heads")
    dev = q.get_device()
    _same_device(dev, cache, page_table, lengths, out, workspace)
    ws, ws_keep = _scratch(workspace, kv4_workspace_bytes(S, n, hq, hk, D, M, dev), q.device, stream)
    _run(dev, load().q4lin_kv4_attention, qp, ldq, cp, tp, _need("lengths", lengths, torch.int32, (S,)), op, ldo, S, n, hq, hk, D,
         M, P, D ** -0.5 if scale is None else scale, ws, _raw_stream(stream, dev))
    return out


def token_logprobs(logits, targets, top_k: int = 0, logprobs=None, entropy=None, top_ids=None, top_logprobs=None,
                   stream=None):
    """Log probabilities of given tokens, the entropy and the top tokens of rows of logits:
    (logprobs fp32 like targets, entropy fp32 [T], top_ids int32 [T, top_k], top_logprobs fp32 [T, top_k]).

    logits bf16 or fp32 [T, V], rows of any stride; targets int32 [T] or [T, n] (outside [0, V): 0);
    top_k up to 32, largest first, ties by the lowest token.  Logits of -inf are never among the top
    (id -1, -inf where too few are left).
    """
    torch = _t()
    T, V = logits.shape
    if top_k < 0:
        raise ValueError("top_k must not be negative")
    wide = logits.dtype is torch.float32
    if not (wide or logits.dtype is torch.bfloat16) or not logits.is_cuda or (logits.stride(1) != 1 and V > 1):
        raise ValueError("logits must be a bf16 or fp32 CUDA tensor [T, V] with contiguous rows")
    if targets.dim() not in (1, 2):
        raise ValueError("targets must be [T] or [T, n]")
    n = 1 if targets.dim() == 1 else targets.shape[1]
    f32 = torch.float32
    index, dev = logits.get_device(), logits.device
    _same_device(index, targets, logprobs, entropy, top_ids, top_logprobs)
    shape = targets.shape
    if shape[0] != T:
        raise ValueError("targets must have a row per row of logits")
    tok = _need("targets", targets, torch.int32, shape)
    lp, logprobs = _out(logprobs, "logprobs", shape, f32, dev, stream)
    ep, entropy = _out(entropy, "entropy", (T,), f32, dev, stream)
    ip, top_ids = _out(top_ids, "top_ids", (T, top_k), torch.int32, dev, stream)
    tp, top_logprobs = _out(top_logprobs, "top_logprobs", (T, top_k), f32, dev, stream)
    _run(index, load().q4lin_token_logprobs, logits.data_ptr(), 1 if wide else 0,
         logits.stride(0) if T > 1 else V, tok, lp, ep, ip, tp, T, V, n, top_k, _raw_stream(stream, index))
    return logprobs, entropy, top_ids, top_logprobs

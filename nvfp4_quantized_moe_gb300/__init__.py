"""Python binding of libftmoe, the sm_103a NVFP4 (W4A16) routed-MoE expert forward.

Argument marshalling only: every function forwards to the C entry point of the same
name in ``libftmoe.so`` (declared in ``include/ft_moe.h``), passing torch tensors'
device pointers and the current CUDA stream. All arithmetic runs in the library's
CUDA kernels; there is no Python or CPU fallback, and importing this package fails
loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "FtMoeError", "MoEConfig", "load", "ft_moe_layout", "ft_moe_pack", "ft_moe_route", "ft_moe_route_gemm",
    "ft_moe_workspace_size", "ft_moe_forward", "ft_moe_align_workspace_size", "ft_moe_align",
    "ft_moe_dequant", "ft_moe_read_status", "ft_last_error", "alloc_banks", "EXPORTS",
    "FT_GU", "FT_GU_SCALE", "FT_GU_GLOBAL", "FT_DN", "FT_DN_SCALE", "FT_DN_GLOBAL",
    "FT_DTYPE_BF16", "FT_DTYPE_F32", "STATUS", "ft_moe_set_stage_events", "ft_moe_launch_count",
    "FT_NSTAGES", "STAGES", "ft_moe_debug_inject_stall", "ft_moe_workspace_size_w4a4", "ft_moe_forward_w4a4",
    "ft_moe_quantize_nvfp4", "ft_moe_group_workspace_size", "ft_moe_group_gemm", "ft_moe_group_gemm_dgrad",
    "ft_moe_group_gemm_wgrad", "ft_moe_group_gemm_fp8", "ft_moe_quantize_fp8", "ft_moe_swiglu",
    "ft_moe_swiglu_quantize_fp8", "ft_moe_swiglu_backward", "ft_moe_debug_group_plan", "FT_GROUP_FORWARD",
    "FT_GROUP_DGRAD", "FT_GROUP_WGRAD", "FT_GROUP_FP8", "FT_GROUP_MXFP4", "ft_moe_group_gemm_mxfp4",
    "ft_moe_quantize_mxfp4", "ft_moe_quantize_mxfp4_weights", "ft_moe_pack_mxfp4_scales",
    "ft_moe_swiglu_quantize_mxfp4", "alloc_mxfp4_scales", "ft_moe_dispatch", "ft_moe_dispatch_backward",
    "ft_moe_combine", "ft_moe_combine_backward", "ft_moe_rmsnorm", "ft_moe_rmsnorm_workspace_size",
    "ft_moe_rmsnorm_backward",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libftmoe.so")

FT_GU, FT_GU_SCALE, FT_GU_GLOBAL, FT_DN, FT_DN_SCALE, FT_DN_GLOBAL, FT_NBANKS = range(7)
FT_DTYPE_U8, FT_DTYPE_E4M3, FT_DTYPE_F32, FT_DTYPE_BF16 = range(4)
FT_FORMAT_NVFP4, FT_FORMAT_FP8_BLOCK = range(2)
STATUS = {0: "FT_OK", 1: "FT_ERR_INVALID_ARG", 2: "FT_ERR_INDIVISIBLE", 3: "FT_ERR_UNSUPPORTED",
          4: "FT_ERR_WORKSPACE", 5: "FT_ERR_CUDA", 6: "FT_ERR_INVALID_ROUTING", 7: "FT_ERR_TIMEOUT",
          8: "FT_ERR_BOUNDS"}
BANK_NAMES = ("gate_up", "gate_up_scale", "gate_up_global", "down", "down_scale", "down_global")

# Every symbol include/ft_moe.h declares.
EXPORTS = ("ft_moe_layout", "ft_moe_pack", "ft_moe_route", "ft_moe_route_gemm", "ft_moe_workspace_size",
           "ft_moe_forward", "ft_moe_align_workspace_size", "ft_moe_align", "ft_moe_dequant", "ft_moe_read_status",
           "ft_last_error", "ft_moe_set_stage_events", "ft_moe_launch_count", "ft_moe_align_static",
           "ft_moe_debug_inject_stall", "ft_moe_workspace_size_w4a4", "ft_moe_forward_w4a4", "ft_moe_quantize_nvfp4",
           "ft_moe_group_workspace_size", "ft_moe_group_gemm", "ft_moe_group_gemm_dgrad", "ft_moe_group_gemm_wgrad",
           "ft_moe_group_gemm_fp8", "ft_moe_quantize_fp8", "ft_moe_swiglu", "ft_moe_swiglu_quantize_fp8",
           "ft_moe_swiglu_backward", "ft_moe_debug_group_plan", "ft_moe_group_gemm_mxfp4", "ft_moe_quantize_mxfp4",
           "ft_moe_quantize_mxfp4_weights", "ft_moe_pack_mxfp4_scales", "ft_moe_swiglu_quantize_mxfp4",
           "ft_moe_dispatch", "ft_moe_dispatch_backward", "ft_moe_combine", "ft_moe_combine_backward",
           "ft_moe_rmsnorm", "ft_moe_rmsnorm_workspace_size", "ft_moe_rmsnorm_backward")
FT_GROUP_FORWARD, FT_GROUP_DGRAD, FT_GROUP_WGRAD, FT_GROUP_FP8, FT_GROUP_MXFP4 = range(5)
FT_NSTAGES = 6
STAGES = ("align", "gate_up", "shared_gate_up", "down", "shared_down", "combine")


class FtMoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class MoEConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("group", ctypes.c_int32), ("shared_intermediate", ctypes.c_int32),
                ("tp_rank", ctypes.c_int32), ("tp_size", ctypes.c_int32), ("shard_begin", ctypes.c_int32),
                ("shard_size", ctypes.c_int32), ("shared_shard_begin", ctypes.c_int32),
                ("shared_shard_size", ctypes.c_int32), ("format", ctypes.c_int32)]

    @classmethod
    def of(cls, shape, tp_rank: int = 0, tp_size: int = 1, shard=None, shared_shard=None) -> "MoEConfig":
        """Even split (tp_rank of tp_size) or explicit (begin, size) ranges of the intermediate."""
        sb, ss = shard if shard else (0, 0)
        hb, hs = shared_shard if shared_shard else (0, 0)
        fmt = FT_FORMAT_FP8_BLOCK if getattr(shape, "fmt", "nvfp4") == "fp8_block" else FT_FORMAT_NVFP4
        return cls(shape.hidden, shape.intermediate, shape.num_experts, shape.top_k, shape.group,
                   shape.shared_intermediate, tp_rank, tp_size, sb, ss, hb, hs, fmt)


class _BankSpec(ctypes.Structure):
    _fields_ = [("shape", ctypes.c_int64 * 3), ("ndim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("bytes", ctypes.c_int64)]


class _Banks(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p * FT_NBANKS)]


class _Pieces(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate", "gate_scale", "gate_global", "up", "up_scale", "up_global",
                                               "down", "down_scale", "down_global")] + [("on_device", ctypes.c_int32)]


_lib = None


def load():
    """Load libftmoe.so; raise if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libftmoe.so not built at {LIB_PATH}: run nvfp4_quantized_moe_gb300/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        F32 = ctypes.c_float
        sigs = {
            "ft_moe_layout": [P, I32, P],
            "ft_moe_pack": [P, I32, P, P, P],
            "ft_moe_route": [P, I32, I32, I32, P, P, P],
            "ft_moe_route_gemm": [P, I32, I32, P, I32, I32, P, P, P, P],
            "ft_moe_workspace_size": [P, I32, P],
            "ft_moe_forward": [P, P, P, P, I32, P, P, P, I32, P, SZ, P],
            "ft_moe_align_workspace_size": [I32, I32, I32, P],
            "ft_moe_align": [P, I32, I32, I32, I32, P, P, P, P, P, SZ, P],
            "ft_moe_dequant": [P, I32, P, I32, I32, P, P],
            "ft_moe_read_status": [P, P],
            "ft_moe_set_stage_events": [P],
            "ft_moe_debug_inject_stall": [ctypes.c_uint64, I32],
            "ft_moe_workspace_size_w4a4": [P, I32, P],
            "ft_moe_forward_w4a4": [P, P, P, P, I32, P, P, P, I32, P, SZ, P],
            "ft_moe_quantize_nvfp4": [P, I32, I32, I32, P, P, P, P],
            "ft_moe_group_workspace_size": [I32, I32, I32, I32, P],
            "ft_moe_group_gemm": [P, I64, P, P, I32, I32, I32, I32, P, I64, I32, P, SZ, P],
            "ft_moe_group_gemm_dgrad": [P, I64, P, P, I32, I32, I32, I32, P, I64, I32, P, SZ, P],
            "ft_moe_group_gemm_wgrad": [P, I64, P, I64, P, I32, I32, I32, I32, P, I32, I32, P, SZ, P],
            "ft_moe_group_gemm_fp8": [P, I64, P, I64, P, P, P, I32, I32, I32, I32, P, I64, I32, P, SZ, P],
            "ft_moe_quantize_fp8": [P, I32, I64, I32, I32, P, I64, P, I64, P],
            "ft_moe_swiglu": [P, I64, P, I32, I32, P, I64, P],
            "ft_moe_swiglu_quantize_fp8": [P, I64, P, I32, I32, P, I64, P, I64, P],
            "ft_moe_debug_group_plan": [I32, I32, I32, I32, I32, I32, I32, P],
            "ft_moe_swiglu_backward": [P, I64, P, P, I64, I32, I32, P, I64, P, P],
            "ft_moe_group_gemm_mxfp4": [P, I64, P, I64, P, P, P, I32, I32, I32, I32, P, I64, I32, P, SZ, P],
            "ft_moe_quantize_mxfp4": [P, I32, I64, I32, I32, P, I64, P, I64, P],
            "ft_moe_quantize_mxfp4_weights": [P, I32, I32, I32, I32, P, P, P],
            "ft_moe_pack_mxfp4_scales": [P, I32, I32, I32, P, P],
            "ft_moe_swiglu_quantize_mxfp4": [P, I64, P, I32, I32, P, I64, P, I64, P],
            "ft_moe_dispatch": [P, I64, I32, I32, I32, P, I32, P, P, I64, P, I64, I32, P, I64, P, P, P, P],
            "ft_moe_dispatch_backward": [P, I64, I32, P, I32, I32, I32, I32, P, P, I64, I32, P, P],
            "ft_moe_combine": [P, I64, I32, P, P, I32, I32, I32, I32, P, I64, P, I64, I32, P],
            "ft_moe_combine_backward": [P, I64, I32, P, I64, I32, P, P, I32, I32, I32, I32, P, I64, P, P],
            "ft_moe_rmsnorm": [P, I64, P, I64, P, I64, I32, P, I32, F32, F32, I32, I32, P, I64, P, I64, P, I64, P, P],
            "ft_moe_rmsnorm_workspace_size": [I32, I32, P],
            "ft_moe_rmsnorm_backward": [P, I64, P, I64, I32, P, I32, F32, P, P, I64, I32, I32, P, I64, P, I32, P, SZ, P],
        }
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.ft_last_error.argtypes = []
        L.ft_last_error.restype = ctypes.c_char_p
        L.ft_moe_launch_count.argtypes = []
        L.ft_moe_launch_count.restype = ctypes.c_int64
        _lib = L
    return _lib


def ft_last_error() -> str:
    return load().ft_last_error().decode()


def _check(status: int):
    if status != 0:
        raise FtMoeError(status, ft_last_error())


def _launchable(stream, dev):
    """Refuses a call on tensors of device `dev` that would not run there: the library launches on the current device, and
    a stream given as a number does not say whose it is (0 is the default stream of every device)."""
    try:
        current = torch._C._cuda_getDevice()
    except RuntimeError:  # no driver on this machine, so that no device is current
        current = dev
    if dev != current:
        raise ValueError(f"the tensors lie on cuda:{dev}, but cuda:{current} is the current device: make theirs current")
    if stream is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"the tensors lie on cuda:{dev}, but the stream belongs to cuda:{stream.device_index}")


def _stream(stream, *tensors):
    """The stream to launch on: the one given, or the current one of the device on which the call's tensors lie."""
    devs = {t.get_device() for t in tensors if isinstance(t, torch.Tensor)} - {-1}
    for dev in devs:
        _launchable(stream, dev)
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(devs.pop()) if devs else 0)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return ctypes.c_void_p(t.data_ptr())
    return ctypes.c_void_p(t.ctypes.data)  # numpy (host pieces)


_DTYPES = {FT_DTYPE_U8: torch.uint8, FT_DTYPE_E4M3: torch.uint8, FT_DTYPE_F32: torch.float32,
           FT_DTYPE_BF16: torch.bfloat16}


def ft_moe_layout(cfg: MoEConfig, shared: int = 0):
    """[(name, shape, torch dtype, bytes)] for the six rank-local banks."""
    specs = (_BankSpec * FT_NBANKS)()
    _check(load().ft_moe_layout(ctypes.byref(cfg), shared, specs))
    return [(BANK_NAMES[i], tuple(specs[i].shape[:specs[i].ndim]), _DTYPES[specs[i].dtype], specs[i].bytes)
            for i in range(FT_NBANKS)]


def alloc_banks(cfg: MoEConfig, shared: int = 0, device="cuda"):
    """Allocate (with torch) the six banks ft_moe_layout describes."""
    return [torch.empty(shape, dtype=dt, device=device) for _, shape, dt, _ in ft_moe_layout(cfg, shared)]


def _banks(tensors):
    if tensors is None:
        return None
    b = _Banks()
    for i, t in enumerate(tensors):
        b.p[i] = t.data_ptr()
    return b


def ft_moe_pack(cfg: MoEConfig, shared: int, pieces: dict, banks, stream=None):
    """Slice full checkpoint-shaped pieces (all host numpy/CPU tensors or all CUDA tensors) into banks."""
    names = ("gate", "gate_scale", "gate_global", "up", "up_scale", "up_global", "down", "down_scale", "down_global")
    vals = [pieces.get(n) for n in names]  # fp8_block pieces have no globals
    given = [v for v in vals if v is not None]
    on_dev = all(isinstance(v, torch.Tensor) and v.is_cuda for v in given)
    if not on_dev:
        vals = [v.numpy() if isinstance(v, torch.Tensor) else v for v in vals]
    for v in vals:
        if v is not None and not (v.is_contiguous() if isinstance(v, torch.Tensor) else v.flags.c_contiguous):
            raise ValueError("pieces must be contiguous")
    p = _Pieces(*[_ptr(v).value if v is not None else None for v in vals], 1 if on_dev else 0)
    _check(load().ft_moe_pack(ctypes.byref(cfg), shared, ctypes.byref(p), ctypes.byref(_banks(banks)),
                              _stream(stream, *banks, *(vals if on_dev else ()))))


def ft_moe_route(logits: torch.Tensor, k: int, topk_ids: torch.Tensor, topk_w: torch.Tensor, stream=None):
    T, E = logits.shape
    _check(load().ft_moe_route(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _stream(stream, logits, topk_ids, topk_w)))


def ft_moe_route_gemm(x: torch.Tensor, w_router: torch.Tensor, k: int, logits: torch.Tensor, topk_ids: torch.Tensor,
                      topk_w: torch.Tensor, stream=None):
    """Router logits = x . w_router^T (bf16 in, fp32 [T, E] out), then the top-k of ft_moe_route."""
    T, H = x.shape
    E = w_router.shape[0]
    _check(load().ft_moe_route_gemm(_ptr(x), T, H, _ptr(w_router), E, k, _ptr(logits), _ptr(topk_ids),
                                    _ptr(topk_w), _stream(stream, x, w_router, logits, topk_ids, topk_w)))


def ft_moe_workspace_size(cfg: MoEConfig, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ft_moe_workspace_size(ctypes.byref(cfg), T, ctypes.byref(n)))
    return n.value


def ft_moe_forward(cfg: MoEConfig, routed, shared, x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                   out: torch.Tensor, workspace: torch.Tensor, stream=None):
    """Rank-local partial into `out` (bf16 or fp32 [T, H])."""
    out_dtype = {torch.bfloat16: FT_DTYPE_BF16, torch.float32: FT_DTYPE_F32}[out.dtype]
    rb, sb = _banks(routed), _banks(shared)
    _check(load().ft_moe_forward(ctypes.byref(cfg), ctypes.byref(rb), ctypes.byref(sb) if sb is not None else None,
                                 _ptr(x), x.shape[0], _ptr(topk_ids), _ptr(topk_w), _ptr(out), out_dtype,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream, x, *routed, *(shared or ()), topk_ids, topk_w, out, workspace)))


def ft_moe_workspace_size_w4a4(cfg: MoEConfig, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ft_moe_workspace_size_w4a4(ctypes.byref(cfg), T, ctypes.byref(n)))
    return n.value


def ft_moe_forward_w4a4(cfg: MoEConfig, routed, shared, x: torch.Tensor, topk_ids: torch.Tensor,
                        topk_w: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, stream=None):
    """Rank-local partial with NVFP4 activations (W4A4) into `out` (bf16 or fp32 [T, H])."""
    out_dtype = {torch.bfloat16: FT_DTYPE_BF16, torch.float32: FT_DTYPE_F32}[out.dtype]
    rb, sb = _banks(routed), _banks(shared)
    _check(load().ft_moe_forward_w4a4(ctypes.byref(cfg), ctypes.byref(rb),
                                      ctypes.byref(sb) if sb is not None else None, _ptr(x), x.shape[0],
                                      _ptr(topk_ids), _ptr(topk_w), _ptr(out), out_dtype, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream, x, *routed, *(shared or ()), topk_ids, topk_w, out, workspace)))


def ft_moe_quantize_nvfp4(src: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, glob: torch.Tensor,
                          stream=None):
    """NVFP4 codes [rows, K/2], e4m3 scales [rows, K/16] and row scales [rows] of bf16 or fp32 rows."""
    dt = {torch.bfloat16: FT_DTYPE_BF16, torch.float32: FT_DTYPE_F32}[src.dtype]
    rows, K = src.shape
    _check(load().ft_moe_quantize_nvfp4(_ptr(src), dt, rows, K, _ptr(codes), _ptr(scales), _ptr(glob),
                                        _stream(stream, src, codes, scales, glob)))


# A workspace belongs to one call at a time: calls on two streams need one each.
# The expert products and row kernels are short calls: what follows checks what the C call cannot
# see (types, shapes, layouts, and that all tensors lie on the first one's device) and passes plain
# integers.
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_OUT, _E4M3 = (torch.bfloat16, torch.float32), (torch.uint8, torch.float8_e4m3fn)
_U8, _E8M0 = (torch.uint8,), (torch.uint8, torch.float8_e8m0fnu)
_OUT_CODE = {torch.bfloat16: FT_DTYPE_BF16, torch.float32: FT_DTYPE_F32}


def _refuse(name, t, dtypes, shape):
    raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} of shape {tuple(shape)} with contiguous "
                     f"elements on the first operand's device, got {t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


def _rows(name, t, dev, dtypes, rows, cols):
    """Row stride of a [rows, cols] tensor whose rows are contiguous (a single row's does not matter)."""
    if t.dtype not in dtypes or t.shape != (rows, cols) or t.get_device() != dev:
        _refuse(name, t, dtypes, (rows, cols))
    ld, step = t.stride()
    if step != 1 and cols > 1:
        _refuse(name, t, dtypes, (rows, cols))
    return ld if rows > 1 else cols


def _whole(name, t, dev, dtypes, shape):
    """Address of a contiguous tensor of the given shape (None, where it may be left out, stays None)."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _refuse(name, t, dtypes, shape)
    return t.data_ptr()


def _scratch(t, dev):
    """Address and bytes of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on the first operand's device, got strides "
                         f"{t.stride()} on {t.device}")
    return t.data_ptr(), t.nbytes


def _dims(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name}: expected {n} dimensions, got {tuple(t.shape)}")
    return t.shape


def _stream_of(stream, dev):
    """The stream to launch on, as an integer: the one given, or the device's current one."""
    if dev < 0:
        raise ValueError("expected tensors on the GPU")
    _launchable(stream, dev)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _offsets(offs, dev, E):
    if offs is None and E != 1:
        raise ValueError("offs may be None for one expert only")
    return _whole("offs", offs, dev, _I32, (E + 1,))


def ft_moe_group_workspace_size(E: int, P: int, N: int, K: int) -> int:
    n = ctypes.c_size_t()
    status = (_lib or load()).ft_moe_group_workspace_size(E, P, N, K, ctypes.byref(n))
    if status:
        _check(status)
    return n.value


def ft_moe_group_gemm(x: torch.Tensor, w: torch.Tensor, offs, y: torch.Tensor, workspace: torch.Tensor, stream=None):
    """y[p] = w[e] . x[p] for the rows p of every expert e (w bf16 [E, N, K]; y bf16 or fp32)."""
    E, N, K = _dims("w", w, 3)
    P, dev = _dims("x", x, 2)[0], x.get_device()
    status = (_lib or load()).ft_moe_group_gemm(
        x.data_ptr(), _rows("x", x, dev, _BF16, P, K), _whole("w", w, dev, _BF16, (E, N, K)), _offsets(offs, dev, E), E, P,
        N, K, y.data_ptr(), _rows("y", y, dev, _OUT, P, N), _OUT_CODE[y.dtype], *_scratch(workspace, dev),
        _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_group_gemm_dgrad(dy: torch.Tensor, w: torch.Tensor, offs, dx: torch.Tensor, workspace: torch.Tensor,
                            stream=None):
    """dx[p] = w[e]^T . dy[p]: the gradient of ft_moe_group_gemm's rows (dx bf16 or fp32)."""
    E, N, K = _dims("w", w, 3)
    P, dev = _dims("dy", dy, 2)[0], dy.get_device()
    status = (_lib or load()).ft_moe_group_gemm_dgrad(
        dy.data_ptr(), _rows("dy", dy, dev, _BF16, P, N), _whole("w", w, dev, _BF16, (E, N, K)), _offsets(offs, dev, E), E,
        P, N, K, dx.data_ptr(), _rows("dx", dx, dev, _OUT, P, K), _OUT_CODE[dx.dtype], *_scratch(workspace, dev),
        _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_group_gemm_wgrad(dy: torch.Tensor, x: torch.Tensor, offs, dw: torch.Tensor, workspace: torch.Tensor,
                            accumulate: bool = False, stream=None):
    """dw[e] = sum of dy[p] x[p]^T over expert e's rows (dw bf16 or fp32 [E, N, K]); accumulate adds to an fp32 dw."""
    E, N, K = _dims("dw", dw, 3)
    P, dev = _dims("dy", dy, 2)[0], dy.get_device()
    status = (_lib or load()).ft_moe_group_gemm_wgrad(
        dy.data_ptr(), _rows("dy", dy, dev, _BF16, P, N), x.data_ptr(), _rows("x", x, dev, _BF16, P, K),
        _offsets(offs, dev, E), E, P, N, K, _whole("dw", dw, dev, _OUT, (E, N, K)), _OUT_CODE[dw.dtype],
        1 if accumulate else 0, *_scratch(workspace, dev), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_group_gemm_fp8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, offs,
                          y: torch.Tensor, workspace: torch.Tensor, stream=None):
    """ft_moe_group_gemm on e4m3 codes (uint8 or float8_e4m3fn) with fp32 scales: x_scale [ceil(K/128), P],
    w_scale [E, ceil(N/128), ceil(K/128)]."""
    E, N, K = _dims("w", w, 3)
    P, dev = _dims("x", x, 2)[0], x.get_device()
    nb = (K + 127) // 128
    status = (_lib or load()).ft_moe_group_gemm_fp8(
        x.data_ptr(), _rows("x", x, dev, _E4M3, P, K), x_scale.data_ptr(), _rows("x_scale", x_scale, dev, _F32, nb, P),
        _whole("w", w, dev, _E4M3, (E, N, K)), _whole("w_scale", w_scale, dev, _F32, (E, (N + 127) // 128, nb)),
        _offsets(offs, dev, E), E, P, N, K, y.data_ptr(), _rows("y", y, dev, _OUT, P, N), _OUT_CODE[y.dtype],
        *_scratch(workspace, dev), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_debug_group_plan(product: int, E: int, P: int, N: int, K: int, out_dtype=torch.bfloat16,
                            accumulate: bool = False) -> tuple:
    """(CTAs per tile, tile extent, CTAs per contraction, counted) of the kernel that a grouped product takes."""
    plan = (ctypes.c_int32 * 4)()
    _check(load().ft_moe_debug_group_plan(product, E, P, N, K, _OUT_CODE.get(out_dtype, 0), int(accumulate), plan))
    return tuple(plan)


def ft_moe_quantize_fp8(src: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """e4m3 codes [rows, K] and scales [ceil(K/128), rows] of bf16 or fp32 rows."""
    (rows, K), dev = _dims("src", src, 2), src.get_device()
    status = (_lib or load()).ft_moe_quantize_fp8(
        src.data_ptr(), _OUT_CODE.get(src.dtype, 0), _rows("src", src, dev, _OUT, rows, K), rows, K, codes.data_ptr(),
        _rows("codes", codes, dev, _E4M3, rows, K), scales.data_ptr(),
        _rows("scales", scales, dev, _F32, (K + 127) // 128, rows), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_swiglu(gu: torch.Tensor, w, h: torch.Tensor, stream=None):
    """h = w * silu(gate) * up of rows gu = [gate, up] (w: one fp32 weight per row, or None)."""
    (rows, I), dev = _dims("h", h, 2), gu.get_device()
    status = (_lib or load()).ft_moe_swiglu(
        gu.data_ptr(), _rows("gu", gu, dev, _BF16, rows, 2 * I), _whole("w", w, dev, _F32, (rows,)), rows, I,
        h.data_ptr(), _rows("h", h, dev, _BF16, rows, I), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_swiglu_quantize_fp8(gu: torch.Tensor, w, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """ft_moe_swiglu stored as e4m3 codes [rows, I] and scales [ceil(I/128), rows]."""
    (rows, I), dev = _dims("codes", codes, 2), gu.get_device()
    status = (_lib or load()).ft_moe_swiglu_quantize_fp8(
        gu.data_ptr(), _rows("gu", gu, dev, _BF16, rows, 2 * I), _whole("w", w, dev, _F32, (rows,)), rows, I,
        codes.data_ptr(), _rows("codes", codes, dev, _E4M3, rows, I), scales.data_ptr(),
        _rows("scales", scales, dev, _F32, (I + 127) // 128, rows), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_swiglu_backward(gu: torch.Tensor, w, dh: torch.Tensor, dgu: torch.Tensor, dw=None, stream=None):
    """Gradients of ft_moe_swiglu: dgu = [d gate, d up] and, where dw is given, the row weights'."""
    (rows, I), dev = _dims("dh", dh, 2), gu.get_device()
    status = (_lib or load()).ft_moe_swiglu_backward(
        gu.data_ptr(), _rows("gu", gu, dev, _BF16, rows, 2 * I), _whole("w", w, dev, _F32, (rows,)), dh.data_ptr(),
        _rows("dh", dh, dev, _BF16, rows, I), rows, I, dgu.data_ptr(), _rows("dgu", dgu, dev, _BF16, rows, 2 * I),
        _whole("dw", dw, dev, _F32, (rows,)), _stream_of(stream, dev))
    if status:
        _check(status)


def _opt_rows(name, t, dev, dtypes, rows, cols):
    """Address and row stride of a tensor that may be left out."""
    if t is None:
        return None, 0
    return t.data_ptr(), _rows(name, t, dev, dtypes, rows, cols)


def alloc_mxfp4_scales(rows: int, K: int, device="cuda") -> torch.Tensor:
    """Scales uint8 [ceil(K/128), rows, 4] of MXFP4 rows, with the row stride that ft_moe_group_gemm_mxfp4 needs."""
    return torch.empty(((K + 127) // 128, (rows + 3) // 4 * 4, 4), dtype=torch.uint8, device=device)[:, :rows]


def _words(name, t, dev, rows, K):
    """Address and row stride (in words) of MXFP4 scales [ceil(K/128), rows, 4]."""
    nb = (K + 127) // 128
    if t.dtype not in _E8M0 or t.shape != (nb, rows, 4) or t.get_device() != dev:
        _refuse(name, t, _E8M0, (nb, rows, 4))
    ld, word, byte = t.stride()
    if byte != 1 or (word != 4 and rows > 1) or (ld % 4 and nb > 1):
        raise ValueError(f"{name}: expected words of four bytes, 4 bytes apart in rows a multiple of 4 apart, got strides "
                         f"{t.stride()}")
    return t.data_ptr(), ld // 4 if nb > 1 else (rows + 3) // 4 * 4


def ft_moe_group_gemm_mxfp4(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, offs,
                            y: torch.Tensor, workspace: torch.Tensor, stream=None):
    """ft_moe_group_gemm on MXFP4 operands: codes uint8 x [P, K/2] and w [E, N, K/2]; x_scale uint8
    [ceil(K/128), P, 4] (see alloc_mxfp4_scales), w_scale uint8 [E, ceil(N/128), ceil(K/128), 512]."""
    E, N, half = _dims("w", w, 3)
    P, dev, K = _dims("x", x, 2)[0], x.get_device(), 2 * half
    status = (_lib or load()).ft_moe_group_gemm_mxfp4(
        x.data_ptr(), _rows("x", x, dev, _U8, P, half), *_words("x_scale", x_scale, dev, P, K),
        _whole("w", w, dev, _U8, (E, N, half)),
        _whole("w_scale", w_scale, dev, _U8, (E, (N + 127) // 128, (K + 127) // 128, 512)), _offsets(offs, dev, E), E, P, N, K,
        y.data_ptr(), _rows("y", y, dev, _OUT, P, N), _OUT_CODE[y.dtype], *_scratch(workspace, dev), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_quantize_mxfp4(src: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """MXFP4 codes uint8 [rows, K/2] and scales uint8 [ceil(K/128), rows, 4] of bf16 or fp32 rows."""
    (rows, K), dev = _dims("src", src, 2), src.get_device()
    status = (_lib or load()).ft_moe_quantize_mxfp4(
        src.data_ptr(), _OUT_CODE.get(src.dtype, 0), _rows("src", src, dev, _OUT, rows, K), rows, K, codes.data_ptr(),
        _rows("codes", codes, dev, _U8, rows, K // 2), *_words("scales", scales, dev, rows, K), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_quantize_mxfp4_weights(src: torch.Tensor, codes: torch.Tensor, tiles: torch.Tensor, stream=None):
    """MXFP4 codes uint8 [E, N, K/2] and scale tiles uint8 [E, ceil(N/128), ceil(K/128), 512] of bf16 or fp32
    weights [E, N, K]."""
    (E, N, K), dev = _dims("src", src, 3), src.get_device()
    status = (_lib or load()).ft_moe_quantize_mxfp4_weights(
        _whole("src", src, dev, _OUT, (E, N, K)), _OUT_CODE.get(src.dtype, 0), E, N, K,
        _whole("codes", codes, dev, _U8, (E, N, K // 2)),
        _whole("tiles", tiles, dev, _U8, (E, (N + 127) // 128, (K + 127) // 128, 512)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_pack_mxfp4_scales(src: torch.Tensor, tiles: torch.Tensor, stream=None):
    """Scale tiles uint8 [E, ceil(N/128), ceil(K/128), 512] of a checkpoint's scale bytes [E, N, K/32]."""
    (E, N, blocks), dev = _dims("src", src, 3), src.get_device()
    status = (_lib or load()).ft_moe_pack_mxfp4_scales(
        _whole("src", src, dev, _E8M0, (E, N, blocks)), E, N, 32 * blocks,
        _whole("tiles", tiles, dev, _U8, (E, (N + 127) // 128, (blocks + 3) // 4, 512)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_swiglu_quantize_mxfp4(gu: torch.Tensor, w, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """ft_moe_swiglu stored as MXFP4 codes uint8 [rows, I/2] and scales uint8 [ceil(I/128), rows, 4]."""
    (rows, half), dev = _dims("codes", codes, 2), gu.get_device()
    I = 2 * half
    status = (_lib or load()).ft_moe_swiglu_quantize_mxfp4(
        gu.data_ptr(), _rows("gu", gu, dev, _BF16, rows, 2 * I), _whole("w", w, dev, _F32, (rows,)), rows, I,
        codes.data_ptr(), _rows("codes", codes, dev, _U8, rows, half), *_words("scales", scales, dev, rows, I),
        _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_dispatch(x: torch.Tensor, slot: torch.Tensor, k: int, out: torch.Tensor, x_scale=None, out_scale=None, w=None,
                    row_w=None, pos=None, count=None, stream=None):
    """out[p] = x[slot[p] // k] (rows of any type), with block scales ([blocks, T] to [blocks, P], fp32, or
    [blocks, T, 4] to [blocks, P, 4], uint8), row weights (w fp32 [T, k] to row_w [P]) and pos int32 [T, k], the rows of
    the slots. count int32 [1]: rows in use."""
    (T, cols), dev, size = _dims("x", x, 2), x.get_device(), x.element_size()
    P = _dims("slot", slot, 1)[0]
    blocks, xs, os_ = 0, (None, 0), (None, 0)
    if (x_scale is None) != (out_scale is None) or (w is None) != (row_w is None):
        raise ValueError("x_scale and out_scale, and w and row_w, are given together")
    if x_scale is not None:
        blocks = x_scale.shape[0]
        if x_scale.dim() == 3:
            xs, os_ = _words("x_scale", x_scale, dev, T, 128 * blocks), _words("out_scale", out_scale, dev, P, 128 * blocks)
        else:
            xs = x_scale.data_ptr(), _rows("x_scale", x_scale, dev, _F32, blocks, T)
            os_ = out_scale.data_ptr(), _rows("out_scale", out_scale, dev, _F32, blocks, P)
    status = (_lib or load()).ft_moe_dispatch(
        x.data_ptr(), _rows("x", x, dev, (x.dtype,), T, cols) * size, cols * size, T, k,
        _whole("slot", slot, dev, _I32, (P,)), P, _whole("count", count, dev, _I32, (1,)), out.data_ptr(),
        _rows("out", out, dev, (x.dtype,), P, cols) * size, *xs, blocks, *os_, _whole("w", w, dev, _F32, (T, k)),
        _whole("row_w", row_w, dev, _F32, (P,)), _whole("pos", pos, dev, _I32, (T, k)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_dispatch_backward(dout: torch.Tensor, pos: torch.Tensor, dx: torch.Tensor, drow_w=None, dw=None, stream=None):
    """dx[t] = sum of dout[pos[t, j]] over j (bf16 or fp32 each); dw[t, j] = drow_w[pos[t, j]] where given."""
    (P, H), dev, (T, k) = _dims("dout", dout, 2), dout.get_device(), _dims("pos", pos, 2)
    if (drow_w is None) != (dw is None):
        raise ValueError("drow_w and dw are given together")
    status = (_lib or load()).ft_moe_dispatch_backward(
        dout.data_ptr(), _rows("dout", dout, dev, _OUT, P, H), _OUT_CODE[dout.dtype], _whole("pos", pos, dev, _I32, (T, k)), T, k,
        P, H, _whole("drow_w", drow_w, dev, _F32, (P,)), dx.data_ptr(), _rows("dx", dx, dev, _OUT, T, H), _OUT_CODE[dx.dtype],
        _whole("dw", dw, dev, _F32, (T, k)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_combine(y: torch.Tensor, pos: torch.Tensor, w, out: torch.Tensor, add=None, stream=None):
    """out[t] = sum of w[t, j] * y[pos[t, j]] over j, plus add[t] (of out's type, or None); w fp32 [T, k], None for 1."""
    (P, H), dev, (T, k) = _dims("y", y, 2), y.get_device(), _dims("pos", pos, 2)
    status = (_lib or load()).ft_moe_combine(
        y.data_ptr(), _rows("y", y, dev, _OUT, P, H), _OUT_CODE[y.dtype], _whole("pos", pos, dev, _I32, (T, k)),
        _whole("w", w, dev, _F32, (T, k)), T, k, P, H, *_opt_rows("add", add, dev, (out.dtype,), T, H), out.data_ptr(),
        _rows("out", out, dev, _OUT, T, H), _OUT_CODE[out.dtype], _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_combine_backward(dout: torch.Tensor, y, pos: torch.Tensor, w, dy: torch.Tensor, dw=None, stream=None):
    """dy[pos[t, j]] = w[t, j] * dout[t] (bf16) and, where dw is given, dw[t, j] = <dout[t], y[pos[t, j]]>."""
    (P, H), dev, (T, k) = _dims("dy", dy, 2), dout.get_device(), _dims("pos", pos, 2)
    if y is None and dw is not None:
        raise ValueError("dw needs y")
    status = (_lib or load()).ft_moe_combine_backward(
        dout.data_ptr(), _rows("dout", dout, dev, _OUT, T, H), _OUT_CODE[dout.dtype], *_opt_rows("y", y, dev, _OUT, P, H),
        FT_DTYPE_BF16 if y is None else _OUT_CODE[y.dtype], _whole("pos", pos, dev, _I32, (T, k)),
        _whole("w", w, dev, _F32, (T, k)), T, k, P, H, dy.data_ptr(), _rows("dy", dy, dev, _BF16, P, H),
        _whole("dw", dw, dev, _F32, (T, k)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, y=None, residual=None, total=None, codes=None,
                   scales=None, rstd=None, weight_offset: float = 0.0, stream=None):
    """total = x + residual, y = total / rms(total) * (weight_offset + weight), into y (bf16), into e4m3 codes [rows, H] and
    scales [ceil(H/128), rows], or both; rstd fp32 [rows] for the backward pass."""
    (rows, H), dev = _dims("x", x, 2), x.get_device()
    if (residual is None) != (total is None) or (codes is None) != (scales is None):
        raise ValueError("residual and total, and codes and scales, are given together")
    kind = _BF16 if residual is None else (residual.dtype,)
    status = (_lib or load()).ft_moe_rmsnorm(
        x.data_ptr(), _rows("x", x, dev, _BF16, rows, H), *_opt_rows("residual", residual, dev, _OUT, rows, H),
        *_opt_rows("total", total, dev, kind, rows, H), _OUT_CODE[kind[0]], _whole("weight", weight, dev, _OUT, (H,)),
        _OUT_CODE[weight.dtype], weight_offset, eps, rows, H, *_opt_rows("y", y, dev, _BF16, rows, H),
        *_opt_rows("codes", codes, dev, _E4M3, rows, H), *_opt_rows("scales", scales, dev, _F32, (H + 127) // 128, rows),
        _whole("rstd", rstd, dev, _F32, (rows,)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_rmsnorm_workspace_size(rows: int, H: int) -> int:
    n = ctypes.c_size_t()
    status = (_lib or load()).ft_moe_rmsnorm_workspace_size(rows, H, ctypes.byref(n))
    if status:
        _check(status)
    return n.value


def ft_moe_rmsnorm_backward(dy: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                            workspace=None, dw=None, dtotal=None, weight_offset: float = 0.0, accumulate: bool = False,
                            stream=None):
    """Gradients of ft_moe_rmsnorm: dx (of total's type, for x and the residual; dtotal reaches total past the norm) and,
    where given, dw fp32 [H] (which needs the workspace; accumulate adds to it)."""
    (rows, H), dev = _dims("dy", dy, 2), dy.get_device()
    kind = (total.dtype,)
    status = (_lib or load()).ft_moe_rmsnorm_backward(
        dy.data_ptr(), _rows("dy", dy, dev, _BF16, rows, H), total.data_ptr(), _rows("total", total, dev, _OUT, rows, H),
        _OUT_CODE[total.dtype], _whole("weight", weight, dev, _OUT, (H,)), _OUT_CODE[weight.dtype], weight_offset,
        _whole("rstd", rstd, dev, _F32, (rows,)), *_opt_rows("dtotal", dtotal, dev, kind, rows, H), rows, H, dx.data_ptr(),
        _rows("dx", dx, dev, kind, rows, H), _whole("dw", dw, dev, _F32, (H,)), 1 if accumulate else 0,
        *((None, 0) if workspace is None else _scratch(workspace, dev)), _stream_of(stream, dev))
    if status:
        _check(status)


def ft_moe_align_workspace_size(T: int, k: int, E: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ft_moe_align_workspace_size(T, k, E, ctypes.byref(n)))
    return n.value


def ft_moe_align(topk_ids: torch.Tensor, E: int, block: int, sorted_slot, block_expert, expert_off, n_padded,
                 workspace: torch.Tensor, stream=None):
    T, k = topk_ids.shape
    _check(load().ft_moe_align(_ptr(topk_ids), T, k, E, block, _ptr(sorted_slot), _ptr(block_expert),
                               _ptr(expert_off), _ptr(n_padded), _ptr(workspace),
                               workspace.numel() * workspace.element_size(),
                               _stream(stream, topk_ids, sorted_slot, block_expert, expert_off, n_padded, workspace)))


def ft_moe_dequant(cfg: MoEConfig, shared: int, banks, which: int, expert: int, out: torch.Tensor, stream=None):
    _check(load().ft_moe_dequant(ctypes.byref(cfg), shared, ctypes.byref(_banks(banks)), which, expert, _ptr(out),
                                 _stream(stream, out, *banks)))


def ft_moe_set_stage_events(events):
    """Arm per-stage timing of the next ft_moe_forward on this thread (FT_NSTAGES + 1 torch.cuda.Event)."""
    if events is None:
        _check(load().ft_moe_set_stage_events(None))
        return
    arr = (ctypes.c_void_p * (FT_NSTAGES + 1))(*[ev.cuda_event for ev in events])
    _check(load().ft_moe_set_stage_events(arr))


def ft_moe_debug_inject_stall(wait_limit_ns: int, skip_producer: int):
    """Arm fault injection for the next ft_moe_forward on this thread (see ft_moe.h)."""
    _check(load().ft_moe_debug_inject_stall(wait_limit_ns, skip_producer))


def ft_moe_launch_count() -> int:
    return int(load().ft_moe_launch_count())


def ft_moe_read_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and return the device status word (0 = FT_OK)."""
    return load().ft_moe_read_status(_ptr(workspace), _stream(stream, workspace))

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
    "FT_GROUP_DGRAD", "FT_GROUP_WGRAD", "FT_GROUP_FP8",
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
           "ft_moe_swiglu_backward", "ft_moe_debug_group_plan")
FT_GROUP_FORWARD, FT_GROUP_DGRAD, FT_GROUP_WGRAD, FT_GROUP_FP8 = range(4)
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


def _stream(stream, *tensors):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)
    return ctypes.c_void_p(0)


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
                              _stream(stream, *banks)))


def ft_moe_route(logits: torch.Tensor, k: int, topk_ids: torch.Tensor, topk_w: torch.Tensor, stream=None):
    T, E = logits.shape
    _check(load().ft_moe_route(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _stream(stream, logits)))


def ft_moe_route_gemm(x: torch.Tensor, w_router: torch.Tensor, k: int, logits: torch.Tensor, topk_ids: torch.Tensor,
                      topk_w: torch.Tensor, stream=None):
    """Router logits = x . w_router^T (bf16 in, fp32 [T, E] out), then the top-k of ft_moe_route."""
    T, H = x.shape
    E = w_router.shape[0]
    _check(load().ft_moe_route_gemm(_ptr(x), T, H, _ptr(w_router), E, k, _ptr(logits), _ptr(topk_ids),
                                    _ptr(topk_w), _stream(stream, x)))


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
                                 _stream(stream, x)))


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
                                      workspace.numel() * workspace.element_size(), _stream(stream, x)))


def ft_moe_quantize_nvfp4(src: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, glob: torch.Tensor,
                          stream=None):
    """NVFP4 codes [rows, K/2], e4m3 scales [rows, K/16] and row scales [rows] of bf16 or fp32 rows."""
    dt = {torch.bfloat16: FT_DTYPE_BF16, torch.float32: FT_DTYPE_F32}[src.dtype]
    rows, K = src.shape
    _check(load().ft_moe_quantize_nvfp4(_ptr(src), dt, rows, K, _ptr(codes), _ptr(scales), _ptr(glob),
                                        _stream(stream, src)))


# A workspace belongs to one call at a time: calls on two streams need one each.
# The expert products and row kernels are short calls: what follows checks what the C call cannot
# see (types, shapes, layouts, and that all tensors lie on the first one's device) and passes plain
# integers.
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_OUT, _E4M3 = (torch.bfloat16, torch.float32), (torch.uint8, torch.float8_e4m3fn)
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
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch._C._cuda_getCurrentRawStream(dev)


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


def ft_moe_align_workspace_size(T: int, k: int, E: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ft_moe_align_workspace_size(T, k, E, ctypes.byref(n)))
    return n.value


def ft_moe_align(topk_ids: torch.Tensor, E: int, block: int, sorted_slot, block_expert, expert_off, n_padded,
                 workspace: torch.Tensor, stream=None):
    T, k = topk_ids.shape
    _check(load().ft_moe_align(_ptr(topk_ids), T, k, E, block, _ptr(sorted_slot), _ptr(block_expert),
                               _ptr(expert_off), _ptr(n_padded), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream, topk_ids)))


def ft_moe_dequant(cfg: MoEConfig, shared: int, banks, which: int, expert: int, out: torch.Tensor, stream=None):
    _check(load().ft_moe_dequant(ctypes.byref(cfg), shared, ctypes.byref(_banks(banks)), which, expert, _ptr(out),
                                 _stream(stream, out)))


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

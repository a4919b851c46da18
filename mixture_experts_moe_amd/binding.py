"""ctypes binding of the fused MoE C ABI (include/moe.h).

Argument marshalling only: every function takes torch tensors, checks their
shapes, dtypes and devices, and calls the C entry point of the same name with
raw device pointers and a HIP stream (the one given, else torch's current
stream of the tensors' device).  Tensors the binding allocates (outputs,
workspace) are allocated on that stream, so torch's caching allocator only
reuses their memory for work ordered after these kernels.  All computation happens in
the HIP kernels of ``libmoe.so``; there is no fallback of any kind, and if
the library is missing the first call raises.  No call is recorded by torch's
autograd: results never require a gradient, whatever the inputs do, and the
gradients that there are (``*_backward``) are calls of their own.
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

# MOE_LIBRARY may name another build of the same library (e.g. a tuning variant).
_LIB_PATH = os.environ.get("MOE_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_E4M3FN = 2
MOE_DTYPE_I8 = 3
MOE_SCALE_NONE = 0
MOE_SCALE_PER_TENSOR = 1
MOE_SCALE_PER_CHANNEL = 2
MOE_ACT_AS_IS = 0
MOE_ACT_MX_E4M3 = 1
MOE_SCHED_AUTO = 0
MOE_SCHED_STATIC = 1
MOE_SCHED_QUEUE = 2
MOE_KERNEL_COUNT = 8

ENTRY_POINTS = (
    "moe_align_capacity", "moe_workspace_bytes", "moe_forward", "moe_route",
    "moe_route_logits", "moe_align", "moe_route_align", "moe_expert_ffn",
    "moe_quantize_act", "moe_graph_create", "moe_graph_launch", "moe_graph_destroy", "moe_strerror",
    "moe_timing_enable", "moe_timing_collect", "moe_kernel_name", "moe_forward_noalloc",
    "moe_linear_workspace_bytes", "moe_linear", "moe_decode_workspace_bytes", "moe_decode",
    "moe_rmsnorm", "moe_rmsnorm_backward_workspace_bytes", "moe_rmsnorm_backward",
    "moe_quantize_i8", "moe_linear_i8_workspace_bytes", "moe_linear_i8",
    "moe_permute_workspace_bytes", "moe_permute", "moe_unpermute", "moe_unpermute_backward",
)
MOE_ERR_NOALLOC_SIZE = -10
MOE_ERR_OVERLAP = -11
MOE_NOALLOC_WORKSPACE_BYTES = 64 << 20
MOE_DECODE_MAX_TOKENS = 16


class moe_desc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("num_experts", ctypes.c_int64), ("intermediate", ctypes.c_int64),
                ("act_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("block_m", ctypes.c_int32), ("act_quant", ctypes.c_int32),
                ("schedule", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class moe_scales(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p)]


class moe_linear_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("out_features", ctypes.c_int64),
                ("in_features", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64),
                ("ldr", ctypes.c_int64), ("ldo", ctypes.c_int64), ("act_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("fn", ctypes.c_int32), ("gated", ctypes.c_int32),
                ("scale_mode", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class moe_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("ldr", ctypes.c_int64), ("ldsum", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("ldc", ctypes.c_int64), ("eps", ctypes.c_float), ("act_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class moe_linear_i8_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("out_features", ctypes.c_int64),
                ("in_features", ctypes.c_int64), ("num_groups", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("ldo", ctypes.c_int64), ("out_dtype", ctypes.c_int32), ("fn", ctypes.c_int32),
                ("gated", ctypes.c_int32), ("scale_mode", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class moe_permute_desc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("num_experts", ctypes.c_int64), ("num_rows", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldres", ctypes.c_int64),
                ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {strerror(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run `python -m mixture_experts_moe_amd.build`")
    L = ctypes.CDLL(_LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(moe_desc)
    S = ctypes.POINTER(moe_scales)
    LD = ctypes.POINTER(moe_linear_desc)
    ND, PD = ctypes.POINTER(moe_norm_desc), ctypes.POINTER(moe_permute_desc)
    L8 = ctypes.POINTER(moe_linear_i8_desc)
    sig = {
        "moe_align_capacity": (I32, [D, I32, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(I64)]),
        "moe_workspace_bytes": (I32, [D, I32, I32, ctypes.POINTER(SZ)]),
        "moe_forward": (I32, [D, P, P, P, P, I32, S, P, P, SZ, P]),
        "moe_forward_noalloc": (I32, [D, P, P, P, P, I32, S, P, P]),
        "moe_route": (I32, [D, P, P, I32, P, P, P, P]),
        "moe_route_logits": (I32, [D, P, I32, P, P, P]),
        "moe_align": (I32, [D, P, I32, P, P, P, P, P]),
        "moe_route_align": (I32, [D, P, P, I32, P, P, P, P, P, P, P, P]),
        "moe_graph_create": (I32, [D, P, P, P, P, I32, S, P, P, SZ, ctypes.POINTER(P)]),
        "moe_graph_launch": (I32, [P, P]),
        "moe_graph_destroy": (I32, [P]),
        "moe_expert_ffn": (I32, [D, P, P, P, I32, S, P, P, P, P, P, P, SZ, P]),
        "moe_quantize_act": (I32, [D, P, P, P, P]),
        "moe_decode_workspace_bytes": (I32, [D, I32, ctypes.POINTER(SZ)]),
        "moe_decode": (I32, [D, P, P, P, P, I32, S, P, P, P, SZ, P]),
        "moe_linear_workspace_bytes": (I32, [LD, ctypes.POINTER(SZ)]),
        "moe_linear": (I32, [LD, P, P, P, P, P, P, P, SZ, P]),
        "moe_rmsnorm": (I32, [ND, P, P, P, P, P, P, P, P]),
        "moe_rmsnorm_backward_workspace_bytes": (I32, [ND, ctypes.POINTER(SZ)]),
        "moe_rmsnorm_backward": (I32, [ND, P, P, P, P, P, P, P, SZ, P]),
        "moe_quantize_i8": (I32, [ND, P, P, P, P]),
        "moe_linear_i8_workspace_bytes": (I32, [L8, ctypes.POINTER(SZ)]),
        "moe_linear_i8": (I32, [L8, P, P, P, P, P, P, P, P, P, SZ, P]),
        "moe_permute_workspace_bytes": (I32, [PD, ctypes.POINTER(SZ)]),
        "moe_permute": (I32, [PD, P, P, P, P, P, P, P, P, P, SZ, P]),
        "moe_unpermute": (I32, [PD, P, P, P, P, P, P]),
        "moe_unpermute_backward": (I32, [PD, P, P, P, P, P, P, P]),
        "moe_strerror": (ctypes.c_char_p, [I32]),
        "moe_timing_enable": (I32, [I32]),
        "moe_timing_collect": (I32, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64), I32]),
        "moe_kernel_name": (ctypes.c_char_p, [I32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


# ------------------------------------------------------------ attainable-rate probes

BENCH_ENTRY_POINTS = ("moe_bench_hbm_read", "moe_bench_mfma_bf16", "moe_bench_mfma_fp8",
                      "moe_bench_fp8_dot")
_BENCH_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_bench.so")
_bench_lib = None


def bench_lib() -> ctypes.CDLL:
    """Load libmoe_bench.so (once).  Raises if it has not been built."""
    global _bench_lib
    if _bench_lib is not None:
        return _bench_lib
    if not os.path.exists(_BENCH_LIB_PATH):
        raise RuntimeError(f"{_BENCH_LIB_PATH} is not built; run `python -m mixture_experts_moe_amd.build`")
    L = ctypes.CDLL(_BENCH_LIB_PATH)
    P, I32, SZ, D = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(ctypes.c_double)
    L.moe_bench_hbm_read.restype = I32
    L.moe_bench_hbm_read.argtypes = [P, SZ, I32, D, P]
    L.moe_bench_mfma_bf16.restype = I32
    L.moe_bench_mfma_bf16.argtypes = [I32, I32, D, P]
    L.moe_bench_mfma_fp8.restype = I32
    L.moe_bench_mfma_fp8.argtypes = [I32, I32, D, P]
    L.moe_bench_fp8_dot.restype = I32
    L.moe_bench_fp8_dot.argtypes = [P, P, P, P, I32, P]
    _bench_lib = L
    return L


def bench_hbm_read(buf: torch.Tensor, reps: int = 5, stream=None) -> float:
    """Attainable streaming-read rate (GB/s) over the device buffer `buf`."""
    dev = _dev(buf)
    r = ctypes.c_double()
    _check("moe_bench_hbm_read", bench_lib().moe_bench_hbm_read(
        _ptr(buf), buf.numel() * buf.element_size(), int(reps), ctypes.byref(r),
        _stream(dev, stream)))
    return r.value


def bench_mfma_bf16(iters: int = 4096, reps: int = 4, device="cuda", stream=None) -> float:
    """Attainable bf16 MFMA rate (TFLOP/s) of an LDS-fed loop on random data."""
    dev = torch.device(device)
    r = ctypes.c_double()
    _check("moe_bench_mfma_bf16", bench_lib().moe_bench_mfma_bf16(
        int(iters), int(reps), ctypes.byref(r), _stream(dev, stream)))
    return r.value


def bench_mfma_fp8(iters: int = 4096, reps: int = 4, device="cuda", stream=None) -> float:
    """Attainable e4m3fn (block-scaled) MFMA rate (TFLOP/s) of the W8A8 tile's
    LDS-fed loop on random codes."""
    dev = torch.device(device)
    r = ctypes.c_double()
    _check("moe_bench_mfma_fp8", bench_lib().moe_bench_mfma_fp8(
        int(iters), int(reps), ctypes.byref(r), _stream(dev, stream)))
    return r.value


def bench_fp8_dot(a: torch.Tensor, b: torch.Tensor, c: torch.Tensor, stream=None) -> torch.Tensor:
    """c[t] + A[t] . B[t] for e4m3fn code rows a, b [n, 128] (uint8) and
    fp32 c [n], as the scaled fp8 MFMA computes it (unit block scales)."""
    dev = _dev(a, b, c)
    if a.dtype != torch.uint8 or b.dtype != torch.uint8 or c.dtype != torch.float32:
        raise TypeError("a, b must be uint8 codes and c float32")
    n = a.shape[0]
    if tuple(a.shape) != (n, 128) or tuple(b.shape) != (n, 128) or tuple(c.shape) != (n,):
        raise ValueError("a, b must be [n, 128] and c [n]")
    out = torch.empty((n, 256), dtype=torch.float32, device=dev)
    _check("moe_bench_fp8_dot", bench_lib().moe_bench_fp8_dot(
        _ptr(a), _ptr(b), _ptr(c), _ptr(out), int(n), _stream(dev, stream)))
    if not bool((out == out[:, :1]).all()):
        raise RuntimeError("moe_bench_fp8_dot: the tile's 256 outputs differ")
    return out[:, 0].contiguous()


def strerror(status: int) -> str:
    return lib().moe_strerror(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MoEError(fn, status)


# ------------------------------------------------------------ marshalling

def _act_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return MOE_DTYPE_BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")


def _w_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return MOE_DTYPE_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MOE_DTYPE_E4M3FN
    raise TypeError(f"weights must be float32, bfloat16 or e4m3fn bytes, got {t.dtype}")


def _act_quant_code(act_quant: Optional[str]) -> int:
    if act_quant is None:
        return MOE_ACT_AS_IS
    if act_quant == "mx_e4m3":
        return MOE_ACT_MX_E4M3
    raise ValueError(f"act_quant must be None or 'mx_e4m3', got {act_quant!r}")


_SCHEDULES = {"auto": MOE_SCHED_AUTO, "static": MOE_SCHED_STATIC, "queue": MOE_SCHED_QUEUE}


def _schedule_code(schedule: str) -> int:
    if schedule not in _SCHEDULES:
        raise ValueError(f"schedule must be one of {sorted(_SCHEDULES)}, got {schedule!r}")
    return _SCHEDULES[schedule]


def make_desc(T: int, d: int, E: int, I: int, act_dtype: int, weight_dtype: int,
              block_m: int = 0, act_quant: Optional[str] = None,
              schedule: str = "auto") -> moe_desc:
    return moe_desc(int(T), int(d), int(E), int(I), int(act_dtype), int(weight_dtype),
                    int(block_m), _act_quant_code(act_quant), _schedule_code(schedule), 0)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(*ts: Optional[torch.Tensor]) -> torch.device:
    dev = None
    for t in ts:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError("all tensors must be on the GPU")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on one device")
    return dev


def _stream(dev: torch.device, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return ctypes.c_void_p(s.cuda_stream)


def _scales(w13: torch.Tensor, scales) -> Optional[moe_scales]:
    if _w_code(w13) != MOE_DTYPE_E4M3FN:
        if scales is not None:
            raise ValueError("scales are only for e4m3fn weights")
        return None
    if scales is None:
        raise ValueError("e4m3fn weights need (s13, s2) scales")
    s13, s2 = scales
    if s13.dtype != torch.float32 or s2.dtype != torch.float32:
        raise TypeError("scales must be float32")
    if _dev(w13, s13, s2) != w13.device:
        raise ValueError("scales must be on the weights' device")
    E, two_i, d = w13.shape
    if s13.dim() == 2:
        mode = MOE_SCALE_PER_CHANNEL
        if tuple(s13.shape) != (E, two_i) or tuple(s2.shape) != (E, d):
            raise ValueError(f"per-channel scales must be [{E}, {two_i}] and [{E}, {d}]")
    else:
        mode = MOE_SCALE_PER_TENSOR
        if tuple(s13.shape) != (E,) or tuple(s2.shape) != (E,):
            raise ValueError(f"per-tensor scales must be [{E}] and [{E}]")
    return moe_scales(mode, 0, s13.data_ptr(), s2.data_ptr())


def _shapes(x, w_gate, w13, w2):
    """(T, d, E, I) from the tensors' shapes; raises before any launch when
    shapes or dtypes do not fit together (metadata only: no device access)."""
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], got shape {tuple(x.shape)}")
    T, d = x.shape
    if w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("w13 must be [E, 2I, d] and w2 [E, d, I]")
    if _w_code(w2) != _w_code(w13) or w2.element_size() != w13.element_size():
        raise TypeError(f"w13 and w2 must have one weight format, got {w13.dtype} and {w2.dtype}")
    E, twoI, d13 = w13.shape
    I = twoI // 2
    if d13 != d or twoI != 2 * I or tuple(w2.shape) != (E, d, I):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w13 {tuple(w13.shape)}, w2 {tuple(w2.shape)}")
    if w_gate is not None:
        if w_gate.dtype != torch.float32 or tuple(w_gate.shape) != (E, d):
            raise ValueError(f"w_gate must be float32 [{E}, {d}]")
    return T, d, E, I


def _launch_stream(dev: torch.device, stream=None):
    """The torch stream the kernels are enqueued on."""
    return stream if stream is not None else torch.cuda.current_stream(dev)


def _alloc(shape, dtype, dev, stream) -> torch.Tensor:
    """A new device tensor owned by `stream` in torch's caching allocator, so
    that once it is dropped its memory is only handed to later work on that
    same stream, i.e. after the kernels enqueued here have used it."""
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(nbytes: int, dev, workspace: Optional[torch.Tensor], stream) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return _alloc((max(nbytes, 1),), torch.uint8, dev, stream)


def _check_out(out: torch.Tensor, x: torch.Tensor) -> None:
    if tuple(out.shape) != tuple(x.shape) or out.dtype != x.dtype:
        raise ValueError(f"out must match x in shape and dtype: out {tuple(out.shape)} "
                         f"{out.dtype}, x {tuple(x.shape)} {x.dtype}")


def _check_routing(T: int, top_k: int, topk_w: torch.Tensor, sorted_ids: torch.Tensor,
                   block_expert: torch.Tensor, num_padded: torch.Tensor, cap: int,
                   bm: int) -> None:
    """The routing tensors moe_expert_ffn reads: gates fp32 [T, k], the
    regrouped layout int32 and at least as long as the capacity."""
    if topk_w.dtype != torch.float32 or tuple(topk_w.shape) != (T, top_k):
        raise ValueError(f"topk_w must be float32 [{T}, {top_k}], got {topk_w.dtype} "
                         f"{tuple(topk_w.shape)}")
    for name, t in (("sorted_ids", sorted_ids), ("block_expert", block_expert),
                    ("num_padded", num_padded)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32, got {t.dtype}")
    if sorted_ids.numel() < cap or block_expert.numel() < cap // bm:
        raise ValueError("sorted_ids / block_expert smaller than the layout capacity")
    if num_padded.numel() < 1:
        raise ValueError("num_padded must hold one int32")


# ------------------------------------------------------------ entry points

def moe_align_capacity(desc: moe_desc, top_k: int) -> Tuple[int, int]:
    """(block_m, capacity) of the regrouped layout for `desc`."""
    bm = ctypes.c_int32()
    cap = ctypes.c_int64()
    _check("moe_align_capacity", lib().moe_align_capacity(ctypes.byref(desc), int(top_k),
                                                         ctypes.byref(bm), ctypes.byref(cap)))
    return bm.value, cap.value


def moe_workspace_bytes(desc: moe_desc, top_k: int, with_routing: bool = True) -> int:
    n = ctypes.c_size_t()
    _check("moe_workspace_bytes", lib().moe_workspace_bytes(ctypes.byref(desc), int(top_k),
                                                           int(bool(with_routing)), ctypes.byref(n)))
    return n.value


def moe_forward(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                top_k: int, scales: Optional[Sequence[torch.Tensor]] = None,
                out: Optional[torch.Tensor] = None, *, block_m: int = 0,
                workspace: Optional[torch.Tensor] = None, stream=None,
                act_quant: Optional[str] = None, schedule: str = "auto") -> torch.Tensor:
    """out [T, d] = fused MoE layer of x (same dtype as x).  act_quant="mx_e4m3"
    selects the W8A8 mode (e4m3fn weights; x and h block-scaled e4m3fn);
    schedule ("auto", "static", "queue") how the 128-token-block expert
    kernels hand out their tiles."""
    T, d, E, I = _shapes(x, w_gate, w13, w2)
    if out is not None:
        _check_out(out, x)
    dev = _dev(x, w_gate, w13, w2, out)
    desc = make_desc(T, d, E, I, _act_code(x), _w_code(w13), block_m, act_quant, schedule)
    sc = _scales(w13, scales)
    s = _launch_stream(dev, stream)
    if out is None:
        out = _alloc((T, d), x.dtype, dev, s)
    nbytes = moe_workspace_bytes(desc, top_k, True)
    ws = _workspace(nbytes, dev, workspace, s)
    st = lib().moe_forward(ctypes.byref(desc), _ptr(x), _ptr(w_gate), _ptr(w13), _ptr(w2),
                           int(top_k), ctypes.byref(sc) if sc is not None else None, _ptr(out),
                           _ptr(ws), nbytes, ctypes.c_void_p(s.cuda_stream))
    _check("moe_forward", st)
    return out


def moe_forward_noalloc(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor,
                        w2: torch.Tensor, top_k: int, out: torch.Tensor,
                        scales: Optional[Sequence[torch.Tensor]] = None, *, block_m: int = 0,
                        stream=None, act_quant: Optional[str] = None,
                        schedule: str = "auto") -> torch.Tensor:
    """moe_forward into the caller's `out` with the library's static
    workspace (the C entry point allocates nothing; nor does this wrapper).
    Raises MoEError (status MOE_ERR_NOALLOC_SIZE) when the layer needs more
    than MOE_NOALLOC_WORKSPACE_BYTES of workspace.  Calls that may overlap on
    one GPU share that workspace and race."""
    T, d, E, I = _shapes(x, w_gate, w13, w2)
    _check_out(out, x)
    dev = _dev(x, w_gate, w13, w2, out)
    desc = make_desc(T, d, E, I, _act_code(x), _w_code(w13), block_m, act_quant, schedule)
    sc = _scales(w13, scales)
    s = _launch_stream(dev, stream)
    st = lib().moe_forward_noalloc(ctypes.byref(desc), _ptr(x), _ptr(w_gate), _ptr(w13),
                                   _ptr(w2), int(top_k),
                                   ctypes.byref(sc) if sc is not None else None, _ptr(out),
                                   ctypes.c_void_p(s.cuda_stream))
    _check("moe_forward_noalloc", st)
    return out


def moe_route(x: torch.Tensor, w_gate: torch.Tensor, top_k: int, *, stream=None):
    """(logits [T,E] fp32, topk_ids [T,k] int32, topk_w [T,k] fp32)."""
    dev = _dev(x, w_gate)
    s = _launch_stream(dev, stream)
    T, d = x.shape
    E = w_gate.shape[0]
    if w_gate.dtype != torch.float32 or w_gate.shape[1] != d:
        raise ValueError("w_gate must be float32 [E, d]")
    desc = make_desc(T, d, E, 64, _act_code(x), _act_code(x))
    logits = _alloc((T, E), torch.float32, dev, s)
    ids = _alloc((T, top_k), torch.int32, dev, s)
    w = _alloc((T, top_k), torch.float32, dev, s)
    _check("moe_route", lib().moe_route(ctypes.byref(desc), _ptr(x), _ptr(w_gate), int(top_k),
                                        _ptr(logits), _ptr(ids), _ptr(w), ctypes.c_void_p(s.cuda_stream)))
    return logits, ids, w


def moe_route_logits(logits: torch.Tensor, top_k: int, *, stream=None):
    """(topk_ids [T,k] int32, topk_w [T,k] fp32) from given fp32 logits [T,E]."""
    dev = _dev(logits)
    s = _launch_stream(dev, stream)
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError("logits must be float32 [T, E]")
    T, E = logits.shape
    desc = make_desc(T, 64, E, 64, MOE_DTYPE_F32, MOE_DTYPE_F32)
    ids = _alloc((T, top_k), torch.int32, dev, s)
    w = _alloc((T, top_k), torch.float32, dev, s)
    _check("moe_route_logits", lib().moe_route_logits(ctypes.byref(desc), _ptr(logits), int(top_k),
                                                      _ptr(ids), _ptr(w), ctypes.c_void_p(s.cuda_stream)))
    return ids, w


def moe_quantize_act(x: torch.Tensor, *, stream=None):
    """W8A8 activation quantisation of bf16 x [T, d]: (codes [T, d] uint8
    e4m3fn bytes, exps [T, d/32] uint8 E8M0 bytes, scale 2^(byte - 127))."""
    dev = _dev(x)
    s = _launch_stream(dev, stream)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be bfloat16 [T, d]")
    T, d = x.shape
    inter = 256
    desc = make_desc(T, d, 1, inter, MOE_DTYPE_BF16, MOE_DTYPE_E4M3FN, 0, "mx_e4m3")
    codes = _alloc((T, d), torch.uint8, dev, s)
    exps = _alloc((T, d // 32), torch.uint8, dev, s)
    _check("moe_quantize_act", lib().moe_quantize_act(ctypes.byref(desc), _ptr(x), _ptr(codes),
                                                      _ptr(exps), ctypes.c_void_p(s.cuda_stream)))
    return codes, exps


def moe_align(topk_ids: torch.Tensor, num_experts: int, *, block_m: int = 0, hidden: int = 64,
              intermediate: int = 64, act_dtype: int = MOE_DTYPE_BF16,
              weight_dtype: int = MOE_DTYPE_BF16, stream=None, act_quant: Optional[str] = None):
    """Regroup slots by expert: (counts [E], sorted_ids [cap], block_expert [cap/B],
    num_padded [1], block_m).  The default block_m depends on the whole
    descriptor, so pass the layer's dims/dtypes/act_quant to get the one
    moe_forward uses."""
    dev = _dev(topk_ids)
    s = _launch_stream(dev, stream)
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be int32 [T, k]")
    T, k = topk_ids.shape
    desc = make_desc(T, hidden, num_experts, intermediate, act_dtype, weight_dtype, block_m,
                     act_quant)
    B, cap = moe_align_capacity(desc, k)
    counts = _alloc(num_experts, torch.int32, dev, s)
    sorted_ids = _alloc(max(cap, 1), torch.int32, dev, s)
    block_expert = _alloc(max(cap // B, 1), torch.int32, dev, s)
    num_padded = _alloc((4,), torch.int32, dev, s)
    _check("moe_align", lib().moe_align(ctypes.byref(desc), _ptr(topk_ids), int(k), _ptr(counts),
                                        _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded),
                                        ctypes.c_void_p(s.cuda_stream)))
    return counts, sorted_ids[:cap], block_expert[:cap // B], num_padded[:1], B


def moe_route_align(x: torch.Tensor, w_gate: torch.Tensor, top_k: int, *, intermediate: int = 64,
                    weight_dtype: int = MOE_DTYPE_BF16, block_m: int = 0, stream=None):
    """Routing then regrouping in one call: (logits, topk_ids, topk_w, counts,
    sorted_ids, block_expert, num_padded, block_m), as moe_route followed by
    moe_align with the same descriptor (pass the layer's intermediate size
    and weight dtype to get the block size moe_forward uses)."""
    dev = _dev(x, w_gate)
    s = _launch_stream(dev, stream)
    T, d = x.shape
    E = w_gate.shape[0]
    if w_gate.dtype != torch.float32 or w_gate.shape[1] != d:
        raise ValueError("w_gate must be float32 [E, d]")
    desc = make_desc(T, d, E, intermediate, _act_code(x), weight_dtype, block_m)
    B, cap = moe_align_capacity(desc, top_k)
    logits = _alloc((T, E), torch.float32, dev, s)
    ids = _alloc((T, top_k), torch.int32, dev, s)
    w = _alloc((T, top_k), torch.float32, dev, s)
    counts = _alloc(E, torch.int32, dev, s)
    sorted_ids = _alloc(max(cap, 1), torch.int32, dev, s)
    block_expert = _alloc(max(cap // B, 1), torch.int32, dev, s)
    num_padded = _alloc((4,), torch.int32, dev, s)
    _check("moe_route_align", lib().moe_route_align(
        ctypes.byref(desc), _ptr(x), _ptr(w_gate), int(top_k), _ptr(logits), _ptr(ids), _ptr(w),
        _ptr(counts), _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded),
        ctypes.c_void_p(s.cuda_stream)))
    return logits, ids, w, counts, sorted_ids[:cap], block_expert[:cap // B], num_padded[:1], B


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _one_gpu(*ts: Optional[torch.Tensor]) -> int:
    """The index of the GPU that holds every tensor given."""
    index = -2  # (get_device() is -1 off the GPU)
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i != index:
            if not t.is_cuda:
                raise ValueError("all tensors must be on the GPU")
            if index >= 0:
                raise ValueError("all tensors must be on one device")
            index = i
    return index


def _allocator(x: torch.Tensor, index: int, stream):
    """(hipStream_t, allocate(shape, dtype=x's)): tensors belong to the launch
    stream, which torch's allocator takes without a stream switch where it is
    the current one of x's device."""
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None or stream.cuda_stream == current:
        return current, x.new_empty
    return stream.cuda_stream, lambda *shape, dtype=x.dtype: _alloc(
        shape if isinstance(shape[0], int) else shape[0], dtype, x.device, stream)


class _Here:
    """No device switch."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(index: int):
    """The tensors' device made current for the launch, where it is not."""
    return _HERE if index == torch._C._cuda_getDevice() else torch.cuda.device(index)


def _ws(workspace: Optional[torch.Tensor], nbytes: int, index: int, new) -> torch.Tensor:
    """The caller's workspace if it will do, or a new one."""
    if workspace is None:
        return new((nbytes,), dtype=torch.uint8)
    if _one_gpu(workspace) != index:
        raise ValueError("workspace must be on the tensors' device")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    return workspace


def moe_decode_workspace_bytes(desc: moe_desc, top_k: int) -> int:
    n = ctypes.c_size_t()
    _check("moe_decode_workspace_bytes",
           lib().moe_decode_workspace_bytes(ctypes.byref(desc), int(top_k), ctypes.byref(n)))
    return n.value


def moe_decode(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
               top_k: int, scales: Optional[Sequence[torch.Tensor]] = None,
               out: Optional[torch.Tensor] = None, *, residual: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None,
               schedule: str = "auto") -> torch.Tensor:
    """out [T, d] = residual + MoE(x) for at most MOE_DECODE_MAX_TOKENS tokens,
    in two launches (moe_forward's layer; other arguments as there).
    residual [T, d] in x's dtype, or None.  out may be the residual, but not
    while that is x: an out that overlaps an input in any other way raises
    MoEError (MOE_ERR_OVERLAP)."""
    T, d, E, I = _shapes(x, w_gate, w13, w2)
    if out is not None:
        _check_out(out, x)
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError(f"residual must match x in shape and dtype: residual "
                         f"{tuple(residual.shape)} {residual.dtype}, x {tuple(x.shape)} {x.dtype}")
    given = (x, w_gate, w13, w2, residual, out)
    index = _one_gpu(*given)
    if not all(t is None or t.is_contiguous() for t in given):
        raise ValueError("all tensors must be contiguous")
    desc = make_desc(T, d, E, I, _act_code(x), _w_code(w13), 0, None, schedule)
    ref = ctypes.byref(desc)
    sc = _scales(w13, scales)
    s, new = _allocator(x, index, stream)
    if out is None:
        out = new((T, d))
    nbytes = ctypes.c_size_t()
    _check("moe_decode_workspace_bytes",
           lib().moe_decode_workspace_bytes(ref, int(top_k), nbytes))
    ws = _ws(workspace, max(nbytes.value, 1), index, new)
    with _on(index):
        _check("moe_decode", lib().moe_decode(
            ref, x.data_ptr(), w_gate.data_ptr(), w13.data_ptr(), w2.data_ptr(), int(top_k),
            ctypes.byref(sc) if sc is not None else None, _addr(residual), out.data_ptr(),
            ws.data_ptr(), nbytes.value, s))
    return out


_FNS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _rows(name: str, t: torch.Tensor, shape) -> int:
    """The row stride of a matrix of the given shape whose rows are dense."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have dense rows, got strides {(ld, step)}")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap: strides {(ld, step)} for {list(shape)}")
    return ld


def moe_linear(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
               activation: Optional[str] = None, gated: bool = False,
               scale: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """out [M, N] = act((x . w^T) * scale + bias) + residual, in x's dtype: the
    dense product beside the experts.  x [M, K] and w [N, K] (or [2N, K] with
    gated=True, gate rows first: act(gate) * up) in one of the layer's dtype
    pairs; activation None, "relu", "silu", "gelu" or "gelu_tanh"; bias fp32
    [rows of w]; scale fp32 [rows of w] or [1], for e4m3fn weights; residual
    and out [M, N].  Rows may be longer in memory than K or N (views of wider
    matrices) and of any length; every tensor starts at a multiple of 16 bytes
    (a slice that does not raises MoEError, MOE_ERR_MISALIGNED).  out may be
    the residual (the same view of it), but not while that is x: an out that
    shares elements with an input in any other way raises MoEError
    (MOE_ERR_OVERLAP)."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [M, K] and w [rows, K]")
    if activation not in _FNS:
        raise ValueError(f"activation must be one of {list(_FNS)}, got {activation!r}")
    M, K = x.shape
    R = w.shape[0]
    if gated and R % 2:
        raise ValueError(f"a gated product needs an even number of weight rows, got {R}")
    N = R // 2 if gated else R
    act, wdt = _act_code(x), _w_code(w)
    ldx, ldw = _rows("x", x, (M, K)), _rows("w", w, (R, K))
    mode = MOE_SCALE_NONE
    if wdt == MOE_DTYPE_E4M3FN:
        if scale is None:
            raise ValueError("e4m3fn weights need a scale")
        if scale.dtype != torch.float32 or tuple(scale.shape) not in ((R,), (1,)):
            raise ValueError(f"scale must be float32 [{R}] or [1]")
        mode = MOE_SCALE_PER_CHANNEL if scale.shape[0] == R else MOE_SCALE_PER_TENSOR
    elif scale is not None:
        raise ValueError("scale is only for e4m3fn weights")
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (R,)):
        raise ValueError(f"bias must be float32 [{R}]")
    ldr = ldo = 0
    if residual is not None:
        if residual.dtype != x.dtype:
            raise TypeError(f"residual must be {x.dtype}, got {residual.dtype}")
        ldr = _rows("residual", residual, (M, N))
    if out is not None:
        if out.dtype != x.dtype:
            raise TypeError(f"out must be {x.dtype}, got {out.dtype}")
        ldo = _rows("out", out, (M, N))
    index = _one_gpu(x, w, scale, bias, residual, out)
    for t in (scale, bias):
        if t is not None and not t.is_contiguous():
            raise ValueError("scale and bias must be contiguous")
    desc = moe_linear_desc(M, N, K, ldx, ldw, ldr, ldo, act, wdt, _FNS[activation],
                           1 if gated else 0, mode, 0)
    ref = ctypes.byref(desc)
    s, new = _allocator(x, index, stream)
    if out is None:
        out = new((M, N))
    nbytes = ctypes.c_size_t()
    _check("moe_linear_workspace_bytes", lib().moe_linear_workspace_bytes(ref, nbytes))
    ws = _ws(workspace, nbytes.value, index, new) if nbytes.value else None
    with _on(index):
        _check("moe_linear", lib().moe_linear(
            ref, x.data_ptr(), w.data_ptr(), _addr(scale), _addr(bias), _addr(residual),
            out.data_ptr(), _addr(ws), nbytes.value, s))
    return out


# ------------------------------------------------------------ norm, 8-bit rows

class RmsNorm(NamedTuple):
    """What moe_rmsnorm returns; None for what was not asked for."""

    y: Optional[torch.Tensor]
    sum: Optional[torch.Tensor]         # x + residual, or x unless y replaced it
    codes: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]


def _vector(name: str, t: torch.Tensor, n: int, dtype=torch.float32) -> None:
    if t.dtype != dtype or tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} [{n}], got {t.dtype} {list(t.shape)}")


def _stride(name: str, t: torch.Tensor, shape) -> int:
    """The row stride of a matrix of the given shape, 0 where its rows are dense."""
    if t.is_contiguous() and t.shape == shape:
        return 0
    return _rows(name, t, shape)


def _result(name: str, t: Optional[torch.Tensor], shape, dtype, new) -> Tuple[torch.Tensor, int]:
    """A result matrix and its row stride: the caller's `t`, or a new one."""
    if t is None:
        return new(*shape, dtype=dtype), 0  # (sizes one by one: 0.2 us less than a tuple)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t, _stride(name, t, shape)


def _result_like(name: str, t: Optional[torch.Tensor], x: torch.Tensor, like) -> Tuple[torch.Tensor, int]:
    """The same for a matrix of x's shape and dtype, a new one from `like` (_like)."""
    if t is None:
        return like(x), 0
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, got {t.dtype}")
    return t, _stride(name, t, x.shape)


def _like(x: torch.Tensor, new):
    """allocate(x, dtype=x's) of x's shape on the launch stream (empty_like takes 0.3 us
    less than new_empty).  new: of _allocator."""
    if new == x.new_empty:
        return torch.empty_like
    return lambda t, dtype=None: new(tuple(t.shape), dtype=dtype or t.dtype)


def _matrix_like(name: str, t: Optional[torch.Tensor], like: torch.Tensor) -> int:
    """The row stride of an input of another's shape and dtype (0 without one)."""
    if t is None:
        return 0
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    return _stride(name, t, like.shape)


_NORM_OUTPUTS = {"y": (True, False), "i8": (False, True), "both": (True, True)}


def moe_rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6, *,
                residual: Optional[torch.Tensor] = None, outputs: str = "y",
                sum_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream=None) -> RmsNorm:
    """Root-mean-square norm of h = x + residual (or of x): y = h / sqrt(mean(h^2)
    + eps) * weight, with x, residual and y [T, d] float32 or bfloat16 and weight
    float32 [d], or None for ones.  outputs: "y"; "i8", int8 codes [T, d] with a
    float32 scale [T] instead (y = codes * scale, scale = max |y| / 127); or
    "both".  Returns RmsNorm(y, sum, codes, scale); sum is h, rounded to x's
    dtype before it is normalised.  sum_out and out take sum and y; each may be
    x or residual itself (the same view of it), which updates it in place; without a
    residual an out that is x leaves no h, and sum is None.  Rows may be longer in
    memory than d; tensors start at multiples of 16 bytes."""
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], got {list(x.shape)}")
    if outputs not in _NORM_OUTPUTS:
        raise ValueError(f"outputs must be one of {list(_NORM_OUTPUTS)}, got {outputs!r}")
    if residual is None and sum_out is not None:
        raise ValueError("sum_out is only for a norm with a residual")
    want_y, want_i8 = _NORM_OUTPUTS[outputs]
    if out is not None and not want_y:
        raise ValueError("out is only for outputs with y")
    T, d = x.shape
    act = _act_code(x)
    ldx, ldr = _stride("x", x, x.shape), _matrix_like("residual", residual, x)
    if weight is not None:
        _vector("weight", weight, d)
    index = _one_gpu(x, weight, residual, sum_out, out)
    s, new = _allocator(x, index, stream)
    like = _like(x, new)
    h = y = codes = scale = None
    ldsum = ldy = 0
    if residual is not None:
        h, ldsum = _result_like("sum_out", sum_out, x, like)
    if want_y:
        y, ldy = _result_like("out", out, x, like)
    if want_i8:
        codes, scale = like(x, dtype=torch.int8), new(T, dtype=torch.float32)
    desc = moe_norm_desc(T, d, ldx, ldr, ldsum, ldy, 0, eps, act, 0)
    with _on(index):
        _check("moe_rmsnorm", lib().moe_rmsnorm(
            ctypes.byref(desc), x.data_ptr(), _addr(residual), _addr(weight), _addr(h), _addr(y),
            _addr(codes), _addr(scale), s))
    if h is None and (out is None or T == 0 or out.data_ptr() != x.data_ptr()):
        h = x
    return RmsNorm(y, h, codes, scale)


def moe_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor],
                         eps: float = 1e-6, *, dsum: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gradient of moe_rmsnorm's y: (dx [T, d], dweight float32 [d], or None
    without a weight).  h is what was normalised (RmsNorm.sum); dx, in h's dtype,
    is the gradient of x and of the residual; dsum [T, d], the gradient that
    reaches sum from elsewhere, is added to it.  out takes dx and may be dy, h
    or dsum itself."""
    if h.dim() != 2:
        raise ValueError(f"h must be [T, d], got {list(h.shape)}")
    T, d = h.shape
    act = _act_code(h)
    ldh = _stride("h", h, h.shape)
    ldy, lds = _matrix_like("dy", dy, h), _matrix_like("dsum", dsum, h)
    if weight is not None:
        _vector("weight", weight, d)
    index = _one_gpu(dy, h, weight, dsum, out)
    s, new = _allocator(h, index, stream)
    dx, ldx = _result_like("out", out, h, _like(h, new))
    dweight = None
    if weight is not None:
        dweight = new(d, dtype=torch.float32)
        if T == 0:
            with torch.cuda.stream(stream or torch.cuda.current_stream(h.device)):
                dweight.zero_()
    desc = moe_norm_desc(T, d, ldx, lds, ldh, ldy, 0, eps, act, 0)
    ref = ctypes.byref(desc)
    nbytes = ctypes.c_size_t()
    _check("moe_rmsnorm_backward_workspace_bytes",
           lib().moe_rmsnorm_backward_workspace_bytes(ref, nbytes))
    ws = _ws(workspace, nbytes.value, index, new) if nbytes.value else None
    with _on(index):
        _check("moe_rmsnorm_backward", lib().moe_rmsnorm_backward(
            ref, dy.data_ptr(), h.data_ptr(), _addr(weight), _addr(dsum), dx.data_ptr(),
            _addr(dweight), _addr(ws), nbytes.value, s))
    return dx, dweight


def moe_quantize_i8(x: torch.Tensor, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes int8 [T, d], scale float32 [T]) of x [T, d] float32 or bfloat16: a
    row of x is about codes * scale, scale = max |x| / 127.  Of activations, or
    of weights [channels, K] with one scale per channel."""
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], got {list(x.shape)}")
    T, d = x.shape
    act = _act_code(x)
    ldx = _stride("x", x, x.shape)
    index = _one_gpu(x)
    s, new = _allocator(x, index, stream)
    codes, scale = _like(x, new)(x, dtype=torch.int8), new(T, dtype=torch.float32)
    desc = moe_norm_desc(T, d, ldx, 0, 0, 0, 0, 0.0, act, 0)
    with _on(index):
        _check("moe_quantize_i8", lib().moe_quantize_i8(
            ctypes.byref(desc), x.data_ptr(), codes.data_ptr(), scale.data_ptr(), s))
    return codes, scale


def moe_linear_i8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                  *, offsets: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  activation: Optional[str] = None, gated: bool = False,
                  residual: Optional[torch.Tensor] = None,
                  out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [M, N] = act((x . w^T) * x_scale * w_scale + bias) + residual for int8
    x [M, K] and w [N, K] (or [2N, K] with gated=True, gate rows first: act(gate)
    * up), float32 x_scale [M] and w_scale [rows of w] or [1]; sums in int32.
    With offsets (int32 [E + 1], as moe_permute writes them) w is [E, rows, K],
    w_scale [E, rows] or [E], bias [E, rows], and rows offsets[e] ..
    offsets[e + 1] - 1 of x meet w[e]; rows of out outside them are left as they
    are (a new out: undefined).  out is out_dtype, float32 or bfloat16; the rest
    as moe_linear."""
    grouped = offsets is not None
    if x.dim() != 2 or w.dim() != (3 if grouped else 2):
        raise ValueError("x must be [M, K] and w [rows, K], or [E, rows, K] with offsets")
    if x.dtype != torch.int8 or w.dtype != torch.int8:
        raise TypeError(f"x and w must be int8, got {x.dtype} and {w.dtype}")
    if activation not in _FNS:
        raise ValueError(f"activation must be one of {list(_FNS)}, got {activation!r}")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    M, K = x.shape
    E, R = (w.shape[0] if grouped else 0), w.shape[-2]
    if gated and R % 2:
        raise ValueError(f"a gated product needs an even number of weight rows, got {R}")
    N = R // 2 if gated else R
    if w.shape[-1] != K:
        raise ValueError(f"w must have rows of {K}, got {list(w.shape)}")
    ldx = _stride("x", x, x.shape)
    if grouped:
        if w.is_contiguous():
            ldw = 0
        elif w.stride(2) != 1 and K > 1 or E > 1 and R > 1 and w.stride(0) != R * w.stride(1):
            raise ValueError(f"w must have dense rows and experts, got strides {w.stride()}")
        else:
            ldw = w.stride(1) if R > 1 else K if E <= 1 else w.stride(0)
            if ldw < K:
                raise ValueError(f"w's rows overlap: strides {w.stride()} for {list(w.shape)}")
        _vector("offsets", offsets, E + 1, torch.int32)
        shapes = ((E, R), (E,))
    else:
        ldw = _stride("w", w, w.shape)
        shapes = ((R,), (1,))
    _vector("x_scale", x_scale, M)
    if w_scale.dtype != torch.float32 or tuple(w_scale.shape) not in shapes:
        raise ValueError(f"w_scale must be float32 {list(shapes[0])} or {list(shapes[1])}")
    mode = MOE_SCALE_PER_CHANNEL if tuple(w_scale.shape) == shapes[0] else MOE_SCALE_PER_TENSOR
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != shapes[0]):
        raise ValueError(f"bias must be float32 {list(shapes[0])}")
    for t in (w_scale, bias):
        if t is not None and not t.is_contiguous():
            raise ValueError("w_scale and bias must be contiguous")
    ldr = 0
    if residual is not None:
        if residual.dtype != out_dtype:
            raise TypeError(f"residual must be {out_dtype}, got {residual.dtype}")
        ldr = _stride("residual", residual, (M, N))
    index = _one_gpu(x, x_scale, w, w_scale, offsets, bias, residual, out)
    s, new = _allocator(x, index, stream)
    out, ldo = _result("out", out, (M, N), out_dtype, new)
    desc = moe_linear_i8_desc(M, N, K, E, ldx, ldw, ldr, ldo,
                              MOE_DTYPE_F32 if out_dtype == torch.float32 else MOE_DTYPE_BF16,
                              _FNS[activation], 1 if gated else 0, mode, 0)
    ref = ctypes.byref(desc)
    nbytes = ctypes.c_size_t()
    _check("moe_linear_i8_workspace_bytes", lib().moe_linear_i8_workspace_bytes(ref, nbytes))
    ws = _ws(workspace, nbytes.value, index, new) if nbytes.value else None
    with _on(index):
        _check("moe_linear_i8", lib().moe_linear_i8(
            ref, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), _addr(bias),
            _addr(offsets), _addr(residual), out.data_ptr(), _addr(ws), nbytes.value, s))
    return out


# ------------------------------------------------------------ tokens sorted by expert

class Permuted(NamedTuple):
    """What moe_permute returns."""

    rows: torch.Tensor                  # [T * top_k, d]
    scale: Optional[torch.Tensor]       # [T * top_k], with 8-bit rows
    offsets: torch.Tensor               # [E + 1]: expert e's rows
    row_slot: torch.Tensor              # [T * top_k]: the slot of each row
    slot_row: torch.Tensor              # [T, top_k]: the row of each slot, or -1


def _rows_code(t: torch.Tensor) -> int:
    return MOE_DTYPE_I8 if t.dtype == torch.int8 else _act_code(t)


def moe_permute(x: torch.Tensor, topk_ids: torch.Tensor, num_experts: int, *,
                scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_scale: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> Permuted:
    """Tokens sorted by expert: a copy of x[t] for every slot (t, j) whose
    topk_ids[t, j] (int32 [T, k], as moe_route writes them) lies in [0,
    num_experts), an expert's slots in ascending order.  x [T, d] float32,
    bfloat16, or int8 with scale float32 [T].  out [T * k, d] and out_scale take
    the rows and their scales; behind the last row both are left as they are (new
    ones: undefined)."""
    if x.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("x must be [T, d] and topk_ids [T, k]")
    T, d = x.shape
    k = topk_ids.shape[1]
    code = _rows_code(x)
    ldx = _stride("x", x, x.shape)
    if topk_ids.dtype != torch.int32 or topk_ids.shape[0] != T or not topk_ids.is_contiguous():
        raise ValueError(f"topk_ids must be contiguous int32 [{T}, k], got {topk_ids.dtype} "
                         f"{list(topk_ids.shape)}")
    if (scale is None) != (out_scale is None) and out_scale is not None:
        raise ValueError("out_scale is only for rows with scales")
    if scale is not None:
        if code != MOE_DTYPE_I8:
            raise ValueError("scale is only for int8 rows")
        _vector("scale", scale, T)
    if out_scale is not None:
        _vector("out_scale", out_scale, T * k)
    index = _one_gpu(x, topk_ids, scale, out, out_scale)
    s, new = _allocator(x, index, stream)
    rows, ldr = _result("out", out, (T * k, d), x.dtype, new)
    if scale is not None and out_scale is None:
        out_scale = new(T * k, dtype=torch.float32)
    n = int(num_experts)
    offsets = new(max(n, 0) + 1, dtype=torch.int32)
    row_slot, slot_row = new(T * k, dtype=torch.int32), _like(x, new)(topk_ids, dtype=torch.int32)
    if T == 0:
        with torch.cuda.stream(stream or torch.cuda.current_stream(x.device)):
            offsets.zero_()
    desc = moe_permute_desc(T, d, n, 0, ldx, ldr, 0, k, code, 0)
    ref = ctypes.byref(desc)
    nbytes = ctypes.c_size_t()
    _check("moe_permute_workspace_bytes", lib().moe_permute_workspace_bytes(ref, nbytes))
    ws = _ws(workspace, nbytes.value, index, new) if nbytes.value else None
    with _on(index):
        _check("moe_permute", lib().moe_permute(
            ref, x.data_ptr(), _addr(scale), topk_ids.data_ptr(), rows.data_ptr(),
            _addr(out_scale), offsets.data_ptr(), row_slot.data_ptr(), slot_row.data_ptr(),
            _addr(ws), nbytes.value, s))
    return Permuted(rows, out_scale, offsets, row_slot, slot_row)


def _slots(slot_row: torch.Tensor, weights: Optional[torch.Tensor]) -> Tuple[int, int]:
    """(T, k) of the slots' rows and weights."""
    if slot_row.dim() != 2 or slot_row.dtype != torch.int32 or not slot_row.is_contiguous():
        raise ValueError(f"slot_row must be contiguous int32 [T, k], got {slot_row.dtype} "
                         f"{list(slot_row.shape)}")
    if weights is not None and (weights.dtype != torch.float32 or weights.shape != slot_row.shape
                                or not weights.is_contiguous()):
        raise ValueError(f"weights must be contiguous float32 {list(slot_row.shape)}, got "
                         f"{weights.dtype} {list(weights.shape)}")
    return slot_row.shape[0], slot_row.shape[1]


def moe_unpermute(rows: torch.Tensor, slot_row: torch.Tensor, *,
                  weights: Optional[torch.Tensor] = None,
                  residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """out [T, d] = residual + sum over j of weights[t, j] * rows[slot_row[t, j]]:
    the way back from moe_permute (slot_row as it wrote it; slots without a row
    add nothing).  rows [n, d] float32 or bfloat16; weights float32 [T, k] (the
    gates), or None for ones, which makes it the gradient of moe_permute's x;
    residual and out [T, d]; out may be the residual itself."""
    if rows.dim() != 2:
        raise ValueError(f"rows must be [n, d], got {list(rows.shape)}")
    T, k = _slots(slot_row, weights)
    n, d = rows.shape
    act = _act_code(rows)
    ldr = _stride("rows", rows, rows.shape)
    ldres = 0
    if residual is not None:
        if residual.dtype != rows.dtype:
            raise TypeError(f"residual must be {rows.dtype}, got {residual.dtype}")
        ldres = _stride("residual", residual, (T, d))
    index = _one_gpu(rows, slot_row, weights, residual, out)
    s, new = _allocator(rows, index, stream)
    out, ldo = _result("out", out, (T, d), rows.dtype, new)
    desc = moe_permute_desc(T, d, 0, n, ldo, ldr, ldres, k, act, 0)
    with _on(index):
        _check("moe_unpermute", lib().moe_unpermute(
            ctypes.byref(desc), rows.data_ptr(), slot_row.data_ptr(), _addr(weights),
            _addr(residual), out.data_ptr(), s))
    return out


def moe_unpermute_backward(dout: torch.Tensor, rows: torch.Tensor, slot_row: torch.Tensor,
                           weights: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradient of moe_unpermute with weights: (drows [n, d] in rows' dtype,
    dweights float32 [T, k]).  dout [T, d], the other arguments as there; the
    residual's gradient is dout itself.  out takes drows and may be rows itself
    where no two slots name one row, as moe_permute writes them; rows that no slot
    names are left as they are (a new drows: undefined)."""
    if rows.dim() != 2:
        raise ValueError(f"rows must be [n, d], got {list(rows.shape)}")
    if weights is None:
        raise ValueError("weights are needed")
    T, k = _slots(slot_row, weights)
    n, d = rows.shape
    act = _act_code(rows)
    ldr = _stride("rows", rows, rows.shape)
    if dout.dtype != rows.dtype:
        raise TypeError(f"dout must be {rows.dtype}, got {dout.dtype}")
    ldo = _stride("dout", dout, (T, d))
    index = _one_gpu(dout, rows, slot_row, weights, out)
    s, new = _allocator(rows, index, stream)
    drows, ldd = _result_like("out", out, rows, _like(rows, new))
    dweights = _like(rows, new)(weights)
    desc = moe_permute_desc(T, d, 0, n, ldo, ldr, ldd, k, act, 0)
    with _on(index):
        _check("moe_unpermute_backward", lib().moe_unpermute_backward(
            ctypes.byref(desc), dout.data_ptr(), rows.data_ptr(), slot_row.data_ptr(),
            weights.data_ptr(), drows.data_ptr(), dweights.data_ptr(), s))
    return drows, dweights


class MoeGraph:
    """moe_forward recorded once into a HIP graph (moe_graph_create) and
    replayed with one launch per call.  Holds references to every buffer it
    was recorded with: write new tokens into `x` in place and call launch()."""

    def __init__(self, x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor,
                 w2: torch.Tensor, top_k: int, scales: Optional[Sequence[torch.Tensor]] = None,
                 out: Optional[torch.Tensor] = None, *, block_m: int = 0,
                 workspace: Optional[torch.Tensor] = None, act_quant: Optional[str] = None,
                 schedule: str = "auto"):
        self._h = None
        T, d, E, I = _shapes(x, w_gate, w13, w2)
        if out is not None:
            _check_out(out, x)
        dev = _dev(x, w_gate, w13, w2, out)
        desc = make_desc(T, d, E, I, _act_code(x), _w_code(w13), block_m, act_quant, schedule)
        self._sc = _scales(w13, scales)
        s = torch.cuda.current_stream(dev)
        own_out = out is None
        if own_out:
            out = _alloc((T, d), x.dtype, dev, s)
        nbytes = moe_workspace_bytes(desc, top_k, True)
        ws = _workspace(nbytes, dev, workspace, s)
        # the graph keeps these addresses: keep the tensors alive with it
        self._keep = (x, w_gate, w13, w2, tuple(scales) if scales is not None else None, ws)
        # tensors allocated here, which a replay on another stream must keep
        # from being reused before it has run
        self._owned = ([ws] if workspace is None else []) + ([out] if own_out else [])
        self.x, self.out, self.device = x, out, dev
        h = ctypes.c_void_p()
        _check("moe_graph_create", lib().moe_graph_create(
            ctypes.byref(desc), _ptr(x), _ptr(w_gate), _ptr(w13), _ptr(w2), int(top_k),
            ctypes.byref(self._sc) if self._sc is not None else None, _ptr(out), _ptr(ws), nbytes,
            ctypes.byref(h)))
        self._h = h

    def launch(self, stream=None) -> torch.Tensor:
        if self._h is None:
            raise RuntimeError("graph already destroyed")
        s = _launch_stream(self.device, stream)
        _check("moe_graph_launch", lib().moe_graph_launch(self._h, ctypes.c_void_p(s.cuda_stream)))
        if s != torch.cuda.current_stream(self.device):
            for t in self._owned:
                t.record_stream(s)
        return self.out

    def close(self) -> None:
        if self._h is not None:
            h, self._h = self._h, None
            _check("moe_graph_destroy", lib().moe_graph_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_expert_ffn(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, top_k: int,
                   topk_w: torch.Tensor, sorted_ids: torch.Tensor, block_expert: torch.Tensor,
                   num_padded: torch.Tensor, scales: Optional[Sequence[torch.Tensor]] = None,
                   out: Optional[torch.Tensor] = None, *, block_m: int = 0,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   act_quant: Optional[str] = None, schedule: str = "auto") -> torch.Tensor:
    """Expert networks + combine for a given routing (layout from moe_align
    with the same block_m and act_quant)."""
    T, d, E, I = _shapes(x, None, w13, w2)
    if out is not None:
        _check_out(out, x)
    desc = make_desc(T, d, E, I, _act_code(x), _w_code(w13), block_m, act_quant, schedule)
    B, cap = moe_align_capacity(desc, top_k)
    _check_routing(T, int(top_k), topk_w, sorted_ids, block_expert, num_padded, cap, B)
    dev = _dev(x, w13, w2, topk_w, sorted_ids, block_expert, num_padded, out)
    sc = _scales(w13, scales)
    s = _launch_stream(dev, stream)
    if out is None:
        out = _alloc((T, d), x.dtype, dev, s)
    nbytes = moe_workspace_bytes(desc, top_k, False)
    ws = _workspace(nbytes, dev, workspace, s)
    st = lib().moe_expert_ffn(ctypes.byref(desc), _ptr(x), _ptr(w13), _ptr(w2), int(top_k),
                              ctypes.byref(sc) if sc is not None else None, _ptr(topk_w),
                              _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded), _ptr(out),
                              _ptr(ws), nbytes, ctypes.c_void_p(s.cuda_stream))
    _check("moe_expert_ffn", st)
    return out


MOE_TIMING_ALL = (1 << MOE_KERNEL_COUNT) - 1
KERNEL_KINDS = {"route_logits": 0, "route_topk": 1, "align": 2, "ffn13": 3, "ffn2": 4, "combine": 5,
                "quant_x": 6, "ffn_fused": 7}


def moe_timing_enable(kinds=True) -> None:
    """Time the given kernel kinds: True = all, False/None = none, or an
    iterable of kind names ("ffn13", ...)."""
    if kinds is True:
        mask = MOE_TIMING_ALL
    elif not kinds:
        mask = 0
    else:
        mask = 0
        for k in kinds:
            mask |= 1 << KERNEL_KINDS[k]
    _check("moe_timing_enable", lib().moe_timing_enable(mask))


def moe_timing_collect(reset: bool = True) -> dict:
    """{kernel name: (total ms, launches)} for the kernels timed so far."""
    ms = (ctypes.c_double * MOE_KERNEL_COUNT)()
    n = (ctypes.c_int64 * MOE_KERNEL_COUNT)()
    _check("moe_timing_collect", lib().moe_timing_collect(ms, n, int(bool(reset))))
    return {moe_kernel_name(i): (ms[i], n[i]) for i in range(MOE_KERNEL_COUNT)}


def moe_kernel_name(kind: int) -> str:
    return lib().moe_kernel_name(int(kind)).decode()

"""ctypes binding of libtdgemm.so (the C ABI in include/tdgemm.h).

Argument marshalling only: every step of the product runs in the library's
HIP kernels.  Tensors give device pointers, shapes and row strides; the
stream is torch's current stream on the operands' device.  There is no CPU
fallback -- a missing library or device raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtdgemm.so")

TDG_OK = 0
TDG_ERR_INVALID_ARG = -1
TDG_ERR_UNSUPPORTED = -2
TDG_ERR_LAUNCH = -3
TDG_ERR_NO_DEVICE = -4
TDG_ERR_SCRATCH = -5
TDG_NOALLOC_SCRATCH_BYTES = 32 << 20

TDG_DTYPE_F16F32 = 0
TDG_DTYPE_I8I32 = 1
TDG_DTYPE_F32F32 = 2

TDG_VARIANT_AUTO = 0
TDG_VARIANT_SINGLE = 1
TDG_VARIANT_REG_PREFETCH = 2
TDG_VARIANT_DIRECT_LDS = 3
TDG_DEBUG_POISON_LDS = 1
TDG_DEBUG_NO_K_ROTATION = 2

VARIANT_NAMES = {0: "auto", 1: "single", 2: "reg_prefetch", 3: "direct_lds"}

TDG_TRANSPOSE_AUTO = 0
TDG_TRANSPOSE_NAIVE = 1
TDG_TRANSPOSE_LDS = 2
TDG_TRANSPOSE_LDS_PADDED = 3
TDG_TRANSPOSE_LDS_SWIZZLED = 4
TDG_TRANSPOSE_VEC = 5

TRANSPOSE_NAMES = {1: "naive", 2: "lds", 3: "lds_padded", 4: "lds_swizzled", 5: "vec"}

# Every symbol include/tdgemm.h declares.
EXPORTED = (
    "gemm_f16f32", "gemm_i8i32", "gemm_f16f32_pipelined", "gemm_i8i32_pipelined",
    "gemm_f16f32_ex", "gemm_i8i32_ex", "gemm_f32f32", "gemm_f32f32_pipelined", "gemm_f32f32_ex",
    "tdg_plan", "tdg_plan_operands", "tdg_tile_figures", "tdg_config_count",
    "tdg_config_at", "tdg_status_string", "tdg_set_debug_flags", "tdg_copy_f32", "tdg_transpose_f32",
    "tdg_mfma_probe", "tdg_mfma_probe_ops", "tdg_mfma_probe_sink_floats", "tdg_lds_probe",
    "tdg_lds_probe_bytes",
    "gemm_f16f32_splitk", "gemm_i8i32_splitk", "gemm_f32f32_splitk", "tdg_splitk_plan",
    "tdg_config_resources", "gemm_splitk_noalloc", "tdg_predict_us",
    "tdg_route_workspace", "tdg_route_plan", "tdg_rows_dispatch", "tdg_rows_combine",
    "tdg_rows_combine_grad", "gemm_f16f32_grouped", "gemm_f16f32_grouped_nt",
    "gemm_f16f32_grouped_tn", "tdg_lora_workspace", "gemm_f16f32_lora",
    "tdg_w4_quantize", "tdg_w4_dequantize", "gemm_f16w4f32", "gemm_f16w4f32_grouped",
    "tdg_expert_layer_workspace", "tdg_expert_layer",
)


class TdgKernelResources(ctypes.Structure):
    _fields_ = [("vgprs", ctypes.c_int), ("spill_bytes", ctypes.c_int), ("lds_bytes", ctypes.c_int),
                ("threads", ctypes.c_int), ("wg_per_cu", ctypes.c_int)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class TdgConfig(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int), ("bn", ctypes.c_int), ("bk", ctypes.c_int),
                ("waves", ctypes.c_int), ("lds_stages", ctypes.c_int), ("variant", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class TdgPlanInfo(ctypes.Structure):
    _fields_ = [("ratio", ctypes.c_double), ("band", ctypes.c_int), ("lds_bytes", ctypes.c_size_t),
                ("wg_per_cu", ctypes.c_int), ("num_tiles", ctypes.c_int64),
                ("grid", ctypes.c_int64), ("est_regs", ctypes.c_int), ("guarded", ctypes.c_int),
                ("need_bytes_per_clk", ctypes.c_double), ("mfma_per_load", ctypes.c_double),
                ("pipelined", ctypes.c_int), ("k_rotated", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class TdgError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libtdgemm.so (built by tiled_dense_gemm_loop_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    # torch ships its own HIP runtime under the same soname
    # (libamdhip64.so.7).  Loading torch first makes this library bind to
    # that one runtime, so device pointers and torch's hipStream_t handles
    # mean the same thing on both sides; loading the library first would put
    # a second HIP runtime into the process.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(path):
        raise ImportError("libtdgemm.so is not built (%s); run __graft_entry__.build() or "
                          "python tiled_dense_gemm_loop_amd/build.py" % path)
    lib = ctypes.CDLL(path)
    i64, vp, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    gemm_args = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    for name in ("gemm_f16f32", "gemm_i8i32", "gemm_f16f32_pipelined", "gemm_i8i32_pipelined",
                 "gemm_f32f32", "gemm_f32f32_pipelined"):
        fn = getattr(lib, name)
        fn.argtypes = gemm_args
        fn.restype = c_int
    for name in ("gemm_f16f32_ex", "gemm_i8i32_ex", "gemm_f32f32_ex"):
        fn = getattr(lib, name)
        fn.argtypes = gemm_args + [ctypes.POINTER(TdgConfig)]
        fn.restype = c_int
    lib.tdg_plan.argtypes = [c_int, i64, i64, i64, ctypes.POINTER(TdgConfig),
                             ctypes.POINTER(TdgPlanInfo)]
    lib.tdg_plan.restype = c_int
    lib.tdg_plan_operands.argtypes = [c_int, i64, i64, i64, ctypes.c_void_p, i64, ctypes.c_void_p, i64,
                                      ctypes.POINTER(TdgConfig), ctypes.POINTER(TdgPlanInfo)]
    lib.tdg_plan_operands.restype = c_int
    lib.tdg_tile_figures.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int, c_int, i64, i64,
                                     i64, ctypes.POINTER(TdgPlanInfo)]
    lib.tdg_tile_figures.restype = c_int
    lib.tdg_config_count.argtypes = [c_int]
    lib.tdg_config_count.restype = c_int
    lib.tdg_config_at.argtypes = [c_int, c_int, ctypes.POINTER(TdgConfig)]
    lib.tdg_config_at.restype = c_int
    lib.tdg_config_resources.argtypes = [c_int, c_int, ctypes.POINTER(TdgKernelResources)]
    lib.tdg_config_resources.restype = c_int
    lib.tdg_status_string.argtypes = [c_int]
    lib.tdg_status_string.restype = ctypes.c_char_p
    lib.tdg_set_debug_flags.argtypes = [c_int]
    lib.tdg_set_debug_flags.restype = c_int
    for name in ("gemm_f16f32_splitk", "gemm_i8i32_splitk", "gemm_f32f32_splitk"):
        fn = getattr(lib, name)
        fn.argtypes = gemm_args[:9] + [c_int, vp, ctypes.c_size_t, vp]
        fn.restype = c_int
    lib.tdg_predict_us.argtypes = [c_int, c_int, c_int, c_int, c_int, i64, i64, i64,
                                   ctypes.POINTER(ctypes.c_double)]
    lib.tdg_predict_us.restype = c_int
    lib.gemm_splitk_noalloc.argtypes = [c_int] + gemm_args[:9] + [c_int, vp]
    lib.gemm_splitk_noalloc.restype = c_int
    lib.tdg_splitk_plan.argtypes = [c_int, i64, i64, i64, ctypes.POINTER(c_int),
                                    ctypes.POINTER(ctypes.c_size_t)]
    lib.tdg_splitk_plan.restype = c_int
    lib.tdg_copy_f32.argtypes = [i64, i64, vp, i64, vp, i64, vp]
    lib.tdg_copy_f32.restype = c_int
    lib.tdg_transpose_f32.argtypes = [c_int, i64, i64, vp, i64, vp, i64, vp]
    lib.tdg_transpose_f32.restype = c_int
    lib.tdg_mfma_probe.argtypes = [c_int, i64, vp, vp]
    lib.tdg_mfma_probe.restype = c_int
    lib.tdg_mfma_probe_ops.argtypes = [c_int, i64]
    lib.tdg_mfma_probe_ops.restype = i64
    lib.tdg_mfma_probe_sink_floats.argtypes = []
    lib.tdg_mfma_probe_sink_floats.restype = i64
    lib.tdg_lds_probe.argtypes = [c_int, i64, vp, vp]
    lib.tdg_lds_probe.restype = c_int
    lib.tdg_lds_probe_bytes.argtypes = [c_int, i64]
    lib.tdg_lds_probe_bytes.restype = i64
    size_p, size_t = ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t
    for name, args in {
        "tdg_route_workspace": [i64] * 3 + [size_p],
        "tdg_route_plan": [i64] * 3 + [vp, i64, vp, vp, vp, vp, size_t, vp],
        "tdg_rows_dispatch": [c_int] + [i64] * 3 + [vp, i64, vp, i64, vp, i64, vp],
        "tdg_rows_combine": [c_int] * 2 + [i64] * 3 + [vp, i64, i64, vp, vp, i64, vp, i64, vp],
        "tdg_rows_combine_grad": [c_int] * 2 + [i64] * 3 + [vp, i64, vp, i64, i64, vp, vp, i64, vp, i64,
                                                            vp, i64, vp],
        "gemm_f16f32_grouped": [i64, vp] + [i64] * 3 + [vp, i64, vp, i64, i64, vp, i64, vp],
        "gemm_f16f32_grouped_nt": [i64, vp] + [i64] * 3 + [vp, i64, vp, i64, i64, vp, i64, vp],
        "gemm_f16f32_grouped_tn": [i64, vp] + [i64] * 3 + [vp, i64, vp, i64, vp, i64, i64, vp],
        "tdg_lora_workspace": [i64] * 5 + [size_p],
        "gemm_f16f32_lora": [i64] * 3 + [vp, i64, vp, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, vp,
                                         i64, vp, size_t, vp],
        "tdg_w4_quantize": [i64] * 4 + [vp, i64, i64] * 4 + [vp],
        "tdg_w4_dequantize": [c_int] + [i64] * 4 + [vp, i64, i64] * 4 + [vp],
        "gemm_f16w4f32": [i64] * 4 + [vp, i64] * 5 + [vp],
        "gemm_f16w4f32_grouped": [i64, vp] + [i64] * 4 + [vp, i64] + [vp, i64, i64] * 3 + [vp, i64, vp],
        "tdg_expert_layer_workspace": [i64] * 5 + [size_p],
        "tdg_expert_layer": [c_int] + [i64] * 5 + [vp, i64] * 3 + [vp, i64, i64] * 2 + [vp, i64, vp, size_t, vp],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().tdg_status_string(status).decode()


# ------------------------------------------------------------------ raw calls

_FNS = {}


def _fn(name: str):
    """The library's entry point `name` (looked up once)."""
    f = _FNS.get(name)
    if f is None:
        f = _FNS[name] = getattr(load_library(), name)
    return f


def call_raw(name: str, M, N, K, a_ptr, lda, b_ptr, ldb, c_ptr, ldc, stream=0, cfg=None) -> int:
    """Call a GEMM entry point with raw device pointers; returns the status."""
    fn = getattr(load_library(), name)
    args = [M, N, K, a_ptr, lda, b_ptr, ldb, c_ptr, ldc, stream]
    if name.endswith("_ex"):
        args.append(ctypes.byref(cfg) if cfg is not None else None)
    return fn(*args)


# -------------------------------------------------------------- torch tensors

def _torch():
    import torch
    return torch


_raw_stream_fn = None


def _stream_handle(device_index: int) -> int:
    """The hipStream_t of torch's current stream on a device.  torch's raw
    query returns the handle directly (~0.1 us); the public
    torch.cuda.current_stream(...).cuda_stream builds a Stream object first
    (~2.7 us per call, most of a small GEMM's host cost), so it is only the
    fallback."""
    global _raw_stream_fn
    torch = _torch()
    if _raw_stream_fn is None:
        fn = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream_fn = fn if fn is not None else (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    return _raw_stream_fn(device_index)


def _matrix(t, dtypes, what):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (what, tuple(shape)))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s; expected one of %s" % (what, t.dtype, dtypes))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % what)
    rows, cols = shape
    if rows == 0 or cols == 0:
        return rows, cols, t.data_ptr(), max(cols, 1)
    st = t.stride()
    if cols > 1 and st[1] != 1:
        raise ValueError("%s: elements within a row must be contiguous" % what)
    ld = st[0] if rows > 1 else cols
    return rows, cols, t.data_ptr(), max(ld, 1)


def _gemm(name, A, B, C, cfg, f16, splitk=None):
    """f16: True (binary16 in), False (int8 in) or "f32" (binary32 in)."""
    torch = _torch()
    if f16 == "f32":
        in_types = (torch.float32,)
    else:
        in_types = (torch.float16, torch.int16) if f16 else (torch.int8,)
    M, K, pa, lda = _matrix(A, in_types, "A")
    K2, N, pb, ldb = _matrix(B, in_types, "B")
    if K != K2:
        raise ValueError("inner dimensions differ: A is %dx%d, B is %dx%d" % (M, K, K2, N))
    if A.device != B.device:
        raise ValueError("A and B are on different devices")
    out_type = torch.float32 if f16 else torch.int32  # "f32" is truthy
    if C is None:
        C = torch.empty((M, N), dtype=out_type, device=A.device)
    Mc, Nc, pc, ldc = _matrix(C, (out_type,), "C")
    if (Mc, Nc) != (M, N):
        raise ValueError("C has shape %s, expected %s" % ((Mc, Nc), (M, N)))
    if C.device != A.device:
        raise ValueError("C is on %s, A and B on %s" % (C.device, A.device))
    fn = _fn(name)
    tail = (ctypes.byref(cfg) if cfg is not None else None,) if name.endswith("_ex") else ()
    mid = ()
    if splitk is not None:  # (parts, workspace tensor or None)
        parts, ws = splitk
        parts = int(parts)
        if parts < 0:
            raise ValueError("parts must be >= 0 (0: the planner's choice), got %d" % parts)
        if ws is None:
            if parts == 0:  # the planner's choice, planned here to size the workspace
                parts, need = tdg_splitk_plan(
                    {"gemm_f16f32_splitk": TDG_DTYPE_F16F32, "gemm_i8i32_splitk": TDG_DTYPE_I8I32,
                     "gemm_f32f32_splitk": TDG_DTYPE_F32F32}[name], M, N, K)
            else:
                need = parts * M * N * 4 if parts > 1 else 0
            # parts == 1 runs the plain product, which needs no workspace
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=A.device) if parts > 1 else None
        elif not ws.is_cuda or ws.device != A.device or not ws.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % A.device)
        mid = (parts, ws.data_ptr() if ws is not None else None,
               ws.numel() * ws.element_size() if ws is not None else 0)
    dev = A.device.index
    cur = torch.cuda.current_device()
    if dev is None or dev == cur:
        rc = fn(M, N, K, pa, lda, pb, ldb, pc, ldc, *mid, _stream_handle(cur), *tail)
    else:
        with torch.cuda.device(A.device):
            rc = fn(M, N, K, pa, lda, pb, ldb, pc, ldc, *mid, _stream_handle(dev), *tail)
    if rc != TDG_OK:
        raise TdgError(rc, name)
    return C


def _cfg(cfg):
    if cfg is None or isinstance(cfg, TdgConfig):
        return cfg
    c = TdgConfig()
    for k, v in dict(cfg).items():
        setattr(c, k, int(v))
    return c


def gemm_f16f32(A, B, C=None):
    """Sequential single-buffer baseline: C (float32) = A . B (float16)."""
    return _gemm("gemm_f16f32", A, B, C, None, True)


def gemm_i8i32(A, B, C=None):
    """Sequential single-buffer baseline: C (int32) = A . B (int8)."""
    return _gemm("gemm_i8i32", A, B, C, None, False)


def gemm_f16f32_pipelined(A, B, C=None):
    """Software-pipelined double-buffered K loop, FP16 -> FP32."""
    return _gemm("gemm_f16f32_pipelined", A, B, C, None, True)


def gemm_i8i32_pipelined(A, B, C=None):
    """Software-pipelined double-buffered K loop, INT8 -> INT32."""
    return _gemm("gemm_i8i32_pipelined", A, B, C, None, False)


def gemm_f16f32_ex(A, B, C=None, cfg=None):
    """Explicit configuration (dict or TdgConfig; zero fields are planned)."""
    return _gemm("gemm_f16f32_ex", A, B, C, _cfg(cfg), True)


def gemm_i8i32_ex(A, B, C=None, cfg=None):
    return _gemm("gemm_i8i32_ex", A, B, C, _cfg(cfg), False)


def gemm_f32f32(A, B, C=None):
    """Sequential single-buffer baseline: C (float32) = A . B (float32)."""
    return _gemm("gemm_f32f32", A, B, C, None, "f32")


def gemm_f32f32_pipelined(A, B, C=None):
    """Software-pipelined double-buffered K loop, FP32 -> FP32."""
    return _gemm("gemm_f32f32_pipelined", A, B, C, None, "f32")


def gemm_f32f32_ex(A, B, C=None, cfg=None):
    return _gemm("gemm_f32f32_ex", A, B, C, _cfg(cfg), "f32")


def tdg_plan(dtype: int, M: int, N: int, K: int, cfg=None):
    """(config dict, plan-info dict) the planner picks for this shape."""
    c = _cfg(cfg) or TdgConfig()
    info = TdgPlanInfo()
    rc = load_library().tdg_plan(dtype, M, N, K, ctypes.byref(c), ctypes.byref(info))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_plan")
    return c.as_dict(), info.as_dict()


def tdg_plan_operands(dtype: int, M: int, N: int, K: int, a_addr: int, lda: int, b_addr: int, ldb: int,
                      cfg=None):
    """(config dict, plan-info dict) a call on operands at these addresses
    and leading dimensions would run; the addresses are only compared."""
    c = _cfg(cfg) or TdgConfig()
    info = TdgPlanInfo()
    rc = load_library().tdg_plan_operands(dtype, M, N, K, ctypes.c_void_p(a_addr), lda,
                                          ctypes.c_void_p(b_addr), ldb, ctypes.byref(c), ctypes.byref(info))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_plan_operands")
    return c.as_dict(), info.as_dict()


def tdg_tile_figures(dtype: int, bm: int, bn: int, bk: int, waves: int = 4, stages: int = 1,
                     variant: int = TDG_VARIANT_SINGLE, M: int = 0, N: int = 0, K: int = 0) -> dict:
    """The planner's arithmetic (ratio, band, LDS bytes, WG/CU, ...) for any tile."""
    info = TdgPlanInfo()
    rc = load_library().tdg_tile_figures(dtype, bm, bn, bk, waves, stages, variant, M, N, K,
                                         ctypes.byref(info))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_tile_figures")
    return info.as_dict()


def tdg_predict_us(dtype: int, bm: int, bn: int, waves: int, stages: int, M: int, N: int,
                   K: int) -> float:
    """The planner's predicted kernel time (us) of one measured configuration
    for an M x N x K product."""
    us = ctypes.c_double()
    rc = load_library().tdg_predict_us(dtype, bm, bn, waves, stages, M, N, K, ctypes.byref(us))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_predict_us")
    return us.value


def tdg_splitk_plan(dtype: int, M: int, N: int, K: int):
    """(parts, workspace bytes) the split-K entry points choose for this product."""
    parts, ws = ctypes.c_int(), ctypes.c_size_t()
    rc = load_library().tdg_splitk_plan(dtype, M, N, K, ctypes.byref(parts), ctypes.byref(ws))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_splitk_plan")
    return parts.value, ws.value


def gemm_f16f32_splitk(A, B, C=None, parts: int = 0, workspace=None):
    """C (float32) = A . B (float16) with K split over `parts` (0: planner's
    choice); the workspace is allocated here when not given."""
    return _gemm("gemm_f16f32_splitk", A, B, C, None, True, splitk=(parts, workspace))


def gemm_i8i32_splitk(A, B, C=None, parts: int = 0, workspace=None):
    """C (int32) = A . B (int8) with K split over `parts`; exact."""
    return _gemm("gemm_i8i32_splitk", A, B, C, None, False, splitk=(parts, workspace))


def gemm_f32f32_splitk(A, B, C=None, parts: int = 0, workspace=None):
    """C (float32) = A . B (float32) with K split over `parts`."""
    return _gemm("gemm_f32f32_splitk", A, B, C, None, "f32", splitk=(parts, workspace))


def gemm_splitk_noalloc(A, B, C=None, parts: int = 0):
    """C = A . B with K split over `parts` (0: the planner's count among those
    that fit), the partial products kept in the library's built-in scratch
    array: the library allocates nothing (C is allocated here when not
    given).  The dtype follows A and B: float16 -> float32 C, int8 -> int32,
    float32 -> float32.  Calls that overlap in time on one GPU race on the
    array; calls on one stream do not."""
    torch = _torch()
    dt = {torch.float16: TDG_DTYPE_F16F32, torch.int16: TDG_DTYPE_F16F32,
          torch.int8: TDG_DTYPE_I8I32, torch.float32: TDG_DTYPE_F32F32}.get(A.dtype)
    if dt is None:
        raise TypeError("A has dtype %s; expected float16, int8 or float32" % A.dtype)
    in_types = {TDG_DTYPE_F16F32: (torch.float16, torch.int16), TDG_DTYPE_I8I32: (torch.int8,),
                TDG_DTYPE_F32F32: (torch.float32,)}[dt]
    M, K, pa, lda = _matrix(A, in_types, "A")
    K2, N, pb, ldb = _matrix(B, in_types, "B")
    if K != K2:
        raise ValueError("inner dimensions differ: A is %dx%d, B is %dx%d" % (M, K, K2, N))
    if A.device != B.device:
        raise ValueError("A and B are on different devices")
    out_type = torch.int32 if dt == TDG_DTYPE_I8I32 else torch.float32
    if C is None:
        C = torch.empty((M, N), dtype=out_type, device=A.device)
    Mc, Nc, pc, ldc = _matrix(C, (out_type,), "C")
    if (Mc, Nc) != (M, N):
        raise ValueError("C has shape %s, expected %s" % ((Mc, Nc), (M, N)))
    if C.device != A.device:
        raise ValueError("C is on %s, A and B on %s" % (C.device, A.device))
    with torch.cuda.device(A.device):
        rc = _fn("gemm_splitk_noalloc")(dt, M, N, K, pa, lda, pb, ldb, pc, ldc, int(parts),
                                         _stream_handle(A.device.index))
    if rc != TDG_OK:
        raise TdgError(rc, "gemm_splitk_noalloc")
    return C


def tdg_set_debug_flags(flags: int) -> int:
    """Sets the process-wide TDG_DEBUG_* bits; returns the previous ones."""
    rc = load_library().tdg_set_debug_flags(flags)
    if rc < 0:
        raise TdgError(rc, "tdg_set_debug_flags")
    return rc


def tdg_config_count(dtype: int) -> int:
    return load_library().tdg_config_count(dtype)


def tdg_config_at(dtype: int, index: int) -> dict:
    c = TdgConfig()
    rc = load_library().tdg_config_at(dtype, index, ctypes.byref(c))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_config_at")
    return c.as_dict()


def tdg_config_resources(dtype: int, index: int) -> dict:
    """Registers, spill bytes, LDS bytes, threads and runtime workgroups per
    CU of the index-th built configuration's kernel (needs the GPU)."""
    r = TdgKernelResources()
    rc = load_library().tdg_config_resources(dtype, index, ctypes.byref(r))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_config_resources")
    return r.as_dict()


def tdg_status_string(status: int) -> str:
    return status_string(status)


# ------------------------------------------------------ copy / transpose ladder

def _move(x, out, transpose, method):
    torch = _torch()
    rows, cols, px, ldi = _matrix(x, (torch.float32,), "in")
    shape = (cols, rows) if transpose else (rows, cols)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    orow, ocol, po, ldo = _matrix(out, (torch.float32,), "out")
    if (orow, ocol) != shape:
        raise ValueError("out has shape %s, expected %s" % ((orow, ocol), shape))
    if out.device != x.device:
        raise ValueError("out is on %s, in on %s" % (out.device, x.device))
    lib = load_library()
    with torch.cuda.device(x.device):
        stream = torch.cuda.current_stream(x.device).cuda_stream
        if transpose:
            rc = lib.tdg_transpose_f32(int(method), rows, cols, px, ldi, po, ldo, stream)
        else:
            rc = lib.tdg_copy_f32(rows, cols, px, ldi, po, ldo, stream)
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_transpose_f32" if transpose else "tdg_copy_f32")
    return out


def tdg_copy_f32(x, out=None):
    """out[i][j] = x[i][j] (float32, device tensors; rows may be strided)."""
    return _move(x, out, False, 0)


def tdg_transpose_f32(x, out=None, method=TDG_TRANSPOSE_AUTO):
    """out[j][i] = x[i][j] with one of the ladder's methods."""
    return _move(x, out, True, method)


# ------------------------------------------------------ measured compute ceiling

def tdg_mfma_probe_ops(dtype: int, iters: int) -> int:
    """Operations one tdg_mfma_probe launch performs."""
    return load_library().tdg_mfma_probe_ops(dtype, iters)


def tdg_mfma_probe_sink_floats() -> int:
    return load_library().tdg_mfma_probe_sink_floats()


LDS_PROBE_MODES = {"b128": 0, "b64_tr_b16": 1, "b64": 2}


def tdg_lds_probe_bytes(mode: int, iters: int) -> int:
    """Bytes one workgroup of tdg_lds_probe reads."""
    return load_library().tdg_lds_probe_bytes(mode, iters)


def tdg_lds_probe(mode: int, iters: int = 4096, out=None) -> float:
    """Run the LDS read-rate kernel on the current stream and wait for it;
    returns the mean bytes per shader clock per compute unit."""
    torch = _torch()
    if out is None:
        out = torch.zeros(512, dtype=torch.int32, device="cuda")
    if out.dtype != torch.int32 or out.numel() < 512 or not out.is_cuda:
        raise ValueError("out must be a device int32 tensor of at least 512 elements")
    lib = load_library()
    with torch.cuda.device(out.device):
        stream = torch.cuda.current_stream(out.device).cuda_stream
        rc = lib.tdg_lds_probe(mode, iters, out.data_ptr(), stream)
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_lds_probe")
    torch.cuda.synchronize(out.device)
    cycles = out[:256].cpu().long() & 0xFFFFFFFF
    return tdg_lds_probe_bytes(mode, iters) / float(cycles.double().mean())


def tdg_mfma_probe(dtype: int, iters: int, sink=None):
    """Launch the MFMA-only kernel on the current stream; returns the sink
    tensor (allocated when not given)."""
    torch = _torch()
    n = tdg_mfma_probe_sink_floats()
    if sink is None:
        sink = torch.empty(n, dtype=torch.float32, device="cuda")
    if sink.dtype != torch.float32 or sink.numel() < n or not sink.is_cuda:
        raise ValueError("sink must be a device float32 tensor of at least %d elements" % n)
    lib = load_library()
    with torch.cuda.device(sink.device):
        stream = torch.cuda.current_stream(sink.device).cuda_stream
        rc = lib.tdg_mfma_probe(dtype, iters, sink.data_ptr(), stream)
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_mfma_probe")
    return sink


# ------------------------------------------------------ rows that pick their weights

TDG_ELEM_F16 = 0
TDG_ELEM_F32 = 1
TDG_LORA_MAX_RANK = 256


_FLOATS = _HALF = _SINGLE = _BYTE = _INT = None  # dtype tuples, once torch is loaded


def _types():
    """Loads torch's names that the calls below use, once."""
    global _FLOATS, _HALF, _SINGLE, _BYTE, _INT, _empty, _device_now
    torch = _torch()
    _empty = torch.empty_strided  # a microsecond less than torch.empty with a device
    _device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _FLOATS, _HALF = (torch.float16, torch.float32), (torch.float16, torch.int16)
    _SINGLE, _BYTE = (torch.float32,), (torch.uint8,)
    _INT = (torch.int32,)  # the last: callers in other threads look at it


def _mat(t, types, what, dev=None):
    """Checks a device matrix with contiguous rows, on device `dev` where one
    is given: (rows, cols, address, ld, device index)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (what, tuple(shape)))
    if t.dtype not in types:
        raise TypeError("%s has dtype %s; expected one of %s" % (what, t.dtype, types))
    at = t.get_device()
    if at < 0:
        raise ValueError("%s must be a device tensor" % what)
    if dev is not None and at != dev:
        raise ValueError("%s is on device %d, expected %d" % (what, at, dev))
    rows, cols = shape
    if rows == 0 or cols == 0:
        return rows, cols, t.data_ptr(), cols or 1, at
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s: elements within a row must be contiguous" % what)
    return rows, cols, t.data_ptr(), ld if rows > 1 else cols, at


def _stack(t, types, what, dev):
    """A stack of such matrices: (count, rows, cols, address, ld, stride)."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must be 3-D, got shape %s" % (what, tuple(shape)))
    if t.dtype not in types:
        raise TypeError("%s has dtype %s; expected one of %s" % (what, t.dtype, types))
    if t.get_device() != dev:
        raise ValueError("%s must be a device tensor on device %d" % (what, dev))
    count, rows, cols = shape
    if count == 0 or rows == 0 or cols == 0:
        return count, rows, cols, t.data_ptr(), cols or 1, rows * (cols or 1)
    stride, ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s: elements within a row must be contiguous" % what)
    if rows == 1:
        ld = cols
    return count, rows, cols, t.data_ptr(), ld, stride if count > 1 else rows * ld


def _whole_numbers(t, what, dev, shape):
    """Checks a dense device int32 tensor; returns its address."""
    if t.dtype not in _INT:
        raise TypeError("%s has dtype %s; expected torch.int32" % (what, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be a device tensor on device %d" % (what, dev))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


def _launch(name, dev, *args):
    """Calls entry point `name` with torch's current stream of device `dev`."""
    if _device_now() == dev:
        rc = _fn(name)(*args, _stream_handle(dev))
    else:
        with _torch().cuda.device(dev):
            rc = _fn(name)(*args, _stream_handle(dev))
    if rc != TDG_OK:
        raise TdgError(rc, name)


def _workspace(ws, need, t):
    """(tensor, address, bytes) of a workspace on t's device, allocated when
    not given."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = _empty((need,), (1,), dtype=_torch().uint8, device=t.device)
        return ws, ws.data_ptr(), need
    if ws.get_device() != t.get_device() or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % t.device)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def tdg_route_workspace(tokens: int, top_k: int, experts: int) -> int:
    """Bytes of workspace that tdg_route_plan needs."""
    need = ctypes.c_size_t()
    rc = _fn("tdg_route_workspace")(tokens, top_k, experts, ctypes.byref(need))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_route_workspace")
    return need.value


def tdg_route_plan(ids, experts: int, offsets=None, order=None, slots=None, workspace=None):
    """Sorts the choices ids (tokens x top_k, int32; an id outside
    [0, experts) is dropped) by expert, stably.  Returns (offsets, order,
    slots): expert g's sorted rows are offsets[g] .. offsets[g + 1] - 1,
    order[i] is the entry token * top_k + j of sorted row i (-1 behind the
    last), slots[t, j] the sorted row of an entry (-1 when dropped)."""
    if _INT is None:
        _types()
    tokens, top_k, p_ids, ld, dev = _mat(ids, _INT, "ids")
    experts, n = int(experts), tokens * top_k
    need = tdg_route_workspace(tokens, top_k, experts)  # refuses bad sizes
    if offsets is None:
        offsets = _empty((experts + 1,), (1,), dtype=ids.dtype, device=ids.device)
        p_off = offsets.data_ptr()
    else:
        p_off = _whole_numbers(offsets, "offsets", dev, (experts + 1,))
    if order is None:
        order = _empty((n,), (1,), dtype=ids.dtype, device=ids.device)
        p_ord = order.data_ptr()
    else:
        p_ord = _whole_numbers(order, "order", dev, (n,))
    if slots is None:
        slots = _empty((tokens, top_k), (top_k, 1), dtype=ids.dtype, device=ids.device)
        p_slots = slots.data_ptr()
    else:
        p_slots = _whole_numbers(slots, "slots", dev, (tokens, top_k))
    ws, p_ws, ws_bytes = _workspace(workspace, need, ids)
    _launch("tdg_route_plan", dev, tokens, top_k, experts, p_ids, ld, p_off, p_ord, p_slots, p_ws, ws_bytes)
    return offsets, order, slots


def _slots_of(slots, dev):
    if len(slots.shape) != 2:
        raise ValueError("slots must be 2-D, got shape %s" % (tuple(slots.shape),))
    tokens, top_k = slots.shape
    return tokens, top_k, _whole_numbers(slots, "slots", dev, slots.shape)


def _weights_of(w, slots, what, dev):
    """(address, ld) of tokens x top_k FP32 weights."""
    tokens, top_k, p, ld, _ = _mat(w, _SINGLE, what, dev)
    if w.shape != slots.shape:
        raise ValueError("%s has shape %s, expected %s" % (what, (tokens, top_k), tuple(slots.shape)))
    return p, ld


def tdg_rows_dispatch(x, slots, out=None):
    """out[slots[t, j]] = x[t] (float16 or float32).  `out` (rows x cols) has
    tokens * top_k rows when allocated here; rows that no slot names are left
    as they are."""
    if _INT is None:
        _types()
    T, cols, px, ldx, dev = _mat(x, _FLOATS, "x")
    tokens, top_k, p_slots = _slots_of(slots, dev)
    if tokens != T:
        raise ValueError("x has %d rows, slots %d" % (T, tokens))
    if out is None:
        out = _empty((tokens * top_k, cols), (cols, 1), dtype=x.dtype, device=x.device)
    rows, oc, po, ldo, _ = _mat(out, (x.dtype,), "out", dev)
    if oc != cols:
        raise ValueError("out has %d columns, x %d" % (oc, cols))
    _launch("tdg_rows_dispatch", dev, _FLOATS.index(x.dtype), tokens, top_k, cols, px, ldx, p_slots, rows, po, ldo)
    return out


def tdg_rows_combine(z, slots, weights=None, out=None, out_dtype=None):
    """y[t] = sum over j of weights[t, j] * z[slots[t, j]], in FP32, rounded
    once to `out`'s type (out_dtype, else z's, when allocated here).  Without
    weights it is the gradient of tdg_rows_dispatch."""
    if _INT is None:
        _types()
    rows, cols, pz, ldz, dev = _mat(z, _FLOATS, "z")
    tokens, top_k, p_slots = _slots_of(slots, dev)
    if out is None:
        out = _empty((tokens, cols), (cols, 1), dtype=out_dtype or z.dtype, device=z.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out has dtype %s, out_dtype is %s" % (out.dtype, out_dtype))
    orow, oc, po, ldo, _ = _mat(out, _FLOATS, "out", dev)
    if orow != tokens or oc != cols:
        raise ValueError("out has shape %s, expected %s" % ((orow, oc), (tokens, cols)))
    pw, ldw = (None, top_k) if weights is None else _weights_of(weights, slots, "weights", dev)
    _launch("tdg_rows_combine", dev, _FLOATS.index(z.dtype), _FLOATS.index(out.dtype), tokens, top_k, cols, pz, ldz,
            rows, p_slots, pw, ldw, po, ldo)
    return out


def tdg_rows_combine_grad(dy, z, slots, weights=None, dz=None, dweights=None):
    """The gradient of tdg_rows_combine: (dz, dweights) with
    dz[slots[t, j]] = weights[t, j] * dy[t] (z's type) and dweights[t, j] =
    <dy[t], z[slots[t, j]]> (float32).  Rows of dz that no slot names are left
    as they are."""
    if _INT is None:
        _types()
    rows, cols, pz, ldz, dev = _mat(z, _FLOATS, "z")
    T, dc, pdy, ldy, _ = _mat(dy, _FLOATS, "dy", dev)
    tokens, top_k, p_slots = _slots_of(slots, dev)
    if tokens != T or dc != cols:
        raise ValueError("dy is %dx%d, z has %d columns and slots %d rows" % (T, dc, cols, tokens))
    if dz is None:
        dz = _empty((rows, cols), (cols, 1), dtype=z.dtype, device=z.device)
    zr, zc, pdz, lddz, _ = _mat(dz, (z.dtype,), "dz", dev)
    if zr != rows or zc != cols:
        raise ValueError("dz has shape %s, expected %s" % ((zr, zc), (rows, cols)))
    if dweights is None:
        dweights = _empty((tokens, top_k), (top_k, 1), dtype=_SINGLE[0], device=z.device)
    pw, ldw = (None, top_k) if weights is None else _weights_of(weights, slots, "weights", dev)
    pdw, lddw = _weights_of(dweights, slots, "dweights", dev)
    _launch("tdg_rows_combine_grad", dev, _FLOATS.index(z.dtype), _FLOATS.index(dy.dtype), tokens, top_k, cols, pdy,
            ldy, pz, ldz, rows, p_slots, pw, ldw, pdz, lddz, pdw, lddw)
    return dz, dweights


def _offsets_of(offsets, dev):
    """(groups, address) of groups + 1 row offsets."""
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError("offsets must hold groups + 1 values, got shape %s" % (tuple(shape),))
    return shape[0] - 1, _whole_numbers(offsets, "offsets", dev, shape)


def _grouped(name, A, B, offsets, C, transposed):
    if _INT is None:
        _types()
    M, K, pa, lda, dev = _mat(A, _HALF, "A")
    groups, rb, cb, pb, ldb, stride = _stack(B, _HALF, "B", dev)
    N, K2 = (rb, cb) if transposed else (cb, rb)
    n_off, p_off = _offsets_of(offsets, dev)
    if n_off != groups:
        raise ValueError("offsets name %d groups, B has %d" % (n_off, groups))
    if K != K2:
        raise ValueError("inner dimensions differ: A has %d columns, B's matrices are %dx%d" % (K, rb, cb))
    if C is None:
        C = _empty((M, N), (N, 1), dtype=_SINGLE[0], device=A.device)
    Mc, Nc, pc, ldc, _ = _mat(C, _SINGLE, "C", dev)
    if Mc != M or Nc != N:
        raise ValueError("C has shape %s, expected %s" % ((Mc, Nc), (M, N)))
    _launch(name, dev, groups, p_off, M, N, K, pa, lda, pb, ldb, stride, pc, ldc)
    return C


def gemm_f16f32_grouped(A, B, offsets, C=None):
    """C[i] (float32) = A[i] . B[g] (float16) for the rows offsets[g] <= i <
    offsets[g + 1] of A (M x K); B: groups x K x N; offsets: int32 device
    tensor of groups + 1 values.  Rows of no group are left as they are."""
    return _grouped("gemm_f16f32_grouped", A, B, offsets, C, False)


def gemm_f16f32_grouped_nt(A, B, offsets, C=None):
    """C[i] = A[i] . B[g]^T, B: groups x N x K: with the gradient of
    gemm_f16f32_grouped's result as A and its B, the gradient of its A."""
    return _grouped("gemm_f16f32_grouped_nt", A, B, offsets, C, True)


def gemm_f16f32_grouped_tn(A, B, offsets, C=None):
    """C[g] = A[rows of g]^T . B[rows of g] (groups x M x N): with
    gemm_f16f32_grouped's A and the gradient of its result, the gradient of
    its B.  Zeros for a group without rows."""
    if _INT is None:
        _types()
    rows, M, pa, lda, dev = _mat(A, _HALF, "A")
    rows_b, N, pb, ldb, _ = _mat(B, _HALF, "B", dev)
    if rows != rows_b:
        raise ValueError("A has %d rows, B %d" % (rows, rows_b))
    groups, p_off = _offsets_of(offsets, dev)
    if C is None:
        C = _empty((groups, M, N), (M * N, N, 1), dtype=_SINGLE[0], device=A.device)
    gc, mc, nc, pc, ldc, stride = _stack(C, _SINGLE, "C", dev)
    if (gc, mc, nc) != (groups, M, N):
        raise ValueError("C has shape %s, expected %s" % ((gc, mc, nc), (groups, M, N)))
    _launch("gemm_f16f32_grouped_tn", dev, groups, p_off, rows, M, N, pa, lda, pb, ldb, pc, ldc, stride)
    return C


def tdg_lora_workspace(M: int, N: int, K: int, adapters: int, rank: int) -> int:
    """Bytes of workspace that gemm_f16f32_lora needs (not growing with M
    throughout: for several sizes take the largest)."""
    need = ctypes.c_size_t()
    rc = _fn("tdg_lora_workspace")(M, N, K, adapters, rank, ctypes.byref(need))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_lora_workspace")
    return need.value


def gemm_f16f32_lora(A, B, down, up, adapter, scale=None, C=None, workspace=None):
    """C[t] (float32) = A[t] . B + scale[a] * (A[t] . down[a]) . up[a] with
    a = adapter[t] (int32; a row with a outside the stack gets A[t] . B
    alone).  A: M x K, B: K x N, down: adapters x K x rank, up: adapters x
    rank x N (float16); scale: float32 or None (1).  The workspace is
    allocated here when not given."""
    if _INT is None:
        _types()
    M, K, pa, lda, dev = _mat(A, _HALF, "A")
    K2, N, pb, ldb, _ = _mat(B, _HALF, "B", dev)
    n, kd, rank, pd, ldd, sd = _stack(down, _HALF, "down", dev)
    nu, ru, cu, pu, ldu, su = _stack(up, _HALF, "up", dev)
    if K != K2:
        raise ValueError("inner dimensions differ: A is %dx%d, B is %dx%d" % (M, K, K2, N))
    if kd != K or nu != n or ru != rank or cu != N:
        raise ValueError("down is %s and up %s; expected adapters x %d x rank and adapters x rank x %d"
                         % (tuple(down.shape), tuple(up.shape), K, N))
    p_ad = _whole_numbers(adapter, "adapter", dev, (M,))
    p_sc = None
    if scale is not None:
        if scale.dtype not in _SINGLE or scale.shape != (n,) or not scale.is_contiguous():
            raise ValueError("scale must be a contiguous float32 tensor of %d values" % n)
        if scale.get_device() != dev:
            raise ValueError("scale must be a device tensor on device %d" % dev)
        p_sc = scale.data_ptr()
    if C is None:
        C = _empty((M, N), (N, 1), dtype=_SINGLE[0], device=A.device)
    Mc, Nc, pc, ldc, _ = _mat(C, _SINGLE, "C", dev)
    if Mc != M or Nc != N:
        raise ValueError("C has shape %s, expected %s" % ((Mc, Nc), (M, N)))
    ws, p_ws, ws_bytes = _workspace(workspace, tdg_lora_workspace(M, N, K, n, rank), A)
    _launch("gemm_f16f32_lora", dev, M, N, K, pa, lda, pb, ldb, n, rank, pd, ldd, sd, pu, ldu, su, p_ad, p_sc, pc,
            ldc, p_ws, ws_bytes)
    return C


# ------------------------------------------------------ 4-bit weights with group scales

def _codes_of(t, dev, stack):
    """Checks the codes of a matrix (blocks x N x 64) or of a stack of them:
    (count, blocks, N, address, ld, stride)."""
    shape = t.shape
    if len(shape) != 3 + stack or shape[-1] != 64:
        raise ValueError("codes must be %sblocks x N x 64, got shape %s" % ("count x " * stack, tuple(shape)))
    if t.dtype not in _BYTE:
        raise TypeError("codes has dtype %s; expected torch.uint8" % t.dtype)
    if t.get_device() != dev:
        raise ValueError("codes must be a device tensor on device %d" % dev)
    count = shape[0] if stack else 1
    blocks, N = shape[-3:-1]
    if count == 0 or blocks == 0 or N == 0:
        return count, blocks, N, t.data_ptr(), N or 1, blocks * (N or 1)
    st = t.stride()
    ld, stride = st[-3] if blocks > 1 else N * 64, st[0] if count > 1 else 0
    if st[-1] != 1 or (st[-2] != 64 and N > 1) or ld % 64 or stride % 64:
        raise ValueError("codes: a block's columns must be contiguous, and strides whole pieces of 64")
    return count, blocks, N, t.data_ptr(), ld // 64, stride // 64


def _group_values(t, types, what, dev, count, groups, N):
    """Checks scales or zeros, groups x N or a stack of them (`count` not
    None): (address, ld, stride)."""
    if count is None:
        rows, cols, p, ld, _ = _mat(t, types, what, dev)
        stride = 0
    else:
        n, rows, cols, p, ld, stride = _stack(t, types, what, dev)
    if rows != groups or cols != N or (count is not None and n != count):
        raise ValueError("%s has shape %s, expected %s" % (
            what, tuple(t.shape), (groups, N) if count is None else (count, groups, N)))
    return p, ld, stride


def _w4(codes, scales, zeros, K, group, dev, stack):
    """The checked arguments of 4-bit weights: (count, N, their addresses, leading
    dimensions and strides)."""
    count, blocks, N, pc, ldc, sc = _codes_of(codes, dev, stack)
    group = int(group)
    if group < 32 or group % 32:
        raise ValueError("group must be a multiple of 32, got %d" % group)
    if blocks != (K + 127) // 128:
        raise ValueError("codes have %d blocks, K = %d needs %d" % (blocks, K, (K + 127) // 128))
    of, groups = count if stack else None, (K + group - 1) // group
    ps, lds, ss = _group_values(scales, _HALF, "scales", dev, of, groups, N)
    pz, ldz, sz = (None, N or 1, 0) if zeros is None else _group_values(zeros, _BYTE, "zeros", dev, of, groups, N)
    return count, N, (pc, ldc, sc, ps, lds, ss, pz, ldz, sz)


def _new(shape, dtype, t):
    """A dense tensor on t's device."""
    strides, n = [], 1
    for d in reversed(shape):
        strides.append(n)
        n *= d or 1
    return _empty(shape, strides[::-1], dtype=dtype, device=t.device)


def tdg_w4_quantize(W, group: int = 128, zeros=False, codes=None, scales=None):
    """4-bit weights of W (K x N, or count x K x N; float16): (codes, scales,
    zeros), with zero points where `zeros` is True or a uint8 tensor for them,
    else None.  codes: ceil(K / 128) x N x 64 uint8 in the layout that the
    products take; scales (float16) and zeros: ceil(K / group) x N; a stack's
    have its count in front."""
    if _INT is None:
        _types()
    stack = len(W.shape) == 3
    if stack:
        dev = W.get_device()
        if dev < 0:
            raise ValueError("W must be a device tensor")
        count, K, N, pw, ldw, sw = _stack(W, _HALF, "W", dev)
    else:
        K, N, pw, ldw, dev = _mat(W, _HALF, "W")
        count, sw = 1, 0
    group = int(group)
    if group < 32 or group % 32:
        raise ValueError("group must be a multiple of 32, got %d" % group)
    blocks, groups = (K + 127) // 128, (K + group - 1) // group
    front = (count,) if stack else ()
    fresh = codes is None and scales is None and isinstance(zeros, bool)
    if codes is None:
        codes = _new(front + (blocks, N, 64), _BYTE[0], W)
    if scales is None:
        scales = _new(front + (groups, N), _HALF[0], W)
    if zeros is False:
        zeros = None
    elif zeros is True:
        zeros = _new(front + (groups, N), _BYTE[0], W)
    if fresh:
        ld, sg = N or 1, groups * (N or 1)
        places = (codes.data_ptr(), ld, blocks * ld, scales.data_ptr(), ld, sg,
                  None if zeros is None else zeros.data_ptr(), ld, sg)
    else:
        n, cols, places = _w4(codes, scales, zeros, K, group, dev, stack)
        if n != count or cols != N:
            raise ValueError("codes have shape %s, W %s" % (tuple(codes.shape), tuple(W.shape)))
    _launch("tdg_w4_quantize", dev, count, K, N, group, pw, ldw, sw, *places)
    return codes, scales, zeros


def tdg_w4_dequantize(codes, scales, zeros=None, K=None, group: int = 128, out=None, out_dtype=None):
    """The weights (code - zero) * scale, K x N or a stack of them, rounded
    once to `out`'s type (out_dtype, else float16, when allocated here).  K is
    128 times the codes' blocks, and not more, when not given."""
    if _INT is None:
        _types()
    stack = len(codes.shape) == 4
    dev = codes.get_device()
    if dev < 0:
        raise ValueError("codes must be a device tensor")
    if K is None:
        K = codes.shape[-3] * 128 if len(codes.shape) > 2 else 0
    K, group = int(K), int(group)
    count, N, places = _w4(codes, scales, zeros, K, group, dev, stack)
    if out is None:
        out = _new((count, K, N) if stack else (K, N), out_dtype or _HALF[0], codes)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out has dtype %s, out_dtype is %s" % (out.dtype, out_dtype))
    if stack:
        n, rows, cols, po, ldo, so = _stack(out, _FLOATS, "out", dev)
    else:
        rows, cols, po, ldo, _ = _mat(out, _FLOATS, "out", dev)
        n, so = 1, 0
    if (n, rows, cols) != (count, K, N):
        raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (count,) * stack + (K, N)))
    _launch("tdg_w4_dequantize", dev, _FLOATS.index(out.dtype), count, K, N, group, *places, po, ldo, so)
    return out


def _result(C, M, N, A, dev):
    """(tensor, address, ld) of a product's M x N float32 result on A's device,
    allocated when not given."""
    if C is None:
        C = _empty((M, N), (N, 1), dtype=_SINGLE[0], device=A.device)
        return C, C.data_ptr(), N or 1
    Mc, Nc, p, ld, _ = _mat(C, _SINGLE, "C", dev)
    if Mc != M or Nc != N:
        raise ValueError("C has shape %s, expected %s" % ((Mc, Nc), (M, N)))
    return C, p, ld


def gemm_f16w4f32(A, codes, scales, zeros=None, group: int = 128, C=None):
    """C (float32) = A (M x K, float16) times 4-bit weights as tdg_w4_quantize
    makes them (zeros None: 8)."""
    if _INT is None:
        _types()
    M, K, pa, lda, dev = _mat(A, _HALF, "A")
    _, N, (pc, ldc, _, ps, lds, _, pz, ldz, _) = _w4(codes, scales, zeros, K, group, dev, False)
    C, p_out, ld_out = _result(C, M, N, A, dev)
    _launch("gemm_f16w4f32", dev, M, N, K, int(group), pa, lda, pc, ldc, ps, lds, pz, ldz, p_out, ld_out)
    return C


def gemm_f16w4f32_grouped(A, codes, scales, offsets, zeros=None, group: int = 128, C=None):
    """C[i] (float32) = A[i] times 4-bit matrix g for the rows offsets[g] <= i <
    offsets[g + 1] of A (M x K, float16); codes, scales and zeros are stacks.
    Rows of no group are left as they are."""
    if _INT is None:
        _types()
    M, K, pa, lda, dev = _mat(A, _HALF, "A")
    count, N, places = _w4(codes, scales, zeros, K, group, dev, True)
    n_off, p_off = _offsets_of(offsets, dev)
    if n_off != count:
        raise ValueError("offsets name %d groups, codes have %d" % (n_off, count))
    C, p_out, ld_out = _result(C, M, N, A, dev)
    _launch("gemm_f16w4f32_grouped", dev, count, p_off, M, N, K, int(group), pa, lda, *places, p_out, ld_out)
    return C


# ------------------------------------------------------ a layer of experts for a few tokens

TDG_LAYER_MAX_TOKENS = 64
TDG_LAYER_MAX_TOP_K = 32


def tdg_expert_layer_workspace(tokens: int, top_k: int, experts: int, cols: int, inner: int) -> int:
    """Bytes of workspace that tdg_expert_layer needs (not growing with the
    tokens throughout: for several sizes take the largest)."""
    need = ctypes.c_size_t()
    rc = _fn("tdg_expert_layer_workspace")(tokens, top_k, experts, cols, inner, ctypes.byref(need))
    if rc != TDG_OK:
        raise TdgError(rc, "tdg_expert_layer_workspace")
    return need.value


def tdg_expert_layer(x, ids, weights, up, down, out=None, out_dtype=None, workspace=None):
    """y[t] = sum over j of weights[t, j] * (h . down[e]), e = ids[t, j], h =
    silu(x[t] . up[e][:, :inner]) * (x[t] . up[e][:, inner:]).  x: tokens x cols
    (float16), ids: tokens x top_k (int32; one outside the experts adds nothing),
    weights: float32 or None (1), up: experts x cols x 2 inner, down: experts x
    inner x cols (float16); `out` is float16 or float32 (out_dtype, else float16,
    when allocated here).  Up to 64 tokens with 32 choices each.  The workspace is
    allocated here when not given."""
    if _INT is None:
        _types()
    tokens, cols, px, ldx, dev = _mat(x, _HALF, "x")
    rows, top_k, p_ids, ld_ids, _ = _mat(ids, _INT, "ids", dev)
    if rows != tokens:
        raise ValueError("x has %d rows, ids %d" % (tokens, rows))
    pw, ldw = (None, top_k) if weights is None else _weights_of(weights, ids, "weights", dev)
    n, ku, nu, p_up, ld_up, s_up = _stack(up, _HALF, "up", dev)
    nd, inner, cd, p_down, ld_down, s_down = _stack(down, _HALF, "down", dev)
    if ku != cols or cd != cols or nu != 2 * inner or nd != n:
        raise ValueError("up is %s and down %s; expected experts x %d x 2 inner and experts x inner x %d"
                         % (tuple(up.shape), tuple(down.shape), cols, cols))
    if out is None:
        out = _empty((tokens, cols), (cols, 1), dtype=out_dtype or _HALF[0], device=x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out has dtype %s, out_dtype is %s" % (out.dtype, out_dtype))
    orow, oc, po, ldo, _ = _mat(out, _FLOATS, "out", dev)
    if orow != tokens or oc != cols:
        raise ValueError("out has shape %s, expected %s" % ((orow, oc), (tokens, cols)))
    ws, p_ws, ws_bytes = _workspace(workspace, tdg_expert_layer_workspace(tokens, top_k, n, cols, inner), x)
    _launch("tdg_expert_layer", dev, _FLOATS.index(out.dtype), tokens, top_k, n, cols, inner, px, ldx, p_ids, ld_ids,
            pw, ldw, p_up, ld_up, s_up, p_down, ld_down, s_down, po, ldo, p_ws, ws_bytes)
    return out

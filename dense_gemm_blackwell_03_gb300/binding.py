"""ctypes binding of ``libbwgemm.so`` (C ABI in ``include/bwgemm.h``).

Argument marshalling only: torch tensors are turned into device pointers,
element strides and the current CUDA stream, and every call goes straight to
the library, whose sm_103a kernels do all the arithmetic.  If the library
cannot be loaded the calls raise; there is no host-side fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

BF16 = 0
FP16 = 1
FP32 = 2

E4M3 = 0
E5M2 = 1

BLOCK = 128
BLOCK_ROW = 0
BLOCK_SQUARE = 1

SCHEDULE_AUTO = 0
SCHEDULE_TILES = 1
SCHEDULE_STREAM_K = 2
SCHEDULE_CLC = 3

STATUS_NAMES = {
    0: "BWGEMM_OK",
    1: "BWGEMM_ERR_INVALID_ARG",
    2: "BWGEMM_ERR_ALIGNMENT",
    3: "BWGEMM_ERR_UNSUPPORTED",
    4: "BWGEMM_ERR_NO_DEVICE",
    5: "BWGEMM_ERR_CUDA",
    6: "BWGEMM_ERR_TIMEOUT",
    7: "BWGEMM_ERR_WORKSPACE",
}

# every symbol include/bwgemm.h declares
EXPORTED = [
    "bwgemm_default_options", "bwgemm_create_plan", "bwgemm_destroy", "bwgemm_run",
    "bwgemm_run_host", "bwgemm_get_status", "bwgemm_last_device_status", "bwgemm_check_args",
    "bwgemm_select_config", "bwgemm_plan_last_config", "bwgemm_plan_launch_count",
    "bwgemm_status_string", "bwgemm_version", "bwgemm_run_splitk_noalloc",
    "bwgemm_plan_read_trace", "bwgemm_tune", "bwgemm_plan_tuned_count",
    "bwgemm_probe_tensor_rate", "bwgemm_noalloc_scratch", "bwgemm_bench_load_path",
    "bwgemm_quantize", "bwgemm_run_scaled", "bwgemm_orthogonalize", "bwgemm_orthogonalize_workspace",
    "bwgemm_select_scaled", "bwgemm_select_orthogonalize",
]

# layouts of bwgemm_bench_load_path
LOAD_PATH_LAYOUTS = {0: "128B swizzle", 1: "no swizzle, plain rows (same copies)",
                     2: "no swizzle, interleaved core matrices (8 copies per tile)",
                     3: "128B swizzle, one 256-row copy per K block",
                     4: "128B swizzle, A multicast in halves across two CTAs",
                     5: "128B swizzle, two K blocks (256-byte row pieces) per copy",
                     6: "128B swizzle, 64 KiB stages, A multicast in halves across two CTAs",
                     7: "128B swizzle, 64 KiB stages, no multicast"}

# timeline slots of bwgemm_plan_read_trace
(TRACE_ENTRY, TRACE_READY, TRACE_FIRST_LOAD, TRACE_LAST_LOAD, TRACE_EPI_DONE, TRACE_EXIT, TRACE_SETUP,
 TRACE_UNIT_KNOWN) = range(8)
TRACE_UNIT0 = 8
TRACE_UNITS = 14


class BwgemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        name = STATUS_NAMES.get(self.status, f"status {status}")
        super().__init__(f"{what}: {name}" if what else name)


class PlanOptions(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("tile_n", ctypes.c_int32),
        ("split_k", ctypes.c_int32),
        ("raster_group", ctypes.c_int32),
        ("max_ctas", ctypes.c_int32),
        ("stall_kblock", ctypes.c_int32),
        ("timeout_ns", ctypes.c_uint64),
        ("workspace_bytes", ctypes.c_uint64),
        ("schedule", ctypes.c_int32),
        ("pdl_off", ctypes.c_int32),
        ("trace", ctypes.c_int32),
        ("prefetch", ctypes.c_int32),
        ("swap_ab", ctypes.c_int32),
        ("multicast", ctypes.c_int32),
        ("copy_kblocks", ctypes.c_int32),
        ("cluster_split", ctypes.c_int32),
        ("tuned_table", ctypes.c_int32),
        ("skinny", ctypes.c_int32),
        ("wholek", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 1),
    ]


class Config(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("tile_m", ctypes.c_int32),
        ("tile_n", ctypes.c_int32),
        ("tile_k", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("split_k", ctypes.c_int32),
        ("raster_group", ctypes.c_int32),
        ("num_tiles", ctypes.c_int32),
        ("num_units", ctypes.c_int32),
        ("grid", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64),
        ("schedule", ctypes.c_int32),
        ("dp_tiles", ctypes.c_int32),
        ("sk_tiles", ctypes.c_int32),
        ("workers", ctypes.c_int32),
        ("split_scatter", ctypes.c_int32),
        ("swap_ab", ctypes.c_int32),
        ("multicast", ctypes.c_int32),
        ("copy_kblocks", ctypes.c_int32),
        ("prefetch_kblocks", ctypes.c_int32),
        ("prefetch_b", ctypes.c_int32),
        ("cluster_split", ctypes.c_int32),
        ("tuned", ctypes.c_int32),
        ("skinny", ctypes.c_int32),
        ("wholek", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class Scaled(ctypes.Structure):
    """``bwgemm_scaled_t``: 8-bit values and their scales."""
    _fields_ = [
        ("values", ctypes.c_void_p),
        ("ld", ctypes.c_int64),
        ("scales", ctypes.c_void_p),
        ("ld_scales", ctypes.c_int64),
        ("type", ctypes.c_int32),
        ("block", ctypes.c_int32),
    ]


class ScaledConfig(ctypes.Structure):
    """``bwgemm_scaled_config_t``."""
    _fields_ = [(name, ctypes.c_int32) for name in ("few_rows", "swap_ab", "tile_l", "tile_c", "column_scales", "dp_tiles",
                                                    "sk_tiles", "workers")]
    as_dict = Config.as_dict


class OrthoConfig(ctypes.Structure):
    """``bwgemm_ortho_config_t``."""
    _fields_ = [("tile", ctypes.c_int32), ("splits", ctypes.c_int32), ("tiles", ctypes.c_int64),
                ("workers", ctypes.c_int32)]
    as_dict = Config.as_dict


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    here = os.path.dirname(os.path.abspath(__file__))
    return os.environ.get("BWGEMM_LIBRARY", os.path.join(here, "_build", "libbwgemm.so"))


def load_library(build_if_missing: bool = False):
    """Load ``libbwgemm.so`` (building it first when asked and missing)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            if not build_if_missing:
                raise BwgemmError(4, f"{path} not built (run __graft_entry__.build())")
            from . import build as _build
            path = _build.build()
        lib = ctypes.CDLL(path)
        vp = ctypes.c_void_p
        i64 = ctypes.c_int64
        i32 = ctypes.c_int32
        st = ctypes.c_int
        lib.bwgemm_default_options.argtypes = [ctypes.POINTER(PlanOptions)]
        lib.bwgemm_default_options.restype = None
        lib.bwgemm_create_plan.argtypes = [ctypes.POINTER(vp), ctypes.c_int, ctypes.POINTER(PlanOptions)]
        lib.bwgemm_create_plan.restype = st
        lib.bwgemm_destroy.argtypes = [vp]
        lib.bwgemm_destroy.restype = st
        gemm_args = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, ctypes.c_int, vp]
        lib.bwgemm_run.argtypes = gemm_args
        lib.bwgemm_run.restype = st
        lib.bwgemm_run_host.argtypes = gemm_args
        lib.bwgemm_run_host.restype = st
        lib.bwgemm_run_splitk_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                                  ctypes.c_int, i32, vp]
        lib.bwgemm_run_splitk_noalloc.restype = st
        lib.bwgemm_noalloc_scratch.argtypes = [i32, i32, i64, i64, i64, i32,
                                               ctypes.POINTER(ctypes.c_uint64),
                                               ctypes.POINTER(ctypes.c_uint64)]
        lib.bwgemm_noalloc_scratch.restype = st
        lib.bwgemm_get_status.argtypes = [vp, vp]
        lib.bwgemm_get_status.restype = st
        lib.bwgemm_last_device_status.argtypes = [vp]
        lib.bwgemm_last_device_status.restype = ctypes.c_uint32
        lib.bwgemm_check_args.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, ctypes.c_int]
        lib.bwgemm_check_args.restype = st
        lib.bwgemm_select_config.argtypes = [i32, i32, i32, i64, i64, i64, ctypes.c_int,
                                             ctypes.POINTER(PlanOptions), ctypes.POINTER(Config)]
        lib.bwgemm_select_config.restype = st
        lib.bwgemm_plan_last_config.argtypes = [vp, ctypes.POINTER(Config)]
        lib.bwgemm_plan_last_config.restype = st
        lib.bwgemm_plan_read_trace.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64), i64,
                                               ctypes.POINTER(i32), ctypes.POINTER(i32)]
        lib.bwgemm_plan_read_trace.restype = st
        lib.bwgemm_plan_launch_count.argtypes = [vp]
        lib.bwgemm_plan_launch_count.restype = ctypes.c_uint64
        lib.bwgemm_tune.argtypes = gemm_args + [i32, ctypes.POINTER(Config)]
        lib.bwgemm_tune.restype = st
        lib.bwgemm_plan_tuned_count.argtypes = [vp]
        lib.bwgemm_plan_tuned_count.restype = i32
        lib.bwgemm_status_string.argtypes = [ctypes.c_int]
        lib.bwgemm_status_string.restype = ctypes.c_char_p
        lib.bwgemm_version.argtypes = []
        lib.bwgemm_version.restype = i32
        lib.bwgemm_probe_tensor_rate.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                                 ctypes.POINTER(i32)]
        lib.bwgemm_probe_tensor_rate.restype = st
        lib.bwgemm_bench_load_path.argtypes = [ctypes.c_int, i32, i32, i32, i32, i32,
                                               ctypes.POINTER(ctypes.c_double),
                                               ctypes.POINTER(ctypes.c_double)]
        lib.bwgemm_bench_load_path.restype = st
        ci = ctypes.c_int
        lib.bwgemm_quantize.argtypes = [vp, vp, ci, i64, i64, i64, ci, ci, i32, vp, i64, vp, i64, vp, i64, vp,
                                        i64, vp]
        lib.bwgemm_quantize.restype = st
        # the two bwgemm_scaled_t as addresses or packed bytes: the fastest arguments to pass
        lib.bwgemm_run_scaled.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, ci, i32, vp]
        lib.bwgemm_run_scaled.restype = st
        lib.bwgemm_orthogonalize.argtypes = [vp, vp, ci, vp, ci, i64, i64, i64, i64, i64, i64, i64, i32,
                                             ctypes.POINTER(ctypes.c_float), ctypes.c_float, ctypes.c_float, vp,
                                             ctypes.c_uint64, vp]
        lib.bwgemm_orthogonalize.restype = st
        lib.bwgemm_orthogonalize_workspace.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_uint64)]
        lib.bwgemm_orthogonalize_workspace.restype = st
        lib.bwgemm_select_scaled.argtypes = [i32, i64, i64, i64, ci, ctypes.POINTER(PlanOptions),
                                             ctypes.POINTER(ScaledConfig)]
        lib.bwgemm_select_scaled.restype = st
        lib.bwgemm_select_orthogonalize.argtypes = [i32, i32, i64, i64, i64, ci, i32, ctypes.POINTER(PlanOptions),
                                                    ctypes.POINTER(OrthoConfig)]
        lib.bwgemm_select_orthogonalize.restype = st
        _lib = lib
        return lib


def make_options(**kw) -> PlanOptions:
    lib = load_library()
    o = PlanOptions()
    lib.bwgemm_default_options(ctypes.byref(o))
    for k, v in kw.items():
        if v is None:
            continue
        if not hasattr(o, k) or k == "reserved":
            raise TypeError(f"unknown plan option {k!r}")
        setattr(o, k, v)
    return o


_torch_mod = None
_dtype_codes: dict = {}
_all_dtype_codes: dict = {}  # with fp32, for the calls that take it
_fp8_codes: dict = {}


def _torch():
    """The torch module, imported once (the per-call path looks it up here)."""
    global _torch_mod
    if _torch_mod is None:
        import torch
        _torch_mod = torch
        _dtype_codes.update({torch.bfloat16: BF16, torch.float16: FP16})
        _all_dtype_codes.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
        _fp8_codes.update({torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2})
    return _torch_mod


def _dtype_code(t) -> int:
    _torch()
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"bwgemm takes bfloat16 or float16 tensors, got {t.dtype}")
    return code


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("operands must be K-major / row-major (unit stride along the last dim)")
    return int(t.stride(0)) if t.shape[0] > 1 else max(int(t.shape[1]), 1)


def _padded_empty(rows: int, cols: int, dtype, device, multiple: int):
    """An uninitialised rows x cols matrix whose rows start a multiple of `multiple` elements apart."""
    ld = -(-cols // multiple) * multiple
    if ld == cols:
        return _torch_mod.empty((rows, cols), dtype=dtype, device=device)
    return _torch_mod.empty_strided((rows, cols), (ld, 1), dtype=dtype, device=device)


# bwgemm_scaled_t as a packed record (native sizes and alignment)
_SCALED = struct.Struct("@PqPqii")
assert _SCALED.size == ctypes.sizeof(Scaled)


def _pack_scaled(values, scales, name: str):
    """8-bit `values` (R x K) with `scales` ((K blocks) x (R or row blocks)) as the bytes
    of a bwgemm_scaled_t, R and K.  (A record of its own for every call: other threads
    run while the library reads it.  Strides are read here, not through _ld: this is the
    per-call path.)"""
    code = _fp8_codes.get(values.dtype)
    if code is None:
        raise TypeError(f"{name} must be float8_e4m3fn or float8_e5m2, got {values.dtype}")
    if scales.dtype is not _torch_mod.float32:
        raise TypeError(f"the scales of {name} must be float32, got {scales.dtype}")
    rows, K = values.shape
    blocks, per = scales.shape
    square = per != rows
    if blocks != (K + 127) >> 7 or (square and per != (rows + 127) >> 7):
        raise ValueError(f"the scales of {name} ({rows} x {K}) must be {-(-K // BLOCK)} x {rows} or "
                         f"{-(-K // BLOCK)} x {-(-rows // BLOCK)}, got {tuple(scales.shape)}")
    ld, unit = values.stride()
    lds, unit_s = scales.stride()
    if (unit != 1 and K > 1) or (unit_s != 1 and per > 1):
        raise ValueError(f"{name} and its scales need unit stride along the last dim")
    if rows <= 1:
        ld = (K + 15) & -16  # a single row has no next one
    record = _SCALED.pack(values.data_ptr(), ld, scales.data_ptr(), lds if blocks > 1 else per, code,
                          BLOCK_SQUARE if square else BLOCK_ROW)
    return record, rows, K


def select_config(num_sms: int, M: int, N: int, K: int, dtype: int = BF16, max_pairs: int = 0,
                  max_quads: int = 0, **opts) -> dict:
    """Host-only: the configuration a plan would choose (no GPU needed)."""
    lib = load_library()
    o = make_options(**opts)
    cfg = Config()
    rc = lib.bwgemm_select_config(num_sms, max_pairs, max_quads, M, N, K, dtype, ctypes.byref(o),
                                  ctypes.byref(cfg))
    if rc != 0:
        raise BwgemmError(rc, "bwgemm_select_config")
    return cfg.as_dict()


def select_scaled(num_sms: int, M: int, N: int, K: int, b_blocks: str = "square", **opts) -> dict:
    """Host-only: how a plan would divide gemm_scaled's product (no GPU needed)."""
    cfg = ScaledConfig()
    rc = load_library().bwgemm_select_scaled(num_sms, M, N, K, BLOCK_SQUARE if b_blocks == "square" else BLOCK_ROW,
                                             ctypes.byref(make_options(**opts)), ctypes.byref(cfg))
    if rc != 0:
        raise BwgemmError(rc, "bwgemm_select_scaled")
    return cfg.as_dict()


def select_orthogonalize(num_sms: int, batch: int, rows: int, cols: int, dtype: int = BF16, step: int = 0,
                         max_pairs: int = 0, **opts) -> list:
    """Host-only: how a plan would divide the products S, B and X of orthogonalize's `step`."""
    cfg = (OrthoConfig * 3)()
    rc = load_library().bwgemm_select_orthogonalize(num_sms, max_pairs, batch, rows, cols, dtype, step,
                                                    ctypes.byref(make_options(**opts)), cfg)
    if rc != 0:
        raise BwgemmError(rc, "bwgemm_select_orthogonalize")
    return [c.as_dict() for c in cfg]


def probe_tensor_rate(device: int = 0):
    """(FLOP per SM clock of one SM's tensor pipe, SM count), measured on `device`
    by bwgemm_probe_tensor_rate."""
    lib = load_library()
    rate = ctypes.c_double(0.0)
    sms = ctypes.c_int32(0)
    rc = lib.bwgemm_probe_tensor_rate(int(device), ctypes.byref(rate), ctypes.byref(sms))
    if rc != 0:
        raise BwgemmError(rc, "bwgemm_probe_tensor_rate")
    return rate.value, sms.value


def bench_load_path(layout: int, source: int = 0, ctas: int = 0, stages: int = 6, kblocks: int = 4096,
                    device: int = 0):
    """(GB/s landed by all CTAs, milliseconds) of bwgemm_bench_load_path."""
    lib = load_library()
    gbs = ctypes.c_double(0.0)
    ms = ctypes.c_double(0.0)
    rc = lib.bwgemm_bench_load_path(int(device), int(layout), int(source), int(ctas), int(stages),
                                    int(kblocks), ctypes.byref(gbs), ctypes.byref(ms))
    if rc != 0:
        raise BwgemmError(rc, "bwgemm_bench_load_path")
    return gbs.value, ms.value


def check_args(A_ptr, B_ptr, C_ptr, M, N, K, lda, ldb, ldc, dtype=BF16) -> int:
    """Host-only: the status bwgemm_run would return for these arguments."""
    return int(load_library().bwgemm_check_args(A_ptr, B_ptr, C_ptr, M, N, K, lda, ldb, ldc, dtype))


class Plan:
    """A bwgemm plan on one CUDA device (see ``bwgemm_create_plan``), for one thread and one
    stream at a time: its launches share a workspace and a status word."""

    def __init__(self, device: int | None = None, **opts):
        import torch
        self.lib = load_library()
        if device is None:
            device = torch.cuda.current_device()
        self.device = int(device)
        self.options = make_options(**opts)
        h = ctypes.c_void_p()
        rc = self.lib.bwgemm_create_plan(ctypes.byref(h), self.device, ctypes.byref(self.options))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_create_plan")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            self.lib.bwgemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _check_device(self, *tensors):
        # the library refuses operands that are not memory of the plan's
        # device as well; this names the tensor
        for name, t in zip(("A", "B", "out"), tensors):
            if t.device.type != "cuda" or t.device.index != self.device:
                raise ValueError(f"{name} is on {t.device}, the plan on cuda:{self.device}")

    @staticmethod
    def _stream_handle(stream):
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        return ctypes.c_void_p(int(stream.cuda_stream))

    def run_raw(self, A_ptr: int, B_ptr: int, C_ptr: int, M: int, N: int, K: int, lda: int,
                ldb: int, ldc: int, dtype: int, stream_ptr: int | None) -> int:
        """Direct call of ``bwgemm_run`` with raw pointers; returns the status code."""
        return int(self.lib.bwgemm_run(self.handle, A_ptr, B_ptr, C_ptr, M, N, K, lda, ldb, ldc,
                                       dtype, stream_ptr))

    def gemm(self, A, B, out=None, stream=None):
        """``out = A @ B.T`` for CUDA bf16/fp16 tensors A (M x K) and B (N x K)."""
        torch = _torch()
        dt = _dtype_code(A)
        if B.dtype != A.dtype:
            raise TypeError("A and B must have the same dtype")
        dev = self.device
        # get_device(): the CUDA device index, -1 for host tensors
        if A.get_device() != dev or B.get_device() != dev:
            if not (A.is_cuda and B.is_cuda):
                raise ValueError("A and B must be CUDA tensors (bwgemm has no host path)")
            self._check_device(A, B)
        M, K = A.shape
        N, Kb = B.shape
        if Kb != K:
            raise ValueError(f"K mismatch: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
        if out is None:
            out = torch.empty((M, N), dtype=A.dtype, device=A.device)
        elif out.dtype != A.dtype or out.shape != (M, N) or out.get_device() != dev:
            if out.dtype != A.dtype or tuple(out.shape) != (M, N) or not out.is_cuda:
                raise ValueError("out must be an M x N CUDA tensor of the operands' dtype")
            self._check_device(A, B, out)
        s = (torch.cuda.current_stream(dev) if stream is None else stream).cuda_stream
        rc = self.lib.bwgemm_run(self.handle, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K,
                                 _ld(A), _ld(B), _ld(out), dt, s)
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_run")
        return out

    def gemm_host(self, A, B, out=None, stream=None):
        """``bwgemm_run_host``: A, B, out are CPU tensors (pinned for speed)."""
        import torch
        dt = _dtype_code(A)
        M, K = A.shape
        N, _ = B.shape
        if out is None:
            out = torch.empty((M, N), dtype=A.dtype)
        rc = self.lib.bwgemm_run_host(self.handle, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N,
                                      K, _ld(A), _ld(B), _ld(out), dt, self._stream_handle(stream))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_run_host")
        return out

    def _check_tensor(self, name, t):
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, the plan on cuda:{self.device}")

    def quantize(self, X, blocks: str = "row", transposed: bool = False, pow2: bool = False, dtype=None,
                 stream=None):
        """``bwgemm_quantize``: the 2-D CUDA tensor X (bf16, fp16 or fp32) in 8 bits
        with one fp32 scale per 128 elements of a row (``blocks="row"``) or per
        128 x 128 (``"square"``).

        Returns ``(q, scales)``, and with `transposed` also ``(qt, scales_t)`` of
        the transpose (its own blocks, along X's columns; with "square" the same
        values).  `dtype`: torch.float8_e4m3fn (default) or torch.float8_e5m2;
        `pow2` rounds the scales up to powers of two.  q's rows are padded to 16
        bytes; scales are (column blocks) x rows, or x row blocks."""
        torch = _torch()
        if stream is not None:  # results come from that stream's memory, free there and then
            with torch.cuda.stream(stream):
                return self.quantize(X, blocks, transposed, pow2, dtype)
        dt = _all_dtype_codes.get(X.dtype)
        if dt is None:
            raise TypeError(f"quantize takes bfloat16, float16 or float32 tensors, got {X.dtype}")
        if dtype is None:
            dtype = torch.float8_e4m3fn
        f8 = _fp8_codes.get(dtype)
        if f8 is None:
            raise TypeError(f"quantize makes float8_e4m3fn or float8_e5m2, got {dtype}")
        if blocks not in ("row", "square"):
            raise ValueError(f"blocks must be 'row' or 'square', got {blocks!r}")
        if X.get_device() != self.device:
            self._check_tensor("X", X)
        if X.dim() != 2:
            raise ValueError("X must be 2-D")
        rows, cols = X.shape
        ldx, unit = X.stride()
        if unit != 1 and cols > 1:
            raise ValueError("X must be row-major (unit stride along the last dim)")
        if rows <= 1:
            ldx = (cols + 7) & -8  # a single row has no next one
        square = blocks == "square"
        kb, rb = (cols + 127) >> 7, (rows + 127) >> 7
        per, per_t = (rb, kb) if square else (rows, cols)
        dev = X.device
        q = _padded_empty(rows, cols, dtype, dev, 16)
        s = torch.empty((kb, per), dtype=torch.float32, device=dev)
        result = (q, s)
        args_t = (None, 0, None, 0)
        if transposed:
            qt = _padded_empty(cols, rows, dtype, dev, 16)
            st = torch.empty((rb, per_t), dtype=torch.float32, device=dev)
            args_t = (qt.data_ptr(), (rows + 15) & -16, st.data_ptr(), per_t)
            result = (q, s, qt, st)
        rc = self.lib.bwgemm_quantize(self.handle, X.data_ptr(), dt, rows, cols, ldx,
                                      BLOCK_SQUARE if square else BLOCK_ROW, f8, int(pow2), q.data_ptr(),
                                      (cols + 15) & -16, s.data_ptr(), per, *args_t,
                                      torch._C._cuda_getCurrentRawStream(self.device))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_quantize")
        return result

    def gemm_scaled(self, A, scale_a, B, scale_b, out=None, out_dtype=None, accumulate: bool = False, stream=None):
        """``bwgemm_run_scaled``: ``out = A @ B.T`` of 8-bit CUDA tensors A (M x K) and
        B (N x K) with their block scales, as `quantize` returns them.  `out_dtype`:
        bf16 (default), fp16 or fp32; `accumulate` adds to an fp32 `out`."""
        torch = _torch()
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.gemm_scaled(A, scale_a, B, scale_b, out, out_dtype, accumulate)
        dev = self.device
        if (A.get_device() != dev or B.get_device() != dev or scale_a.get_device() != dev
                or scale_b.get_device() != dev):
            for name, t in (("A", A), ("scale_a", scale_a), ("B", B), ("scale_b", scale_b)):
                self._check_tensor(name, t)
        a, M, K = _pack_scaled(A, scale_a, "A")
        b, N, Kb = _pack_scaled(B, scale_b, "B")
        if Kb != K:
            raise ValueError(f"K mismatch: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs the out tensor to add to")
            if out_dtype is None:
                out_dtype = torch.bfloat16
            ldc = (N + 7) & -8
            out = _padded_empty(M, N, out_dtype, A.device, 8)
        else:
            self._check_tensor("out", out)
            if tuple(out.shape) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
                raise ValueError("out must be an M x N CUDA tensor of out_dtype")
            out_dtype = out.dtype
            ldc = _ld(out)
            if M <= 1:
                ldc = (N + 7) & -8  # a single row has no next one
        dt = _all_dtype_codes.get(out_dtype)
        if dt is None:
            raise TypeError(f"gemm_scaled writes bfloat16, float16 or float32, got {out_dtype}")
        rc = self.lib.bwgemm_run_scaled(self.handle, a, b, out.data_ptr(), M, N, K, ldc, dt,
                                        1 if accumulate else 0,
                                        torch._C._cuda_getCurrentRawStream(dev))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_run_scaled")
        return out

    def orthogonalize(self, G, out=None, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                      scale: float = 1.0, stream=None):
        """``bwgemm_orthogonalize``: the Newton-Schulz iteration on a CUDA matrix, or a
        stack of them (3-D), in bf16, fp16 or fp32.  `coefficients`: one triple
        (a, b, c) for every step, or one per step.  Returns `scale` times the
        result in bf16, or in `out` (bf16 or fp16, G's shape).  Operands are fp16, sums
        fp32: about 1e-3 off before the result's own rounding, whichever type it has."""
        torch = _torch()
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.orthogonalize(G, out, steps, coefficients, eps, scale)
        dt = _all_dtype_codes.get(G.dtype)
        if dt is None:
            raise TypeError(f"orthogonalize takes bfloat16, float16 or float32 tensors, got {G.dtype}")
        self._check_tensor("G", G)
        if G.dim() not in (2, 3):
            raise ValueError("G must be a matrix or a stack of matrices")
        if out is None:
            out = torch.empty(G.shape, dtype=torch.bfloat16, device=G.device)
        else:
            self._check_tensor("out", out)
            if out.shape != G.shape:
                raise ValueError("out must have G's shape")
        dto = _dtype_code(out)
        batch = G.shape[0] if G.dim() == 3 else 1
        rows, cols = G.shape[-2:]
        if cols > 1 and (G.stride(-1) != 1 or out.stride(-1) != 1):
            raise ValueError("G and out need unit stride along the last dim")
        # the true strides: rows closer than their length (expanded, overlapping) are refused
        lds = [int(t.stride(-2)) if rows > 1 else max(int(cols), 1) for t in (G, out)]
        strides = [int(t.stride(0)) if t.dim() == 3 else 0 for t in (G, out)]
        flat = [float(v) for v in coefficients] if not hasattr(coefficients[0], "__len__") else \
            [float(v) for triple in coefficients for v in triple]
        if len(flat) == 3:
            flat = flat * int(steps)
        if len(flat) != 3 * int(steps):
            raise ValueError("coefficients: one (a, b, c), or one for each step")
        need = ctypes.c_uint64()
        rc = self.lib.bwgemm_orthogonalize_workspace(batch, rows, cols, ctypes.byref(need))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_orthogonalize_workspace")
        ws = torch.empty(need.value, dtype=torch.uint8, device=G.device)
        rc = self.lib.bwgemm_orthogonalize(self.handle, G.data_ptr(), dt, out.data_ptr(), dto, batch, rows, cols,
                                           lds[0], strides[0], lds[1], strides[1], int(steps),
                                           (ctypes.c_float * len(flat))(*flat), float(eps), float(scale),
                                           ws.data_ptr(), need.value,
                                           torch._C._cuda_getCurrentRawStream(self.device))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_orthogonalize")
        return out

    def status(self, stream=None) -> int:
        """``bwgemm_get_status``: synchronises the stream, returns and clears the status."""
        return int(self.lib.bwgemm_get_status(self.handle, self._stream_handle(stream)))

    def last_device_status(self) -> int:
        return int(self.lib.bwgemm_last_device_status(self.handle))

    def last_config(self) -> dict:
        cfg = Config()
        rc = self.lib.bwgemm_plan_last_config(self.handle, ctypes.byref(cfg))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_plan_last_config")
        return cfg.as_dict()

    def launch_count(self) -> int:
        return int(self.lib.bwgemm_plan_launch_count(self.handle))

    def tune(self, A, B, out=None, iters: int = 10, stream=None) -> dict:
        """``bwgemm_tune``: time the candidate configurations on A, B, out and
        keep the fastest for this shape; returns its configuration.  `out`
        holds the product afterwards."""
        import torch
        dt = _dtype_code(A)
        if B.dtype != A.dtype or not (A.is_cuda and B.is_cuda):
            raise ValueError("A and B must be CUDA tensors of one dtype")
        M, K = A.shape
        N, _ = B.shape
        if out is None:
            out = torch.empty((M, N), dtype=A.dtype, device=A.device)
        self._check_device(A, B, out)
        cfg = Config()
        rc = self.lib.bwgemm_tune(self.handle, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K,
                                  _ld(A), _ld(B), _ld(out), dt, self._stream_handle(stream), int(iters),
                                  ctypes.byref(cfg))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_tune")
        return cfg.as_dict()

    def tuned_count(self) -> int:
        return int(self.lib.bwgemm_plan_tuned_count(self.handle))

    def read_trace(self):
        """Timeline of the last launch (plan created with trace=1): a
        (ctas, slots) numpy uint64 array of %globaltimer stamps in ns."""
        import numpy as np
        cap = 1 << 16
        buf = (ctypes.c_uint64 * cap)()
        ctas, slots = ctypes.c_int32(), ctypes.c_int32()
        rc = self.lib.bwgemm_plan_read_trace(self.handle, buf, cap, ctypes.byref(ctas),
                                             ctypes.byref(slots))
        if rc != 0:
            raise BwgemmError(rc, "bwgemm_plan_read_trace")
        n = ctas.value * slots.value
        return np.ctypeslib.as_array(buf)[:n].copy().reshape(ctas.value, slots.value)


# (device, thread, stream) -> the default plan of the module's functions there.  A plan
# serves one thread and one stream at a time: its launches share a workspace and a status
# word.  Plans stay (a captured graph may hold their workspace); a thread that takes
# over an ended one's identity takes its plans over too.
_plans: dict = {}


def _default_plan(t, stream=None) -> Plan:
    """The cached default plan of a CUDA tensor's device, for this thread and `stream`
    (the current one if None)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("bwgemm takes CUDA tensors (it has no host path)")
    if stream is None:
        handle = _torch()._C._cuda_getCurrentRawStream(dev)
    else:
        handle = stream.cuda_stream
    key = (dev, threading.get_ident(), handle)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans[key] = Plan(dev)
    return plan


def gemm(A, B, out=None, stream=None):
    """``A @ B.T`` with a cached default plan per device, thread and stream."""
    return _default_plan(A, stream).gemm(A, B, out=out, stream=stream)


def quantize(X, blocks="row", transposed=False, pow2=False, dtype=None, stream=None):
    """`Plan.quantize` with a cached default plan per device, thread and stream."""
    return _default_plan(X, stream).quantize(X, blocks, transposed, pow2, dtype, stream)


def gemm_scaled(A, scale_a, B, scale_b, out=None, out_dtype=None, accumulate=False, stream=None):
    """`Plan.gemm_scaled` with a cached default plan per device, thread and stream."""
    return _default_plan(A, stream).gemm_scaled(A, scale_a, B, scale_b, out, out_dtype, accumulate, stream)


def orthogonalize(G, out=None, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0, stream=None):
    """`Plan.orthogonalize` with a cached default plan per device, thread and stream."""
    return _default_plan(G, stream).orthogonalize(G, out, steps, coefficients, eps, scale, stream)

"""ctypes binding of libw8a16.so: argument marshalling only.

Every step of the operation runs in the library's CUDA kernels; this module only
turns torch tensors into pointers, pitches and a stream handle, and turns the
library's error codes into exceptions. There is no fallback: if the library is
not built or not loadable, every call raises.
"""
from __future__ import annotations

import ctypes
import re
from pathlib import Path

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "_build" / "libw8a16.so"
MARSHAL_PATH = PKG / "_build" / "w8a16_marshal.so"
HEADER = PKG.parent / "include" / "w8a16.h"

# Values mirrored from include/w8a16.h (checked against the header by the tests).
W8A16_OK = 0
FLAG_PDL = 1
VARIANT_AUTO, VARIANT_SIMT, VARIANT_TC, VARIANT_TC8, VARIANT_W8A8, VARIANT_PRESPLIT, VARIANT_GEMV = (
    0, 1, 2, 3, 4, 5, 6)
VARIANT_STREAM = 7
STATUS_OK, STATUS_WAIT_TIMEOUT = 0, 1
STATUS_BAD_INDEX = 2
WEIGHTS_F32, WEIGHTS_BF16 = 0, 1
ACT_BF16, ACT_F16 = 0, 1
NORM_RMS, NORM_LAYER = 0, 1


class Plan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("token_tile", ctypes.c_uint32),
                ("split_k", ctypes.c_uint32), ("stages", ctypes.c_uint32),
                ("ctas_per_sm", ctypes.c_uint32), ("grid", ctypes.c_uint32 * 3),
                ("block", ctypes.c_uint32 * 3), ("cluster", ctypes.c_uint32 * 3),
                ("smem_bytes", ctypes.c_uint32), ("tmem_cols", ctypes.c_uint32),
                ("tail_tiles", ctypes.c_uint32), ("tail_split", ctypes.c_uint32)]

    def as_dict(self) -> dict:
        return {"variant": self.variant, "token_tile": self.token_tile, "split_k": self.split_k,
                "stages": self.stages, "ctas_per_sm": self.ctas_per_sm, "grid": list(self.grid),
                "block": list(self.block), "cluster": list(self.cluster),
                "smem_bytes": self.smem_bytes, "tmem_cols": self.tmem_cols,
                "tail_tiles": self.tail_tiles, "tail_split": self.tail_split}


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64), ("num_pages", ctypes.c_uint32),
                ("page_size", ctypes.c_uint32), ("kv_heads", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32)]


class KvBatchDesc(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("page_table_stride", ctypes.c_int64), ("max_pages", ctypes.c_uint32),
                ("batch", ctypes.c_uint32), ("tokens", ctypes.c_uint32), ("max_q", ctypes.c_uint32)]


class HeadsDesc(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_uint32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_uint32),
                ("rotary_dim", ctypes.c_uint32), ("interleaved", ctypes.c_uint32)]


class KvSpanDesc(ctypes.Structure):
    _fields_ = [("window", ctypes.c_uint32), ("sinks", ctypes.c_uint32), ("prefix_pages", ctypes.c_void_p),
                ("num_prefix_pages", ctypes.c_uint32), ("prefix_len", ctypes.c_uint32)]


class RopeAxesDesc(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64), ("axes", ctypes.c_uint32),
                ("pair_axis", ctypes.c_uint8 * 128)]


class NormDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "residual", "residual_out", "out", "out_scale", "weight", "bias",
                                                "post_weight", "post_bias", "gate")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "residual_stride", "residual_out_stride", "out_stride",
                                                 "out_scale_stride", "gate_stride")]
                + [(n, ctypes.c_uint32) for n in ("M", "H", "gate_rows", "act_dtype", "residual_f32", "weight_f32", "kind")]
                + [("eps", ctypes.c_float), ("scale", ctypes.c_float)])


class W8A16Error(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"w8a16 error {code}: {message}")
        self.code = code


_VP, _U32, _I32, _INT = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int32, ctypes.c_int
_U64 = ctypes.c_uint64
_SIGS = {
    "w8a16_gemm": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32, _VP]),
    "w8a16_gemm_contiguous": (_INT, [_VP, _VP, _VP, _VP, _U32, _U32, _U32, _VP]),
    "w8a16_gemm_ex": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32, _U32, _VP]),
    "w8a16_gemm_host": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32, _VP, _VP, _VP,
                               _VP, _INT, _VP]),
    "w8a16_check_args": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32]),
    "w8a16_plan_for": (_INT, [_U32, _U32, _U32, _U32, ctypes.POINTER(_U32), ctypes.POINTER(Plan)]),
    "w8a16_plan_current": (_INT, [_U32, _U32, _U32, ctypes.POINTER(Plan)]),
    "w8a16_cluster_capacity": (_INT, [_I32, _U32, _U32, ctypes.POINTER(_U32)]),
    "w8a16_plan_variant": (_INT, [_U32, _U32, _U32, _I32, _U32, _U32, _U32, ctypes.POINTER(Plan)]),
    "w8a16_gemm_with_plan": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32,
                                    ctypes.POINTER(Plan), _U32, _VP]),
    "w8a16_quantize_weights": (_INT, [_VP, _U32, _U32, _U32, _U32, _VP, _VP, _VP]),
    "w8a16_quantize_activations": (_INT, [_VP, _U32, _U32, _U32, _VP, _VP, _U32, _VP]),
    "w8a16_workspace_bytes": (_U64, [_U32, _U32]),
    "w8a16_workspace_bytes_for": (_U64, [_U32, _U32, _U32]),
    "w8a16_plan_ws": (_INT, [_U32, _U32, _U32, _U64, ctypes.POINTER(Plan)]),
    "w8a16_gemm_noalloc": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32, _U32, _VP]),
    "w8a16_noalloc_scratch_bytes": (_U64, []),
    "w8a16_split_activations": (_INT, [_VP, _U32, _U32, _U32, _VP, _U64, _VP]),
    "w8a16_gemm_split_terms": (_INT, [_VP, _U64, _VP, _VP, _VP, _U32, _U32, _U32, _U32, _U32, _VP]),
    "w8a16_gemm_ws": (_INT, [_VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32, ctypes.POINTER(Plan), _VP,
                             _U64, _U32, _VP]),
    "w8a16_gemm_w8a8": (_INT, [_VP, _U32, _VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32, _U32, _U32,
                               _VP]),
    "w8a16_gemm_w8a8_with_plan": (_INT, [_VP, _U32, _VP, _U32, _VP, _VP, _VP, _U32, _U32, _U32,
                                         _U32, ctypes.POINTER(Plan), _U32, _VP]),
    "w8a16_kv_append": (_INT, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _U32]
                        + [ctypes.POINTER(HeadsDesc)] * 4 + [ctypes.POINTER(RopeDesc), _VP]),
    "w8a16_kv_append_axes": (_INT, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _U32]
                             + [ctypes.POINTER(HeadsDesc)] * 4
                             + [ctypes.POINTER(RopeDesc), ctypes.POINTER(RopeAxesDesc), _VP]),
    "w8a16_kv_attention": (_INT, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _U32,
                                  ctypes.POINTER(HeadsDesc), ctypes.POINTER(HeadsDesc), ctypes.c_float, _VP,
                                  _U64, _VP]),
    "w8a16_kv_attention_workspace_bytes": (_U64, [ctypes.POINTER(KvCacheDesc), _U32, _U32, _U32]),
    "w8a16_kv_attention_ex": (_INT, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _U32,
                                     ctypes.POINTER(HeadsDesc), ctypes.POINTER(HeadsDesc), ctypes.POINTER(KvSpanDesc),
                                     ctypes.c_float, _VP, _U64, _VP]),
    "w8a16_kv_attention_ex_workspace_bytes": (_U64, [ctypes.POINTER(KvCacheDesc), _U32, _U32, _U32, _U32]),
    "w8a16_gemm_w4": (_INT, [_VP, _U32, _U32, _VP, _VP, _U32, _VP, _U32, _VP, _U32, _U32, _U32, _U32, _U32, _VP]),
    "w8a16_norm_residual": (_INT, [ctypes.POINTER(NormDesc), _U32, _VP]),
    "w8a16_last_error": (ctypes.c_char_p, []),
    "w8a16_strerror": (ctypes.c_char_p, [_INT]),
    "w8a16_device_status": (_INT, [_VP, _INT, ctypes.POINTER(_U32), ctypes.POINTER(_U32),
                                   ctypes.POINTER(_U32)]),
    "w8a16_selftest_wait_timeout": (_INT, [_U32, _VP]),
    "w8a16_version": (ctypes.c_char_p, []),
}

_lib = None


def header_functions() -> list[str]:
    """Names of the functions include/w8a16.h declares."""
    text = HEADER.read_text()
    return sorted(set(re.findall(r"W8A16_API\s+(?:int|uint64_t|const char \*)\s*(w8a16_\w+)\s*\(", text)))


def load(path: Path | str | None = None):
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build it first (python -m fp8_weight_only_gemm_gb300.build "
                           "or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(str(p))
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def last_error() -> str:
    return load().w8a16_last_error().decode()


def strerror(code: int) -> str:
    return load().w8a16_strerror(code).decode()


def _check(rc: int):
    if rc != W8A16_OK:
        raise W8A16Error(rc, last_error() or strerror(rc))


def _stream_handle(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _new(stream, shape, dtype, device, *, kept=True, make=None):
    """A tensor that a call on `stream` makes for itself. torch's allocator gives a freed block away again
    behind the work of the stream that it was taken under, and of no other: under the current stream, a
    block whose last use there is still to come could be handed to kernels on `stream`, and a workspace
    dropped on return to others while they run. kept: returned to the caller, whose current stream
    may be where it is used when it is dropped."""
    import torch
    make = make or torch.empty
    device = torch.device(device)
    if stream is not None and device.type == "cuda":
        current, handle = torch.cuda.current_stream(device), _stream_handle(stream)
        if handle != int(current.cuda_stream):
            if not hasattr(stream, "cuda_stream"):
                stream = (torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device))
            with torch.cuda.stream(stream):
                t = make(shape, dtype=dtype, device=device)
            if kept:
                t.record_stream(current)
            return t
    return make(shape, dtype=dtype, device=device)


# -------------------------------------------------------------- pure host --
def check_args(M, N, K, a_row_stride, c_row_stride, A=0, W=0, scale=0, C=0) -> int:
    return load().w8a16_check_args(A or None, a_row_stride, W or None, scale or None, C or None,
                                   c_row_stride, M, N, K)


def plan_for(M, N, K, sm_count=152, cluster_ctas=None) -> dict:
    """Pure planner. cluster_ctas: optional 17-entry table (index = cluster size)
    of co-resident CTAs, as cluster_capacity() reports for a device."""
    p = Plan()
    tab = None
    if cluster_ctas is not None:
        tab = (_U32 * 17)(*[int(x) for x in cluster_ctas])
    _check(load().w8a16_plan_for(M, N, K, sm_count, tab, ctypes.byref(p)))
    return p.as_dict()


def plan_current(M, N, K) -> dict:
    """The plan w8a16_gemm uses on the current device."""
    p = Plan()
    _check(load().w8a16_plan_current(M, N, K, ctypes.byref(p)))
    return p.as_dict()


def plan_ws(M, N, K, workspace_bytes) -> dict:
    """The plan gemm_ws takes with a workspace of that many bytes (plan=None) on the
    current device."""
    p = Plan()
    _check(load().w8a16_plan_ws(M, N, K, workspace_bytes, ctypes.byref(p)))
    return p.as_dict()


def cluster_capacity(token_tile, stages, variant=VARIANT_TC) -> list[int]:
    out = (_U32 * 17)()
    _check(load().w8a16_cluster_capacity(variant, token_tile, stages, out))
    return list(out)


def plan_variant(M, N, K, variant=VARIANT_TC, split_k=0, stages=0, sm_count=152) -> Plan:
    p = Plan()
    _check(load().w8a16_plan_variant(M, N, K, variant, split_k, stages, sm_count, ctypes.byref(p)))
    return p


# ----------------------------------------------------------- device calls --
# The library sees plain pointers and cannot tell host memory, another device's
# memory or a short buffer from a good one; a kernel handed any of them would
# fault. So every tensor entry point checks placement, dtypes and extents here,
# before it calls the library.
_CODE_DTYPES = ("uint8", "float8_e4m3fn")


def _on_one_gpu(*tensors):
    dev = tensors[0].device
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("all tensors must be on a CUDA device")
        if t.device != dev:
            raise ValueError(f"all tensors must be on one device (got {dev} and {t.device})")


def _scale_shape(scale, N, K, name="block_scale"):
    """Block scales cover the [N, K] weights: [ceil(N/128), K/128]. Checked when K
    is a multiple of 128; otherwise the library reports K itself."""
    want = ((N + 127) // 128, K // 128)
    if K % 128 == 0 and tuple(scale.shape) != want:
        raise ValueError(f"{name} must be {list(want)} for N={N}, K={K}; got {list(scale.shape)}")


def _is_codes(t) -> bool:
    return str(t.dtype).rsplit(".", 1)[-1] in _CODE_DTYPES


def _shapes(A, W, scale, C):
    import torch
    if A.dim() != 2 or W.dim() != 2:
        raise ValueError("A and W must be 2-D")
    if A.dtype != torch.bfloat16:
        raise TypeError(f"A must be bfloat16, got {A.dtype}")
    if W.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"W must be uint8 E4M3 codes or float8_e4m3fn, got {W.dtype}")
    if scale.dtype != torch.float32:
        raise TypeError(f"block_scale must be float32, got {scale.dtype}")
    if A.stride(1) != 1 or (C is not None and C.stride(1) != 1):
        raise ValueError("A and C rows must be contiguous (stride 1 along K / N)")
    if not W.is_contiguous() or not scale.is_contiguous():
        raise ValueError("W and block_scale must be contiguous")
    M, K = A.shape
    N, Kw = W.shape
    if Kw != K:
        raise ValueError(f"A has K={K} columns, W has {Kw}")
    _scale_shape(scale, N, K)
    return M, N, K


def gemm(A, W, scale, C=None, *, stream=None, plan: Plan | None = None, flags: int = 0):
    """C[:, :N] = A @ dequant(W)^T on the GPU. A: bf16 [M, K] (any row pitch, rows
    contiguous); W: uint8/float8_e4m3fn [N, K]; scale: fp32 [ceil(N/128), K/128];
    C: optional bf16 [M, >=N] output view (allocated [M, N] if None)."""
    import torch
    M, N, K = _shapes(A, W, scale, C)
    if C is None:
        C = _new(stream, (M, N), torch.bfloat16, A.device)
    if C.dtype != torch.bfloat16 or C.shape[0] != M or C.shape[1] < N:
        raise ValueError("C must be bfloat16 [M, >=N]")
    _on_one_gpu(A, W, scale, C)
    lib = load()
    args = (A.data_ptr(), A.stride(0), W.data_ptr(), scale.data_ptr(), C.data_ptr(), C.stride(0),
            M, N, K)
    with torch.cuda.device(A.device):
        s = _stream_handle(stream)
        if plan is None:
            rc = lib.w8a16_gemm_ex(*args, flags, s)
        else:
            rc = lib.w8a16_gemm_with_plan(*args, ctypes.byref(plan), flags, s)
    _check(rc)
    return C


def workspace_bytes(M: int, K: int) -> int:
    """Workspace bytes of the pre-split path of gemm_ws at (M, K)."""
    return int(load().w8a16_workspace_bytes(M, K))


def workspace_bytes_for(M: int, N: int, K: int) -> int:
    """Workspace bytes with which gemm_ws takes its fastest plan at (M, N, K) on the
    current device."""
    return int(load().w8a16_workspace_bytes_for(M, N, K))


def gemm_ws(A, W, scale, C=None, *, workspace=None, stream=None, plan: Plan | None = None,
            flags: int = 0):
    """gemm() through w8a16_gemm_ws. workspace: a CUDA uint8 tensor, 16-byte aligned
    (workspace_bytes_for(M, N, K) bytes give the fastest plan; workspace_bytes(M, K)
    the pre-split plan above 16 tokens); None allocates one of the larger of the two
    with torch for this call (a caller that repeats calls should keep one); False
    passes none."""
    import torch
    M, N, K = _shapes(A, W, scale, C)
    if C is None:
        C = _new(stream, (M, N), torch.bfloat16, A.device)
    if C.dtype != torch.bfloat16 or C.shape[0] != M or C.shape[1] < N:
        raise ValueError("C must be bfloat16 [M, >=N]")
    _on_one_gpu(A, W, scale, C)
    if workspace is not None and workspace is not False:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        _on_one_gpu(A, workspace)
    lib = load()
    if workspace is None:
        with torch.cuda.device(A.device):
            need = max(workspace_bytes_for(M, N, K), workspace_bytes(M, K))
        workspace = _new(stream, max(16, need), torch.uint8, A.device, kept=False)
    ws_ptr, ws_bytes = (None, 0) if workspace is False else (workspace.data_ptr(), workspace.numel())
    with torch.cuda.device(A.device):
        rc = lib.w8a16_gemm_ws(A.data_ptr(), A.stride(0), W.data_ptr(), scale.data_ptr(), C.data_ptr(),
                               C.stride(0), M, N, K, ctypes.byref(plan) if plan is not None else None,
                               ws_ptr, ws_bytes, flags, _stream_handle(stream))
    _check(rc)
    return C


def gemm_noalloc(A, W, scale, C=None, *, stream=None, flags: int = 0):
    """gemm() through w8a16_gemm_noalloc (the library's fixed scratch buffer; calls
    must not overlap in time)."""
    import torch
    M, N, K = _shapes(A, W, scale, C)
    if C is None:
        C = _new(stream, (M, N), torch.bfloat16, A.device)
    if C.dtype != torch.bfloat16 or C.shape[0] != M or C.shape[1] < N:
        raise ValueError("C must be bfloat16 [M, >=N]")
    _on_one_gpu(A, W, scale, C)
    with torch.cuda.device(A.device):
        rc = load().w8a16_gemm_noalloc(A.data_ptr(), A.stride(0), W.data_ptr(), scale.data_ptr(),
                                       C.data_ptr(), C.stride(0), M, N, K, flags, _stream_handle(stream))
    _check(rc)
    return C


def gemm_noalloc_ptr(A_ptr, a_row_stride, W_ptr, scale_ptr, C_ptr, c_row_stride, M, N, K, stream=0,
                     flags: int = 0) -> int:
    """Raw-pointer w8a16_gemm_noalloc (returns the library's code; does not raise)."""
    return load().w8a16_gemm_noalloc(A_ptr or None, a_row_stride, W_ptr or None, scale_ptr or None,
                                     C_ptr or None, c_row_stride, M, N, K, flags, stream or None)


def noalloc_scratch_bytes() -> int:
    return int(load().w8a16_noalloc_scratch_bytes())


def gemm_ws_ptr(A_ptr, a_row_stride, W_ptr, scale_ptr, C_ptr, c_row_stride, M, N, K, ws_ptr, ws_bytes,
                stream=0, plan: Plan | None = None, flags: int = 0) -> int:
    """Raw-pointer w8a16_gemm_ws (returns the library's code; does not raise)."""
    return load().w8a16_gemm_ws(A_ptr or None, a_row_stride, W_ptr or None, scale_ptr or None, C_ptr or None,
                                c_row_stride, M, N, K, ctypes.byref(plan) if plan is not None else None,
                                ws_ptr or None, ws_bytes, flags, stream or None)


def split_activations(A, workspace=None, *, stream=None):
    """w8a16_split_activations: the two E4M3 terms of BF16 A [M, K] (row pitch A.stride(0))
    and their factors, written into `workspace` (a CUDA uint8 tensor of at least
    workspace_bytes(M, K) bytes; None allocates one with torch). Returns the workspace."""
    import torch
    if A.dim() != 2 or A.dtype != torch.bfloat16 or A.stride(1) != 1:
        raise ValueError("A must be a bfloat16 [M, K] tensor with unit column stride")
    M, K = A.shape
    if workspace is None:
        workspace = _new(stream, max(16, workspace_bytes(M, K)), torch.uint8, A.device)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _on_one_gpu(A, workspace)
    with torch.cuda.device(A.device):
        rc = load().w8a16_split_activations(A.data_ptr(), A.stride(0), M, K, workspace.data_ptr(),
                                            workspace.numel(), _stream_handle(stream))
    _check(rc)
    return workspace


def gemm_split_terms(workspace, M, W, scale, C=None, *, stream=None, flags: int = 0):
    """w8a16_gemm_split_terms: C [M, >=N] = the product of the activations that
    split_activations() wrote into `workspace` (for M tokens) with W and scale."""
    import torch
    if W.dim() != 2 or not _is_codes(W):
        raise ValueError("W must be a uint8 or float8_e4m3fn [N, K] tensor")
    N, K = W.shape
    _scale_shape(scale, N, K)
    if C is None:
        C = _new(stream, (M, N), torch.bfloat16, W.device)
    if C.dtype != torch.bfloat16 or C.shape[0] != M or C.shape[1] < N or C.stride(1) != 1:
        raise ValueError("C must be bfloat16 [M, >=N] with unit column stride")
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _on_one_gpu(workspace, W, scale, C)
    with torch.cuda.device(W.device):
        rc = load().w8a16_gemm_split_terms(workspace.data_ptr(), workspace.numel(), W.data_ptr(),
                                           scale.data_ptr(), C.data_ptr(), C.stride(0), M, N, K, flags,
                                           _stream_handle(stream))
    _check(rc)
    return C


def gemm_ptr(A_ptr, a_row_stride, W_ptr, scale_ptr, C_ptr, c_row_stride, M, N, K, stream=0,
             plan: Plan | None = None, flags: int = 0) -> int:
    """Raw-pointer call (returns the library's code; does not raise)."""
    lib = load()
    if plan is None:
        return lib.w8a16_gemm_ex(A_ptr, a_row_stride, W_ptr, scale_ptr, C_ptr, c_row_stride, M, N,
                                 K, flags, stream or None)
    return lib.w8a16_gemm_with_plan(A_ptr, a_row_stride, W_ptr, scale_ptr, C_ptr, c_row_stride,
                                    M, N, K, ctypes.byref(plan), flags, stream or None)


def gemm_host(A_host, W_host, scale_host, C_host, dA, dW, dScale, dC, *, copy_weights=True,
              stream=None):
    """Host-buffer call: the library queues H2D copies, the GEMM and the D2H copy.
    Host tensors should be pinned; the device buffers take A and C at the host
    tensors' row pitches (dA, dC), W as [N, K] and the scales at their shape."""
    import torch
    M, N, K = _shapes(A_host, W_host, scale_host, C_host)
    if C_host.dtype != torch.bfloat16 or C_host.shape[0] != M or C_host.shape[1] < N:
        raise ValueError("C_host must be bfloat16 [M, >=N]")
    if any(t.is_cuda for t in (A_host, W_host, scale_host, C_host)):
        raise ValueError("A_host, W_host, scale_host and C_host must be in host memory")
    _on_one_gpu(dA, dW, dScale, dC)
    for name, d, h, rows, cols in (("dA", dA, A_host, M, K), ("dC", dC, C_host, M, N)):
        if (d.dtype != torch.bfloat16 or d.dim() != 2 or d.stride(1) != 1 or d.stride(0) != h.stride(0)
                or d.shape[0] < rows or d.shape[1] < cols):
            raise ValueError(f"{name} must be bfloat16 with at least [{rows}, {cols}] at row pitch {h.stride(0)}")
    if not _is_codes(dW) or not dW.is_contiguous() or tuple(dW.shape) != (N, K):
        raise ValueError(f"dW must be contiguous E4M3 codes [{N}, {K}]")
    if dScale.dtype != torch.float32 or not dScale.is_contiguous() or dScale.shape != scale_host.shape:
        raise ValueError(f"dScale must be contiguous float32 {list(scale_host.shape)}")
    with torch.cuda.device(dA.device):
        rc = load().w8a16_gemm_host(
            A_host.data_ptr(), A_host.stride(0), W_host.data_ptr(), scale_host.data_ptr(),
            C_host.data_ptr(), C_host.stride(0), M, N, K, dA.data_ptr(), dW.data_ptr(),
            dScale.data_ptr(), dC.data_ptr(), 1 if copy_weights else 0, _stream_handle(stream))
    _check(rc)
    return C_host


def quantize_weights(W, *, stream=None):
    """(codes uint8 [N, K], block_scale float32 [ceil(N/128), K/128]) of a CUDA
    float32 or bfloat16 [N, K] weight tensor (rows contiguous, any row pitch)."""
    import torch
    if W.dim() != 2 or W.stride(1) != 1:
        raise ValueError("W must be 2-D with contiguous rows")
    if W.dtype == torch.float32:
        wt = WEIGHTS_F32
    elif W.dtype == torch.bfloat16:
        wt = WEIGHTS_BF16
    else:
        raise TypeError(f"W must be float32 or bfloat16, got {W.dtype}")
    if not W.is_cuda:
        raise ValueError("W must be on a CUDA device")
    N, K = W.shape
    codes = _new(stream, (N, K), torch.uint8, W.device)
    scale = _new(stream, ((N + 127) // 128, K // 128 if K % 128 == 0 else 1), torch.float32, W.device)
    with torch.cuda.device(W.device):
        rc = load().w8a16_quantize_weights(W.data_ptr(), wt, W.stride(0), N, K, codes.data_ptr(),
                                           scale.data_ptr(), _stream_handle(stream))
    _check(rc)
    return codes, scale


def quantize_activations(A, *, stream=None):
    """(codes uint8 [M, K], scales float32 [K/128, S]) of CUDA bfloat16 activations
    [M, K] (rows contiguous, any pitch); S = M rounded up to a multiple of 4, the
    columns past M unused."""
    import torch
    if A.dim() != 2 or A.stride(1) != 1 or A.dtype != torch.bfloat16 or not A.is_cuda:
        raise ValueError("A must be a CUDA bfloat16 [M, K] tensor with contiguous rows")
    M, K = A.shape
    S = (M + 3) // 4 * 4
    codes = _new(stream, (M, K), torch.uint8, A.device)
    scales = _new(stream, (max(K // 128, 1), S), torch.float32, A.device, make=torch.zeros)
    with torch.cuda.device(A.device):
        rc = load().w8a16_quantize_activations(A.data_ptr(), A.stride(0), M, K, codes.data_ptr(),
                                               scales.data_ptr(), S, _stream_handle(stream))
    _check(rc)
    return codes, scales


def gemm_w8a8(A_codes, a_scale, W, scale, C=None, *, stream=None, plan: Plan | None = None,
              flags: int = 0):
    """C[:, :N] (bf16) = (A_codes x a_scale) @ (W x block scales)^T on the GPU.
    A_codes: uint8 [M, K] (row pitch a multiple of 16 bytes); a_scale: float32
    [K/128, >=M] (row pitch a multiple of 4); W: uint8 [N, K]; scale: float32
    [ceil(N/128), K/128]; C: optional bf16 [M, >=N]."""
    import torch
    if A_codes.dim() != 2 or not _is_codes(A_codes) or A_codes.stride(1) != 1:
        raise ValueError("A_codes must be 2-D E4M3 codes (uint8 or float8_e4m3fn) with contiguous rows")
    M, K = A_codes.shape
    if (a_scale.dim() != 2 or a_scale.dtype != torch.float32 or a_scale.stride(1) != 1
            or a_scale.shape[0] < K // 128 or a_scale.shape[1] < M):
        raise ValueError(f"a_scale must be float32 with at least [{K // 128}, {M}] and contiguous rows")
    if W.dim() != 2 or not _is_codes(W) or not W.is_contiguous() or W.shape[1] != K:
        raise ValueError(f"W must be contiguous E4M3 codes [N, {K}]")
    N = W.shape[0]
    if scale.dtype != torch.float32 or not scale.is_contiguous():
        raise ValueError("block_scale must be contiguous float32")
    _scale_shape(scale, N, K)
    if C is None:
        C = _new(stream, (M, N), torch.bfloat16, A_codes.device)
    if C.dtype != torch.bfloat16 or C.dim() != 2 or C.stride(1) != 1 or C.shape[0] != M or C.shape[1] < N:
        raise ValueError("C must be bfloat16 [M, >=N] with contiguous rows")
    _on_one_gpu(A_codes, a_scale, W, scale, C)
    args = (A_codes.data_ptr(), A_codes.stride(0), a_scale.data_ptr(), a_scale.stride(0), W.data_ptr(),
            scale.data_ptr(), C.data_ptr(), C.stride(0), M, N, K)
    with torch.cuda.device(A_codes.device):
        s = _stream_handle(stream)
        if plan is None:
            rc = load().w8a16_gemm_w8a8(*args, flags, s)
        else:
            rc = load().w8a16_gemm_w8a8_with_plan(*args, ctypes.byref(plan), flags, s)
    _check(rc)
    return C


def gemm_w8a8_ptr(A_ptr, a_row_stride, a_scale_ptr, a_scale_stride, W_ptr, scale_ptr, C_ptr,
                  c_row_stride, M, N, K, stream=0, flags: int = 0) -> int:
    """Raw-pointer W8A8 call (returns the library's code; does not raise)."""
    return load().w8a16_gemm_w8a8(A_ptr or None, a_row_stride, a_scale_ptr or None, a_scale_stride,
                                  W_ptr or None, scale_ptr or None, C_ptr or None, c_row_stride, M, N,
                                  K, flags, stream or None)


def quantize_weights_ptr(W_ptr, w_dtype, w_row_stride, N, K, codes_ptr, scale_ptr, stream=0) -> int:
    """Raw-pointer call (returns the library's code; does not raise)."""
    return load().w8a16_quantize_weights(W_ptr or None, w_dtype, w_row_stride, N, K, codes_ptr or None,
                                         scale_ptr or None, stream or None)


# ------------------------------------------------- 8-bit paged key/value cache --
# These calls are short (a decode step's append runs for some 3 us). What they ask of their
# tensors, and the checks that only tensors allow, is in csrc/w8a16_marshal.cpp.
_marshal = None


def _load_marshal():
    global _marshal
    import importlib.machinery
    import importlib.util

    import torch  # noqa: F401  the module resolves torch's libraries, which this loads
    lib = load()
    if not MARSHAL_PATH.exists():
        raise RuntimeError(f"{MARSHAL_PATH} is missing: build it first (python -m fp8_weight_only_gemm_gb300.build "
                           "or __graft_entry__.build()); there is no fallback path")
    loader = importlib.machinery.ExtensionFileLoader("w8a16_marshal", str(MARSHAL_PATH))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("w8a16_marshal", loader))
    loader.exec_module(module)
    module.bind(*(ctypes.cast(fn, ctypes.c_void_p).value
                  for fn in (lib.w8a16_kv_append, lib.w8a16_kv_attention, lib.w8a16_gemm_w4,
                             lib.w8a16_norm_residual, lib.w8a16_kv_append_axes, lib.w8a16_kv_attention_ex)))
    _marshal = module
    return module


class KVCache:
    """A paged key/value cache in E4M3 with one float32 scale per page and head.

    k_codes, v_codes: uint8 or float8_e4m3fn [pages, kv_heads, page_size, head_dim] views
    with unit stride along head_dim and the same strides (a [pages, page_size, kv_heads,
    head_dim] pool is passed as its .transpose(1, 2)); k_scale, v_scale: float32
    [pages, kv_heads]. page_size a power of two in 16..256, head_dim a multiple of 16
    up to 256. The tensors are the caller's and are kept alive by the object."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        import torch
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            if t.dim() != 4 or not _is_codes(t) or t.stride(3) != 1:
                raise ValueError(f"{name} must be E4M3 codes [pages, kv_heads, page_size, head_dim] "
                                 "(uint8 or float8_e4m3fn) with unit stride along head_dim")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or tuple(t.shape) != tuple(k_codes.shape[:2]):
                raise ValueError(f"{name} must be float32 {list(k_codes.shape[:2])}")
        if k_codes.shape != v_codes.shape or k_codes.stride() != v_codes.stride():
            raise ValueError("k_codes and v_codes must have the same shape and strides")
        if k_scale.stride() != v_scale.stride():
            raise ValueError("k_scale and v_scale must have the same strides")
        _on_one_gpu(k_codes, v_codes, k_scale, v_scale)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k_codes.shape
        self._index = k_codes.get_device()
        self._desc = KvCacheDesc(
            k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            k_codes.stride(0), k_codes.stride(1), k_codes.stride(2), k_scale.stride(0), k_scale.stride(1),
            self.num_pages, self.page_size, self.kv_heads, self.head_dim)
        self._ref = ctypes.byref(self._desc)
        self._address = ctypes.addressof(self._desc)

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, device="cuda"):
        """A cache of zeroed pages [pages, kv_heads, page_size, head_dim]."""
        import torch
        kv = [torch.zeros(num_pages, kv_heads, page_size, head_dim, dtype=torch.uint8, device=device)
              for _ in range(2)]
        sc = [torch.zeros(num_pages, kv_heads, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*kv, *sc)


class RopeAxes:
    """Which axis (time, height, width; up to 4) turns each rotary pair of a head.

    pair_axis: the axis of pairs 0, 1, ..., a number for each; RopeAxes.sections gives the usual two orders."""

    def __init__(self, pair_axis):
        self.pair_axis = tuple(int(a) for a in pair_axis)
        if not 1 <= len(self.pair_axis) <= 128 or min(self.pair_axis) < 0 or max(self.pair_axis) > 3:
            raise ValueError("pair_axis must be 1 to 128 numbers in 0..3")
        self.pairs, self.axes = len(self.pair_axis), max(self.pair_axis) + 1
        self._table = (ctypes.c_uint8 * 128)(*self.pair_axis)
        self._address = ctypes.addressof(self._table)

    @classmethod
    def sections(cls, counts, cyclic=False):
        """counts[a] pairs for axis a: a block of pairs for each axis, or, cyclic, dealt in turn until an axis
        has its share."""
        left, out = [int(n) for n in counts], []
        if any(n < 0 for n in left):
            raise ValueError("counts must not be negative")
        while any(left):
            for a, n in enumerate(left):
                take = min(n, 1) if cyclic else n
                out += [a] * take
                left[a] -= take
        return cls(out)


def kv_append(cache, k, v, page_table, lens, cos=None, sin=None, *, q=None, q_out=None, cu_q=None, max_q=None,
              interleaved=False, positions=None, axes=None, stream=None):
    """w8a16_kv_append: writes this call's keys (rotated) and values to the cache, and
    returns the rotated queries.

    k, v: bf16 or fp16 [tokens, kv_heads, head_dim] (any token and head strides that are
    multiples of 8); q: [tokens, heads, head_dim] or None; q_out: where the rotated
    queries go (None: a new tensor; may be q itself). page_table: int32
    [batch, max_pages]; lens: int32 [batch], each sequence's length with the call's
    tokens, which are its last ones. Rows are split evenly among the sequences, or by
    cu_q (int32 [batch + 1] offsets) with max_q the most rows of one. cos, sin: float32
    [positions, rotary_dim / 2], rotary_dim a multiple of 16 up to head_dim (None: no
    rotation); pairs are (i, i + rotary_dim/2), or (2i, 2i + 1) if interleaved.

    positions with axes (a RopeAxes of rotary_dim / 2 pairs): the rows of cos and sin go not by the
    token's place in its sequence but by positions, int32 [axes, tokens], the row of each
    pair's axis (w8a16_kv_append_axes)."""
    if (positions is None) != (axes is None):
        raise ValueError("positions and axes go together: one of them is None")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    elif q_out is None:
        q_out = _new(stream, q.shape, q.dtype, q.device)
    args = (cache._address, cache._index, cache.head_dim, k, v, page_table, lens, cu_q, max_q, q, q_out, cos, sin,
            interleaved, stream if stream is None else _stream_handle(stream))
    if axes is None:
        rc = (_marshal or _load_marshal()).kv_append(*args)
    else:
        rc = (_marshal or _load_marshal()).kv_append_axes(*args, positions, axes.axes, axes.pairs, axes._address)
    if rc:
        _check(rc)
    return q_out


def kv_attention_workspace_bytes(cache, batch, max_q, heads, *, prefix_tokens=0) -> int:
    """Workspace bytes of kv_attention for `batch` sequences of up to `max_q` rows and
    `heads` query heads, on the cache's device. prefix_tokens: of calls with prefix_pages, the
    most rows of q (0: without a shared prefix)."""
    import torch
    with torch.cuda.device(cache._index):
        if prefix_tokens:
            n = int(load().w8a16_kv_attention_ex_workspace_bytes(cache._ref, 1, prefix_tokens, max_q, heads))
        else:
            n = int(load().w8a16_kv_attention_workspace_bytes(cache._ref, batch, max_q, heads))
    if n == 0:
        raise W8A16Error(-13, last_error())
    return n


def kv_attention(cache, q, page_table, lens, out=None, *, softmax_scale=None, cu_q=None, max_q=None,
                 window=None, sinks=0, prefix_pages=None, prefix_len=0, workspace=None, stream=None):
    """w8a16_kv_attention: causal attention of q [tokens, heads, head_dim] (bf16 or fp16,
    already rotated) over the sequences' cached keys and values, the call's own tokens
    (kv_append) included. page_table, lens, cu_q, max_q as in kv_append; softmax_scale
    defaults to head_dim ** -0.5. workspace: a CUDA uint8 tensor of
    kv_attention_workspace_bytes(...) bytes that no concurrent call uses (None allocates
    one for this call). Returns out, [tokens, heads, head_dim] of q's dtype.

    window: a query sees the last `window` keys up to its own, and the sequence's first `sinks`
    ones; pages that no query of the call sees a key of are not read, nor are their entries of
    page_table. prefix_pages, int32 [pages], with prefix_len: the first prefix_len positions of
    every sequence lie on these pages and are read once for all of them; page_table is
    read for the positions behind. (Where those are many more than the prefix, a call without,
    whose page_table names all pages, is the faster one.) Not both (w8a16_kv_attention_ex)."""
    if out is None:
        out = _new(stream, q.shape, q.dtype, q.device)
    if workspace is None:
        import torch
        B = page_table.shape[0]
        most = max_q if max_q is not None else -(-q.shape[0] // max(B, 1))
        shared = {} if prefix_pages is None else {"prefix_tokens": max(q.shape[0], 1)}
        workspace = _new(stream, kv_attention_workspace_bytes(cache, B, most, q.shape[1], **shared), torch.uint8, q.device, kept=False)
    args = (cache._address, cache._index, cache.head_dim, q, out, page_table, lens, cu_q, max_q,
            cache.head_dim ** -0.5 if softmax_scale is None else softmax_scale, workspace,
            stream if stream is None else _stream_handle(stream))
    if window is None and prefix_pages is None and not sinks and not prefix_len:
        rc = (_marshal or _load_marshal()).kv_attention(*args)
    else:
        if window == 0:
            raise ValueError("window must be at least 1 (None: no window)")
        rc = (_marshal or _load_marshal()).kv_attention_ex(*args, 0 if window is None else window, sinks, prefix_pages, prefix_len)
    if rc:
        _check(rc)
    return out


# ------------------------------------------------------------ 4-bit weights --
def gemm_w4(A, W, scale, C=None, *, zeros=None, stream=None, flags: int = 0):
    """w8a16_gemm_w4: C[:, :N] = A @ ((codes - zeros) * scale)^T for a few tokens.
    A: bf16 or fp16 [M, K] (any row pitch that is a multiple of 8); W: uint8 [N, K/2], code
    2j in the low half of byte j and 2j + 1 in its high half; scale: float32 or A's
    dtype, [N, K/group] with group 32, 64 or 128 (taken from its shape); zeros: uint8
    [N, K/group], 0..15 (None: 8); C: optional [M, >=N] of A's dtype."""
    if C is None:
        C = _new(stream, (A.shape[0], W.shape[0]), A.dtype, A.device)
    rc = (_marshal or _load_marshal()).gemm_w4(A, W, scale, C, zeros, flags,
                                               stream if stream is None else _stream_handle(stream))
    if rc:
        _check(rc)
    return C


# ------------------------------------------------- the norms around a block --
def norm_residual(x, residual=None, weight=None, *, bias=None, post_weight=None, post_bias=None, gate=None, scale=1.0,
                  eps=1e-6, kind="rms", out=None, residual_out=None, quantize=False, stream=None, flags: int = 0):
    """w8a16_norm_residual: (y, h) with t = norm(x; post_weight, post_bias) or x,
    h = residual + scale * gate * t, y = norm(h; weight, bias).

    x: bf16 or fp16 [M, H] (any row pitch that is a multiple of 8), H a multiple of 8 up to
    32768. residual: [M, H] of x's type or float32, or None; residual_out: where h goes, of
    residual's type (None: a new tensor; may be residual itself). weight, bias, post_weight,
    post_bias: [H], all of x's type or all float32; without weight there is no y (None).
    gate: [rows, H] of x's type, rows a divisor of M: row m takes gate row m // (M // rows). kind: "rms"
    or "layer", for both norms. out: where y goes (None: a new tensor; may be x itself). quantize: y
    is (codes uint8 [M, H], scales float32 [H/128, S >= M]) as quantize_activations gives and
    gemm_w8a8 takes them, and so is out; H is then a multiple of 128."""
    import torch
    if kind not in ("rms", "layer"):
        raise ValueError(f"kind must be 'rms' or 'layer', got {kind!r}")
    if quantize and weight is None:
        raise ValueError("quantize without weight: there is no y to quantise")
    if residual_out is None:
        residual_out = _new(stream, x.shape, x.dtype if residual is None else residual.dtype, x.device)
    codes, scales = out if quantize and out is not None else (out, None)
    if weight is not None and codes is None:
        if quantize:
            M, H = x.shape
            codes = _new(stream, (M, H), torch.uint8, x.device)
            scales = _new(stream, (max(H // 128, 1), max((M + 3) // 4 * 4, 4)), torch.float32, x.device, make=torch.zeros)
        else:
            codes = _new(stream, x.shape, x.dtype, x.device)
    rc = (_marshal or _load_marshal()).norm_residual(
        x, residual, codes, scales, residual_out, weight, bias, post_weight, post_bias, gate, scale, eps,
        NORM_LAYER if kind == "layer" else NORM_RMS, flags, stream if stream is None else _stream_handle(stream))
    if rc:
        _check(rc)
    return ((codes, scales) if quantize else codes), residual_out


def device_status(stream=None, clear=False) -> tuple[int, int, int]:
    st, wh, de = ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_uint32()
    _check(load().w8a16_device_status(_stream_handle(stream), 1 if clear else 0, ctypes.byref(st),
                                      ctypes.byref(wh), ctypes.byref(de)))
    return st.value, wh.value, de.value


def selftest_wait_timeout(timeout_us: int, stream=None):
    _check(load().w8a16_selftest_wait_timeout(timeout_us, _stream_handle(stream)))


def version() -> str:
    return load().w8a16_version().decode()

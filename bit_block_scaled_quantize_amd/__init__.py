"""Thin Python binding of libnvfp4 (include/nvfp4.h): NVFP4 quantization and block-scaled
GEMMs on MI355X.

Every function marshals torch tensors (device memory, current stream) into the C ABI and
returns; all arithmetic runs in the HIP kernels. If the library is not built the import
still succeeds but every call raises, so nothing can silently fall back to another path.

Names follow the C entry points: quantize, quantize_noalloc, rht_quantize, rht_rows_quantize,
gemm, gemm_ex, grouped_gemm, grouped_gemm_k, amax, amax_pair, mx_quantize, mx_quantize_columns, mx_gemm, dequantize,
gemm_act, act_grad, moe_tokens, adamw.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

NVFP4_OK = 0
_STATUS = {-1: "invalid argument", -2: "unsupported", -3: "workspace", -4: "HIP error"}
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_BLOCK = {"1x16": 0, "16x16": 1}
_ROUND = {"rn": 0, "sr": 1}
OP_QUANTIZE, OP_RHT_QUANTIZE, OP_GEMM, OP_GROUPED_GEMM, OP_AMAX_PAIR, OP_GEMM_EX = 0, 1, 2, 3, 4, 5
OP_ADAMW, OP_GEMM_ACT, OP_ACT_GRAD = 6, 7, 8
SCORES = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"none": 0, "relu2": 1, "gelu": 2, "silu": 3}
OUT_FP32, OUT_FP32_ACCUMULATE, OUT_BF16 = 0, 1, 2

EXPORTED = ("nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_rht_quantize", "nvfp4_gemm", "nvfp4_gemm_ex", "nvfp4_grouped_gemm",
            "mxfp4_quantize", "mxfp4_quantize_columns", "mxfp4_gemm", "nvfp4_rht_rows_quantize",
            "nvfp4_grouped_gemm_k",
            "nvfp4_amax", "nvfp4_amax_pair", "nvfp4_workspace_size", "nvfp4_last_error",
            "nvfp4_dequantize", "nvfp4_gemm_act", "nvfp4_act_grad", "nvfp4_moe_tokens",
            "nvfp4_moe_workspace_size", "nvfp4_adamw", "nvfp4_adamw_table", "nvfp4_adamw_table_size")


class NVFP4Error(RuntimeError):
    pass


class _CTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class _CMXTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class _CMoE(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int64), ("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64),
                ("top_k", ctypes.c_int64), ("router", ctypes.c_void_p), ("router_dt", ctypes.c_int),
                ("w1", _CTensor), ("w2", _CTensor), ("act", ctypes.c_int), ("gated", ctypes.c_int),
                ("score", ctypes.c_int), ("renormalize", ctypes.c_int), ("routed_scale", ctypes.c_float)]


class _CAdamWTensor(ctypes.Structure):
    _fields_ = ([("n", ctypes.c_int64)]
                + [(k, ctypes.c_void_p) for k in ("grad", "p", "p_out", "w_out", "m", "v", "m_out", "v_out",
                                                  "m_scale", "v_scale", "m_scale_out", "v_scale_out")]
                + [("weight_decay", ctypes.c_float), ("grad_dt", ctypes.c_int)])


class _CAdamWHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("max_norm", ctypes.c_double),
                ("seed", ctypes.c_uint64)]


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise NVFP4Error(f"{LIB_PATH} is not built; run bit_block_scaled_quantize_amd.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, u64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    pt = ctypes.POINTER(_CTensor)
    lib.nvfp4_quantize.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_int, ctypes.c_int,
                                   u64, u64, vp, i64, vp, pt, pt, vp, sz, vp]
    lib.nvfp4_quantize_noalloc.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_int, ctypes.c_int,
                                           u64, u64, vp, i64, vp, pt, pt, vp]
    lib.nvfp4_rht_quantize.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_uint16,
                                       ctypes.c_int, u64, u64, vp, i64, vp, pt, vp, sz, vp]
    lib.nvfp4_gemm.argtypes = [pt, pt, vp, i64, vp]
    mpt = ctypes.POINTER(_CMXTensor)
    lib.mxfp4_quantize.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_int, u64, u64, mpt, vp]
    lib.mxfp4_quantize_columns.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_int, u64, u64, mpt, vp]
    lib.mxfp4_gemm.argtypes = [mpt, mpt, vp, i64, vp]
    lib.nvfp4_rht_rows_quantize.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_uint16, ctypes.c_int,
                                            u64, u64, vp, pt, vp, sz, vp]
    lib.nvfp4_gemm_ex.argtypes = [pt, pt, vp, i64, ctypes.c_int, vp, vp, sz, vp]
    lib.nvfp4_gemm_act.argtypes = [pt, pt, vp, i64, vp, ctypes.c_int, ctypes.c_int, vp, i64, vp, i64, vp, vp, sz, vp]
    lib.nvfp4_act_grad.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i64, ctypes.c_int, vp, i64, vp, ctypes.c_int,
                                   vp, sz, vp]
    lib.nvfp4_grouped_gemm.argtypes = [i64, vp, pt, pt, i64, vp, i64, vp, sz, vp]
    lib.nvfp4_grouped_gemm_k.argtypes = [i64, vp, pt, pt, vp, i64, vp]
    lib.nvfp4_amax.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i64, ctypes.c_int,
                               ctypes.c_uint16, vp, vp, sz, vp]
    lib.nvfp4_amax_pair.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_uint16, vp, vp, sz, vp]
    lib.nvfp4_workspace_size.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.nvfp4_workspace_size.restype = sz
    lib.nvfp4_last_error.restype = ctypes.c_char_p
    lib.nvfp4_dequantize.argtypes = [pt, vp, i64, vp, vp]
    lib.nvfp4_moe_tokens.argtypes = [ctypes.POINTER(_CMoE), vp, i64, i64, vp, i64, vp, vp, vp, sz, vp]
    lib.nvfp4_moe_workspace_size.argtypes = [ctypes.POINTER(_CMoE), i64]
    lib.nvfp4_moe_workspace_size.restype = sz
    lib.nvfp4_adamw_table_size.argtypes = [ctypes.POINTER(_CAdamWTensor), i64]
    lib.nvfp4_adamw_table_size.restype = sz
    lib.nvfp4_adamw_table.argtypes = [ctypes.POINTER(_CAdamWTensor), i64, ctypes.c_int, vp, sz, ctypes.POINTER(i64)]
    lib.nvfp4_adamw.argtypes = [vp, i64, i64, ctypes.c_int, ctypes.POINTER(_CAdamWHyper), vp, vp, vp, sz, vp]
    for name in EXPORTED:
        if name not in ("nvfp4_workspace_size", "nvfp4_last_error", "nvfp4_adamw_table_size", "nvfp4_moe_workspace_size"):
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def library():
    """The loaded ctypes library (raises NVFP4Error if it is not built)."""
    return _load()


def _check(status: int):
    if status != NVFP4_OK:
        msg = _load().nvfp4_last_error().decode()
        raise NVFP4Error(f"{_STATUS.get(status, status)}: {msg}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _on_stream(fn):
    """Runs a binding function with its `stream` argument (when given) as torch's current
    stream, so every workspace and default output it allocates belongs to the stream its
    kernels are enqueued on. torch's caching allocator hands a freed block out again only to
    work on the stream it belongs to, so a workspace freed when the function returns cannot be
    given to other work while these kernels may still be using it."""
    names = list(inspect.signature(fn).parameters)
    at = names.index("stream")

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapper


@dataclass
class NVFP4Tensor:
    """Device buffers of one NVFP4 tensor [rows, cols] quantized along cols."""
    codes: torch.Tensor         # uint8 [rows, cols/2]
    scales: torch.Tensor        # uint8 [rows, cols/16] (E4M3 codes)
    global_scale: torch.Tensor  # float32 [nseg]
    rows: int
    cols: int

    @classmethod
    def empty(cls, rows: int, cols: int, nseg: int = 1, device="cuda"):
        return cls(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty((rows, cols // 16), dtype=torch.uint8, device=device),
                   torch.empty((nseg,), dtype=torch.float32, device=device), rows, cols)

    def c(self) -> _CTensor:
        return _CTensor(self.codes.data_ptr(), self.scales.data_ptr(),
                        self.global_scale.data_ptr(), self.rows, self.cols)


@dataclass
class MXFP4Tensor:
    """Device buffers of one MXFP4 tensor [rows, cols] quantized along cols. The E8M0 scales
    are stored K step by K step: [ceil(cols/128), rows, 4], scale j of row r at [j // 4, r,
    j % 4] (one 128-element step's scales of all rows contiguous, as the GEMM reads them)."""
    codes: torch.Tensor         # uint8 [rows, cols/2]
    scales: torch.Tensor        # uint8 [ceil(cols/128), rows, 4] (E8M0 codes)
    rows: int
    cols: int

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        return cls(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty(((cols + 127) // 128, rows, 4), dtype=torch.uint8, device=device), rows, cols)

    def scales_by_row(self) -> torch.Tensor:
        """The scales as [rows, cols/32] (row r's j-th scale at [r, j]), a copy."""
        steps = (self.cols + 127) // 128
        s = self.scales.reshape(steps, self.rows, 4).permute(1, 0, 2).reshape(self.rows, steps * 4)
        return s[:, : self.cols // 32].contiguous()

    def c(self) -> _CMXTensor:
        return _CMXTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)


def _input(x: torch.Tensor):
    if x.dtype not in _DTYPE:
        raise NVFP4Error(f"unsupported input dtype {x.dtype}")
    if x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda:
        raise NVFP4Error("input must be a 2-D GPU tensor with unit column stride")
    return _DTYPE[x.dtype], x.shape[0], x.shape[1], x.stride(0)


def _check_q(q, nseg: int = 1, what: str = "tensor"):
    """The C ABI sees only pointers: make sure the torch buffers behind an NVFP4/MXFP4 tensor
    are as large as its rows and cols say (and contiguous), so no kernel writes past them."""
    mx = isinstance(q, MXFP4Tensor)
    need = ((q.codes, q.rows * (q.cols // 2)),
            (q.scales, q.rows * 4 * ((q.cols + 127) // 128) if mx else q.rows * (q.cols // 16)))
    if not mx:
        need += ((q.global_scale, nseg),)
    for t, n in need:
        if t.numel() < n or not t.is_contiguous() or not t.is_cuda:
            raise NVFP4Error(f"{what}: buffer of {t.numel()} elements (contiguous, on the GPU) needed {n}")


def _check_out(out: torch.Tensor, rows: int, cols: int, dtype, what: str = "out"):
    """A 2-D output with at least rows x cols elements, unit column stride, the given dtype."""
    if out.dtype != dtype or out.dim() != 2 or out.stride(1) != 1 or not out.is_cuda:
        raise NVFP4Error(f"{what} must be a 2-D {dtype} GPU tensor with unit column stride")
    if out.shape[0] < rows or out.shape[1] < cols:
        raise NVFP4Error(f"{what} shape {tuple(out.shape)} smaller than ({rows}, {cols})")


def _row_stride(t: torch.Tensor) -> int:
    """Elements from one row to the next; a single row may have any stride in torch."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _check_table(t, what: str):
    """Segment / offset tables are int64 GPU tensors with at least two entries."""
    if t is not None and (t.dtype != torch.int64 or t.device.type != "cuda" or t.numel() < 2
                          or not t.is_contiguous()):
        raise NVFP4Error(f"{what} must be a contiguous int64 GPU tensor of at least 2 entries")


def _check_vec(t, n: int, what: str):
    if t is not None and (t.dtype != torch.float32 or t.numel() < n or not t.is_cuda
                          or not t.is_contiguous()):
        raise NVFP4Error(f"{what} must be a contiguous float32 GPU tensor of at least {n} elements")


def workspace_size(op: int, rows: int, cols: int, nseg: int = 1) -> int:
    return int(_load().nvfp4_workspace_size(op, rows, cols, nseg))


def _given_workspace(workspace: torch.Tensor) -> int:
    """Bytes of a caller's workspace."""
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise NVFP4Error("workspace must be a contiguous GPU tensor")
    return workspace.numel() * workspace.element_size()


def _workspace(op, rows, cols, nseg, device):
    n = workspace_size(op, rows, cols, nseg)
    return torch.empty((max(n, 1),), dtype=torch.uint8, device=device), n


@_on_stream
def quantize(x: torch.Tensor, block: str = "1x16", rounding: str = "rn", seed: int = 0,
             offset: int = 0, segments: torch.Tensor | None = None, amax: torch.Tensor | None = None,
             emit_transposed: bool = False, out: NVFP4Tensor | None = None,
             out_t: NVFP4Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """nvfp4_quantize. Returns (q, q_t) where q_t is None unless emit_transposed."""
    lib = _load()
    dt, rows, cols, ld = _input(x)
    nseg = 1 if segments is None else segments.numel() - 1
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, nseg, x.device)
    if emit_transposed and out_t is None:
        # a segmented stack of nseg equal blocks: each block's transpose, stacked
        out_t = (NVFP4Tensor.empty(cols, rows, 1, x.device) if segments is None
                 else NVFP4Tensor.empty(nseg * cols, rows // nseg, nseg, x.device))
    ws_n = 0
    if amax is None:
        if workspace is None:
            workspace, ws_n = _workspace(OP_QUANTIZE, rows, cols, nseg, x.device)
        else:
            ws_n = _given_workspace(workspace)
    _check_table(segments, "segments")
    _check_vec(amax, nseg, "amax")
    _check_q(out, nseg, "out")
    if emit_transposed:
        _check_q(out_t, nseg if segments is not None else 1, "out_t")
    oc = out.c()
    otc = out_t.c() if emit_transposed else None
    st = lib.nvfp4_quantize(_ptr(x), dt, rows, cols, ld, _BLOCK[block], _ROUND[rounding],
                            seed & (2 ** 64 - 1), offset & (2 ** 64 - 1), _ptr(segments), nseg,
                            _ptr(amax), ctypes.byref(oc),
                            ctypes.byref(otc) if otc is not None else None,
                            _ptr(workspace) if amax is None else None, ws_n, _stream(stream))
    _check(st)
    return out, (out_t if emit_transposed else None)


@_on_stream
def quantize_noalloc(x: torch.Tensor, block: str = "1x16", rounding: str = "rn", seed: int = 0,
                     offset: int = 0, segments: torch.Tensor | None = None, amax: torch.Tensor | None = None,
                     emit_transposed: bool = False, out: NVFP4Tensor | None = None,
                     out_t: NVFP4Tensor | None = None, stream=None):
    """nvfp4_quantize_noalloc: nvfp4_quantize without a workspace (the library's static device
    array holds the amax partials). With `out` (and `out_t` when emit_transposed) given, this
    allocates nothing; calls overlapping on one device race. Returns (q, q_t)."""
    lib = _load()
    dt, rows, cols, ld = _input(x)
    nseg = 1 if segments is None else segments.numel() - 1
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, nseg, x.device)
    if emit_transposed and out_t is None:
        out_t = (NVFP4Tensor.empty(cols, rows, 1, x.device) if segments is None
                 else NVFP4Tensor.empty(nseg * cols, rows // nseg, nseg, x.device))
    _check_table(segments, "segments")
    _check_vec(amax, nseg, "amax")
    _check_q(out, nseg, "out")
    if emit_transposed:
        _check_q(out_t, nseg if segments is not None else 1, "out_t")
    oc = out.c()
    otc = out_t.c() if emit_transposed else None
    st = lib.nvfp4_quantize_noalloc(_ptr(x), dt, rows, cols, ld, _BLOCK[block], _ROUND[rounding],
                                    seed & (2 ** 64 - 1), offset & (2 ** 64 - 1), _ptr(segments), nseg,
                                    _ptr(amax), ctypes.byref(oc),
                                    ctypes.byref(otc) if otc is not None else None, _stream(stream))
    _check(st)
    return out, (out_t if emit_transposed else None)


@_on_stream
def rht_rows_quantize(x: torch.Tensor, sign_mask: int, rounding: str = "rn", seed: int = 0,
                      offset: int = 0, amax: torch.Tensor | None = None, out: NVFP4Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """nvfp4_rht_rows_quantize: each row's 16-blocks through the random-sign Hadamard
    transform, then 1x16 quantization along the rows (same shape as x)."""
    lib = _load()
    dt, rows, cols, ld = _input(x)
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, 1, x.device)
    ws_n = 0
    if amax is None:
        if workspace is None:
            workspace, ws_n = _workspace(OP_QUANTIZE, rows, cols, 1, x.device)
        else:
            ws_n = _given_workspace(workspace)
    _check_vec(amax, 1, "amax")
    _check_q(out, 1, "out")
    oc = out.c()
    _check(lib.nvfp4_rht_rows_quantize(_ptr(x), dt, rows, cols, ld, sign_mask & 0xFFFF, _ROUND[rounding],
                                       seed & (2 ** 64 - 1), offset & (2 ** 64 - 1), _ptr(amax),
                                       ctypes.byref(oc), _ptr(workspace) if amax is None else None, ws_n,
                                       _stream(stream)))
    return out


@_on_stream
def mx_quantize(x: torch.Tensor, rounding: str = "rn", seed: int = 0, offset: int = 0,
                out: MXFP4Tensor | None = None, stream=None) -> MXFP4Tensor:
    """mxfp4_quantize: x[rows, cols] -> MXFP4 (E8M0 scale per 32 elements)."""
    lib = _load()
    dt, rows, cols, ld = _input(x)
    if out is None:
        out = MXFP4Tensor.empty(rows, cols, x.device)
    _check_q(out, what="out")
    oc = out.c()
    _check(lib.mxfp4_quantize(_ptr(x), dt, rows, cols, ld, _ROUND[rounding], seed & (2 ** 64 - 1),
                              offset & (2 ** 64 - 1), ctypes.byref(oc), _stream(stream)))
    return out


@_on_stream
def mx_quantize_columns(x: torch.Tensor, rounding: str = "rn", seed: int = 0, offset: int = 0,
                        out: MXFP4Tensor | None = None, stream=None) -> MXFP4Tensor:
    """mxfp4_quantize_columns: x[rows, cols] -> MXFP4 of x^T, [cols, rows] (E8M0 per 32 rows)."""
    lib = _load()
    dt, rows, cols, ld = _input(x)
    if out is None:
        out = MXFP4Tensor.empty(cols, rows, x.device)
    _check_q(out, what="out")
    oc = out.c()
    _check(lib.mxfp4_quantize_columns(_ptr(x), dt, rows, cols, ld, _ROUND[rounding], seed & (2 ** 64 - 1),
                                      offset & (2 ** 64 - 1), ctypes.byref(oc), _stream(stream)))
    return out


@_on_stream
def mx_gemm(a: MXFP4Tensor, b: MXFP4Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mxfp4_gemm: D[M, N] = A[M, K] * B[N, K]^T (FP32) on the block-scaled FP4 matrix cores."""
    lib = _load()
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.float32, device=a.codes.device)
    _check_q(a, what="A")
    _check_q(b, what="B")
    _check_out(out, a.rows, b.rows, torch.float32)
    ac, bc = a.c(), b.c()
    _check(lib.mxfp4_gemm(ctypes.byref(ac), ctypes.byref(bc), _ptr(out), out.stride(0), _stream(stream)))
    return out


@_on_stream
def rht_quantize(x: torch.Tensor, sign_mask: int, rounding: str = "rn", seed: int = 0,
                 offset: int = 0, amax: torch.Tensor | None = None,
                 out: NVFP4Tensor | None = None, workspace: torch.Tensor | None = None,
                 segments: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """nvfp4_rht_quantize: x[tokens, cols] -> NVFP4 tensor [cols, tokens] (segments: token
    ranges with one global scale each)."""
    lib = _load()
    dt, tokens, cols, ld = _input(x)
    nseg = 1 if segments is None else segments.numel() - 1
    if out is None:
        out = NVFP4Tensor.empty(cols, tokens, nseg, x.device)
    ws_n = 0
    if amax is None:
        if workspace is None:
            workspace, ws_n = _workspace(OP_RHT_QUANTIZE, tokens, cols, nseg, x.device)
        else:
            ws_n = _given_workspace(workspace)
    _check_table(segments, "segments")
    _check_vec(amax, nseg, "amax")
    _check_q(out, nseg, "out")
    oc = out.c()
    st = lib.nvfp4_rht_quantize(_ptr(x), dt, tokens, cols, ld, sign_mask & 0xFFFF,
                                _ROUND[rounding], seed & (2 ** 64 - 1), offset & (2 ** 64 - 1),
                                _ptr(segments), nseg, _ptr(amax), ctypes.byref(oc),
                                _ptr(workspace) if amax is None else None, ws_n, _stream(stream))
    _check(st)
    return out


@_on_stream
def gemm(a: NVFP4Tensor, b: NVFP4Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_gemm: D[M, N] = A[M, K] * B[N, K]^T (FP32)."""
    lib = _load()
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.float32, device=a.codes.device)
    _check_q(a, what="A")
    _check_q(b, what="B")
    _check_out(out, a.rows, b.rows, torch.float32)
    ac, bc = a.c(), b.c()
    _check(lib.nvfp4_gemm(ctypes.byref(ac), ctypes.byref(bc), _ptr(out), out.stride(0),
                          _stream(stream)))
    return out


@_on_stream
def gemm_ex(a: NVFP4Tensor, b: NVFP4Tensor, out: torch.Tensor | None = None,
            out_dtype: torch.dtype = torch.float32, accumulate: bool = False,
            amax_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """nvfp4_gemm_ex: D = A * B^T stored as float32 or bfloat16, or (accumulate, float32) added
    to `out`; amax_out (float32 [1]) receives max |D| as stored."""
    lib = _load()
    if accumulate:
        if out is None or out.dtype != torch.float32:
            raise NVFP4Error("accumulate needs a float32 `out`")
        kind = OUT_FP32_ACCUMULATE
    else:
        kind = OUT_BF16 if out_dtype == torch.bfloat16 else OUT_FP32
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise NVFP4Error(f"unsupported output dtype {out_dtype}")
        if out is None:
            out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
        elif out.dtype != out_dtype:
            raise NVFP4Error("out dtype does not match out_dtype")
    _check_q(a, what="A")
    _check_q(b, what="B")
    _check_out(out, a.rows, b.rows, out.dtype)
    if amax_out is not None and (amax_out.numel() < 1 or amax_out.dtype != torch.float32):
        raise NVFP4Error("amax_out must be a float32 tensor of at least one element")
    if workspace is None:
        workspace, ws_n = _workspace(OP_GEMM_EX, a.rows, b.rows, 1, a.codes.device)
    else:
        ws_n = _given_workspace(workspace)
    ac, bc = a.c(), b.c()
    _check(lib.nvfp4_gemm_ex(ctypes.byref(ac), ctypes.byref(bc), _ptr(out), out.stride(0), kind,
                             _ptr(amax_out), _ptr(workspace), ws_n, _stream(stream)))
    return out


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise NVFP4Error(f"unknown activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


@_on_stream
def gemm_act(a: NVFP4Tensor, b: NVFP4Tensor, bias: torch.Tensor | None = None, activation: str = "none",
             residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
             preact: torch.Tensor | None = None, amax_out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_gemm_act: D = activation(A * B^T + bias) + residual in BF16. bias: [N], bfloat16 or
    float32; residual: [M, N] bfloat16; preact: a bfloat16 [M, N] tensor that receives A * B^T +
    bias (what act_grad needs); amax_out (float32 [1]) receives max |D| as stored."""
    lib = _load()
    kind = _activation(activation)
    m, n = a.rows, b.rows
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.codes.device)
    _check_q(a, what="A")
    _check_q(b, what="B")
    _check_out(out, m, n, torch.bfloat16)
    if bias is not None and (bias.dtype not in _DTYPE or bias.dim() != 1 or bias.numel() != n
                             or not bias.is_contiguous() or bias.device.type != "cuda"):
        raise NVFP4Error(f"bias must be a contiguous bfloat16 or float32 GPU tensor of {n} elements")
    if residual is not None:
        _check_out(residual, m, n, torch.bfloat16, "residual")
    if preact is not None:
        _check_out(preact, m, n, torch.bfloat16, "preact")
    _check_vec(amax_out, 1, "amax_out")
    if workspace is None:
        ws_n = workspace_size(OP_GEMM_ACT, m, n, a.cols)
        workspace = torch.empty((ws_n,), dtype=torch.uint8, device=a.codes.device) if ws_n else None
    else:
        ws_n = _given_workspace(workspace)
    ac, bc = a.c(), b.c()
    _check(lib.nvfp4_gemm_act(ctypes.byref(ac), ctypes.byref(bc), _ptr(out), _row_stride(out), _ptr(bias),
                              0 if bias is None else _DTYPE[bias.dtype], kind, _ptr(residual),
                              0 if residual is None else _row_stride(residual), _ptr(preact),
                              0 if preact is None else _row_stride(preact), _ptr(amax_out), _ptr(workspace), ws_n,
                              _stream(stream)))
    return out


@_on_stream
def act_grad(dy: torch.Tensor, preact: torch.Tensor | None = None, activation: str = "none",
             dz: torch.Tensor | None = None, dbias: torch.Tensor | None = None, accumulate: bool = False,
             bias_only: bool = False, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """nvfp4_act_grad: dZ = dY * activation'(Z) in BF16 (returned; allocated if dz is left out) and,
    with dbias (float32 [N]), its column sums written or (accumulate) added there. dy: [M, N]
    bfloat16 or float32; preact: gemm_act's. bias_only: no dZ, the column sums alone."""
    lib = _load()
    kind = _activation(activation)
    dt, m, n, ldy = _input(dy)
    if preact is not None:
        _check_out(preact, m, n, torch.bfloat16, "preact")
    if dz is not None:
        _check_out(dz, m, n, torch.bfloat16, "dz")
    elif not bias_only:
        dz = torch.empty((m, n), dtype=torch.bfloat16, device=dy.device)
    _check_vec(dbias, n, "dbias")
    ws_n = 0
    if dbias is not None:
        if workspace is None:
            ws_n = workspace_size(OP_ACT_GRAD, m, n)
            workspace = torch.empty((ws_n,), dtype=torch.uint8, device=dy.device) if ws_n else None
        else:
            ws_n = _given_workspace(workspace)
    _check(lib.nvfp4_act_grad(_ptr(dy), dt, m, n, _row_stride(dy), _ptr(preact), 0 if preact is None else _row_stride(preact),
                              kind, _ptr(dz), 0 if dz is None else _row_stride(dz), _ptr(dbias), int(accumulate),
                              _ptr(workspace), ws_n, _stream(stream)))
    return dz


@_on_stream
def grouped_gemm(m_offsets: torch.Tensor, a: NVFP4Tensor, b: NVFP4Tensor, n: int,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_grouped_gemm: per group g, rows m_offsets[g]:m_offsets[g+1] of A against rows
    g*n:(g+1)*n of B."""
    lib = _load()
    G = m_offsets.numel() - 1
    if out is None:
        out = torch.empty((a.rows, n), dtype=torch.float32, device=a.codes.device)
    _check_q(a, G, "A")
    _check_q(b, G, "B")
    _check_out(out, a.rows, n, torch.float32)
    if m_offsets.dtype != torch.int64 or m_offsets.device.type != "cuda":
        raise NVFP4Error("m_offsets must be an int64 GPU tensor")
    ac, bc = a.c(), b.c()
    _check(lib.nvfp4_grouped_gemm(G, _ptr(m_offsets), ctypes.byref(ac), ctypes.byref(bc), n,
                                  _ptr(out), out.stride(0), None, 0, _stream(stream)))
    return out


@_on_stream
def grouped_gemm_k(k_offsets: torch.Tensor, a: NVFP4Tensor, b: NVFP4Tensor,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_grouped_gemm_k: for each group g, columns k_offsets[g]:k_offsets[g+1] of A [M, K]
    and B [N, K] into rows g*M:(g+1)*M of D [G*M, N] (FP32)."""
    lib = _load()
    G = k_offsets.numel() - 1
    if out is None:
        out = torch.empty((G * a.rows, b.rows), dtype=torch.float32, device=a.codes.device)
    _check_q(a, G, "A")
    _check_q(b, G, "B")
    _check_out(out, G * a.rows, b.rows, torch.float32)
    if k_offsets.dtype != torch.int64 or k_offsets.device.type != "cuda":
        raise NVFP4Error("k_offsets must be an int64 GPU tensor")
    ac, bc = a.c(), b.c()
    _check(lib.nvfp4_grouped_gemm_k(G, _ptr(k_offsets), ctypes.byref(ac), ctypes.byref(bc),
                                    _ptr(out), out.stride(0), _stream(stream)))
    return out


@_on_stream
def amax(x: torch.Tensor, segments: torch.Tensor | None = None, rht: bool | int = False,
         sign_mask: int = 0, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """nvfp4_amax: max|x| per segment, or of the Hadamard-transformed tensor: rht = True (or 1)
    along tokens as rht_quantize, rht = 2 along each row as rht_rows_quantize."""
    lib = _load()
    dt, rows, cols, ld = _input(x)
    nseg = 1 if segments is None else segments.numel() - 1
    if out is None:
        out = torch.empty((nseg,), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace, ws_n = _workspace(OP_RHT_QUANTIZE if int(rht) == 1 else OP_QUANTIZE, rows, cols, nseg, x.device)
    else:
        ws_n = _given_workspace(workspace)
    _check_table(segments, "segments")
    _check_vec(out, nseg, "out")
    _check(lib.nvfp4_amax(_ptr(x), dt, rows, cols, ld, _ptr(segments), nseg, int(rht),
                          sign_mask & 0xFFFF, _ptr(out), _ptr(workspace), ws_n, _stream(stream)))
    return out


@_on_stream
def amax_pair(x: torch.Tensor, sign_mask: int, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_amax_pair: float32 [2] = (max|x|, max of the Hadamard-transformed tensor)."""
    lib = _load()
    dt, tokens, cols, ld = _input(x)
    if out is None:
        out = torch.empty((2,), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace, ws_n = _workspace(OP_AMAX_PAIR, tokens, cols, 1, x.device)
    else:
        ws_n = _given_workspace(workspace)
    _check_vec(out, 2, "out")
    _check(lib.nvfp4_amax_pair(_ptr(x), dt, tokens, cols, ld, sign_mask & 0xFFFF, _ptr(out),
                               _ptr(workspace), ws_n, _stream(stream)))
    return out


@_on_stream
def dequantize(q: NVFP4Tensor, segments: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_dequantize (test helper): FP32 [rows, cols]."""
    lib = _load()
    nseg = 1 if segments is None else segments.numel() - 1
    _check_table(segments, "segments")
    _check_q(q, nseg, "q")
    y = torch.empty((q.rows, q.cols), dtype=torch.float32, device=q.codes.device)
    qc = q.c()
    _check(lib.nvfp4_dequantize(ctypes.byref(qc), _ptr(segments), nseg, _ptr(y), _stream(stream)))
    return y


@dataclass
class MoEWeights:
    """A mixture-of-experts layer's weights and routing rule (nvfp4_moe): router [experts, hidden],
    bfloat16 or float32; w1 [experts*ffn, hidden] (gated: [experts*2*ffn, hidden], each expert's gate
    rows before its up rows) and w2 [experts*hidden, ffn] with one global_scale per expert."""
    router: torch.Tensor
    w1: NVFP4Tensor
    w2: NVFP4Tensor
    top_k: int
    activation: str = "relu2"
    gated: bool = False
    score: str = "softmax"
    renormalize: bool = True
    routed_scale: float = 1.0

    def c(self) -> _CMoE:
        r = self.router
        if r.dtype not in _DTYPE or r.dim() != 2 or not r.is_contiguous() or r.device.type != "cuda":
            raise NVFP4Error("router must be a contiguous 2-D bfloat16 or float32 GPU tensor")
        if self.score not in SCORES:
            raise NVFP4Error(f"unknown score {self.score!r}: one of {', '.join(SCORES)}")
        _check_q(self.w1, r.shape[0], "w1")
        _check_q(self.w2, r.shape[0], "w2")
        return _CMoE(r.shape[0], r.shape[1], self.w2.cols, self.top_k, r.data_ptr(), _DTYPE[r.dtype], self.w1.c(),
                     self.w2.c(), _activation(self.activation), int(self.gated), SCORES[self.score],
                     int(self.renormalize), self.routed_scale)


def moe_workspace(weights: MoEWeights, tokens: int) -> torch.Tensor:
    """A workspace for moe_tokens with up to `tokens` tokens, its counters zeroed on the current stream."""
    n = _load().nvfp4_moe_workspace_size(ctypes.byref(weights.c()), tokens)
    if n == 0:
        raise NVFP4Error(f"no expert layer for {tokens} tokens: {_load().nvfp4_last_error().decode()}")
    return torch.zeros((n,), dtype=torch.uint8, device=weights.router.device)


@_on_stream
def moe_tokens(x: torch.Tensor, weights: MoEWeights, out: torch.Tensor | None = None,
               ids_out: torch.Tensor | None = None, weights_out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_moe_tokens: the whole expert layer for x [tokens <= 64, hidden] (bfloat16). ids_out
    (int32) and weights_out (float32), both [tokens, top_k], receive the routing. workspace: one of
    moe_workspace's, kept between calls (calls that share one have to be ordered)."""
    if workspace is None and x.dim() == 2 and x.shape[0] > 0:
        workspace = moe_workspace(weights, x.shape[0])
    return _moe_call(x, weights.c(), out, ids_out, weights_out, workspace, stream)


def _moe_call(x, layer: _CMoE, out, ids_out, weights_out, workspace, stream):
    lib = _load()
    if x.dtype != torch.bfloat16:
        raise NVFP4Error("x must be bfloat16")
    _, tokens, hidden, _ = _input(x)
    if hidden != layer.hidden:
        raise NVFP4Error(f"x has {hidden} columns, the layer's hidden size is {layer.hidden}")
    if out is None:
        out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=x.device)
    else:
        _check_out(out, tokens, hidden, torch.bfloat16)
    n = tokens * layer.top_k
    for t, dtype, what in ((ids_out, torch.int32, "ids_out"), (weights_out, torch.float32, "weights_out")):
        if t is not None and (t.dtype != dtype or t.numel() < n or not t.is_contiguous() or not t.is_cuda):
            raise NVFP4Error(f"{what} must be a contiguous {dtype} GPU tensor of at least {n} elements")
    _check(lib.nvfp4_moe_tokens(ctypes.byref(layer), _ptr(x), tokens, _row_stride(x), _ptr(out), _row_stride(out),
                                _ptr(ids_out), _ptr(weights_out), _ptr(workspace),
                                0 if workspace is None else _given_workspace(workspace), _stream(stream)))
    return out


@dataclass
class AdamWTensor:
    """One tensor of an AdamW step (nvfp4_adamw_tensor): contiguous GPU tensors of the same number
    of elements. m and v are FP32, or uint8 E4M3 codes (v then holds sqrt(v)) with uint8 E8M0
    scales, one per 32 elements. An output left out is its input (the step is in place); w_out
    receives the BF16 weight."""
    p: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None
    w_out: torch.Tensor | None = None
    p_out: torch.Tensor | None = None
    m_out: torch.Tensor | None = None
    v_out: torch.Tensor | None = None
    m_scale_out: torch.Tensor | None = None
    v_scale_out: torch.Tensor | None = None
    weight_decay: float = 0.0


class AdamWPlan:
    """The device table of the tensors that adamw steps together (nvfp4_adamw_table). It holds
    their addresses and keeps them alive: gradients have to stay where they are from step to
    step (NVFP4Linear.main_grad does; zero a .grad instead of setting it to None)."""

    def __init__(self, tensors):
        tensors = list(tensors)
        if not tensors:
            raise NVFP4Error("an AdamW plan needs at least one tensor")
        lib = _load()
        self.tensors, self.count = tensors, len(tensors)
        self._kept = []                                      # every tensor whose address is in the table
        self.eight_bit = tensors[0].m.dtype == torch.uint8
        self.device = tensors[0].p.device
        array = (_CAdamWTensor * len(tensors))(*(self._entry(i, t) for i, t in enumerate(tensors)))
        size = lib.nvfp4_adamw_table_size(array, len(tensors))
        host = torch.empty((max(size, 1),), dtype=torch.uint8)
        chunks = ctypes.c_int64()
        _check(lib.nvfp4_adamw_table(array, len(tensors), int(self.eight_bit), _ptr(host), size, ctypes.byref(chunks)))
        self.chunks = chunks.value
        self.table = host.to(self.device)

    def _entry(self, i: int, t: AdamWTensor) -> _CAdamWTensor:
        n = t.p.numel()
        state = torch.uint8 if self.eight_bit else torch.float32

        def need(name, x, dtype, count=n):
            if (not isinstance(x, torch.Tensor) or x.dtype != dtype or x.numel() != count or not x.is_contiguous()
                    or x.device.type != "cuda" or x.device != self.device):
                raise NVFP4Error(f"tensor {i}: {name} must be a contiguous {dtype} tensor of {count} elements on "
                                 f"the GPU of the first tensor")
            self._kept.append(x)
            return x.data_ptr()

        if not isinstance(t.grad, torch.Tensor) or t.grad.dtype not in _DTYPE:
            raise NVFP4Error(f"tensor {i}: grad must be a bfloat16 or float32 tensor")
        c = _CAdamWTensor(n=n, weight_decay=float(t.weight_decay), grad_dt=_DTYPE[t.grad.dtype])
        c.grad = need("grad", t.grad, t.grad.dtype)
        c.p = need("p", t.p, torch.float32)
        c.p_out = c.p if t.p_out is None else need("p_out", t.p_out, torch.float32)
        if t.w_out is not None:
            c.w_out = need("w_out", t.w_out, torch.bfloat16)
        for k in ("m", "v"):
            src, dst = getattr(t, k), getattr(t, k + "_out")
            setattr(c, k, need(k, src, state))
            setattr(c, k + "_out", getattr(c, k) if dst is None else need(k + "_out", dst, state))
            if self.eight_bit:
                src, dst, blocks = getattr(t, k + "_scale"), getattr(t, k + "_scale_out"), (n + 31) // 32
                setattr(c, k + "_scale", need(k + "_scale", src, torch.uint8, blocks))
                setattr(c, k + "_scale_out",
                        getattr(c, k + "_scale") if dst is None else need(k + "_scale_out", dst, torch.uint8, blocks))
        return c


@_on_stream
def adamw(plan: AdamWPlan, lr: float, betas=(0.9, 0.95), eps: float = 1e-8, step: int = 1,
          max_norm: float | None = None, seed: int = 0, norm_out: torch.Tensor | None = None,
          amax_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """nvfp4_adamw: one AdamW step (number `step`, from 1) of the plan's tensors. With max_norm the
    gradients are clipped by their norm over all tensors, which norm_out (float32 [1], allocated if
    left out) receives and the call returns; a norm that is not finite leaves every tensor as it
    was. amax_out (float32 [tensors]) receives each tensor's max|weight|, the `amax` of its next
    quantize. seed: of the 8-bit states' stochastic rounding."""
    lib = _load()
    if max_norm is not None and norm_out is None:
        norm_out = torch.empty((1,), dtype=torch.float32, device=plan.device)
    _check_vec(norm_out, 1, "norm_out")
    _check_vec(amax_out, plan.count, "amax_out")
    ws_n = 0
    if max_norm is not None:
        if workspace is None:
            workspace, ws_n = _workspace(OP_ADAMW, 0, 0, 1, plan.device)
        else:
            ws_n = _given_workspace(workspace)
    hyper = _CAdamWHyper(lr, betas[0], betas[1], eps, step, 0.0 if max_norm is None else max_norm, seed & (2 ** 64 - 1))
    _check(lib.nvfp4_adamw(_ptr(plan.table), plan.count, plan.chunks, int(plan.eight_bit), ctypes.byref(hyper),
                           _ptr(norm_out), _ptr(amax_out), _ptr(workspace) if max_norm is not None else None, ws_n,
                           _stream(stream)))
    return norm_out

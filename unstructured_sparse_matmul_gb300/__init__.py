"""Python binding of libusm (CSR SpMM / SDDMM / row swizzle on GB300).

Argument marshalling only: every step runs in the library's CUDA kernels,
called through the C ABI declared in include/usm.h.  PyTorch supplies device
memory and the current stream.  There is no CPU fallback: if the library is
not built, or no CUDA device is present, calls raise.

Source of the operations: "Sparse GPU Kernels for Deep Learning" (Gale,
Zaharia, Young, Elsen, SC 2020), summary card ("Summary"; "Interesting ideas"
I3 for the SDDMM form, I4 for the row swizzle, I5 for plain CSR).
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import struct
import threading

from . import build as _build

USM_F32 = 0
USM_BF16 = 1

STATUS = {
    0: "USM_OK", -1: "USM_ERR_INVALID_ARG", -2: "USM_ERR_ALIGNMENT", -3: "USM_ERR_UNSUPPORTED",
    -4: "USM_ERR_CUDA", -5: "USM_ERR_TIMEOUT", -6: "USM_ERR_WORKSPACE",
}

# Every symbol include/usm.h declares, with its ctypes signature.
_vp, _i, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
SIGNATURES = {
    "csr_spmm": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _vp]),
    "csr_sddmm_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "csr_sddmm": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _i, _vp, _sz, _vp]),
    "row_swizzle_workspace_bytes": (_sz, [_i, _i]),
    "row_swizzle_build": (_i, [_i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "usm_poll_status": (_i, [_vp]),
    "usm_status_string": (ctypes.c_char_p, [_i]),
    "usm_selftest_wait_timeout": (_i, [_ll, _vp]),
    "usm_set_schedule_override": (_i, [_i, _i, _i]),
    "csr_sddmm_static_scratch": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _i, _vp]),
    "csr_transpose_workspace_bytes": (_sz, [_i, _i, _i]),
    "csr_sddmm_general_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "csr_sddmm_general": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _vp, _i, _i, _vp,
                               _sz, _vp]),
    "csr_row_softmax": (_i, [_i, _i, _vp, _vp, _vp, _i, _vp]),
    "csr_transpose": (_i, [_i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "csr_permute_values": (_i, [_i, _vp, _vp, _i, _vp, _vp]),
    "csr_validate": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp]),
    "csr_spmm_row_softmax": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _vp]),
}

SIGNATURES.update({
    "rel_bucket_build": (_i, [_i, _i, _i, _vp, _vp]),
    "csr_rel_bias": (_i, [_i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp]),
    "csr_rel_bias_grad_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "csr_rel_bias_grad": (_i, [_i, _i, _i, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "csr_diff_softmax": (_i, [_i, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp]),
    "csr_diff_softmax_grad_workspace_bytes": (_sz, [_i]),
    "csr_diff_softmax_grad": (_i, [_i, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "csr_row_softmax_grad": (_i, [_i, _i, _vp, _vp, _vp, _i, _vp, _i, _vp]),
    "csr_attention": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _i,
                           ctypes.c_float, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _sz, _vp]),
    "csr_attention_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
})


class RelBias(ctypes.Structure):
    """usm_rel_bias of include/usm.h."""
    _fields_ = [("table", _vp), ("table_dtype", _i), ("num_heads", _i), ("num_buckets", _i), ("bucket_map", _vp),
                ("max_distance", _i), ("seg_cols", _i), ("q_offset", _vp)]


REL_BIAS_MAX_DISTANCE = 8192  # USM_REL_BIAS_MAX_DISTANCE of include/usm.h

_pack_bias = struct.Struct("@PiiiPiiP").pack  # the same as bytes, in a quarter of the time


# csr_validate result codes (usm_csr_check in include/usm.h).
CSR_CHECK = {0: "USM_CSR_VALID", 1: "USM_CSR_FIRST_OFFSET", 2: "USM_CSR_OFFSETS_DECREASE",
             3: "USM_CSR_LAST_OFFSET", 4: "USM_CSR_COLUMN_RANGE", 5: "USM_CSR_COLUMN_ORDER"}
CSR_VALIDATE_INTS = 8

_lib = None
_lock = threading.Lock()


class USMError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code} ({STATUS.get(code, 'unknown')})")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libusm.so (building it first if needed) and bind its symbols."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_build.LIB) or not _build.up_to_date():
            if not build_if_missing:
                raise RuntimeError(f"CUDA library not built: {_build.LIB}")
            _build.build_library()
        lib = ctypes.CDLL(_build.LIB)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(fn: str, code: int):
    if code != 0:
        raise USMError(fn, code)


# ---------------------------------------------------------------------------
# torch helpers (memory and streams only)
# ---------------------------------------------------------------------------
def _torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("no CUDA device: libusm has no CPU fallback")
    return torch


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return USM_F32
    if t.dtype == torch.bfloat16:
        return USM_BF16
    raise TypeError(f"unsupported element type {t.dtype} (fp32 or bf16)")


def _require(t, name, dtypes=None, cuda=True):
    if t is None:
        raise ValueError(f"{name} is required")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _ld(t) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("dense operands must be 2-D with unit column stride")
    return t.stride(0)


def _round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


def _tma_ready(t):
    """The library reads dense inputs with TMA, which needs a 16-byte aligned
    base and a row pitch that is a multiple of 16 bytes.  Inputs that already
    satisfy this pass through untouched; others are copied once into a padded
    buffer (a marshalling copy; pass aligned tensors to avoid it)."""
    es = t.element_size()
    if (t.dim() == 2 and t.stride(1) == 1 and t.data_ptr() % 16 == 0
            and (t.stride(0) * es) % 16 == 0 and t.stride(0) >= t.shape[1]):
        return t
    torch = _torch()
    rows, cols = t.shape
    ld = _round_up(max(cols, 1), 16 // es)
    buf = torch.zeros((rows, ld), dtype=t.dtype, device=t.device)
    buf[:, :cols] = t
    return buf[:, :cols]


def _new_dense_out(rows: int, cols: int, device):
    """fp32 output with a row pitch that is a multiple of 4 elements."""
    torch = _torch()
    ld = _round_up(max(cols, 1), 4)
    return torch.empty((rows, ld), dtype=torch.float32, device=device)[:, :cols]


# ---------------------------------------------------------------------------
# Operations
# ---------------------------------------------------------------------------
def row_swizzle(row_offsets, K: int, seg_rows: int = 0, out=None, stream=None):
    """Row-swizzle order (int32[M]) of a CSR's rows; see row_swizzle_build."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    M = row_offsets.numel() - 1
    out = out if out is not None else torch.empty(M, dtype=torch.int32, device=row_offsets.device)
    ws_bytes = lib.row_swizzle_workspace_bytes(M, K)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=row_offsets.device)
    _check("row_swizzle_build", lib.row_swizzle_build(M, K, seg_rows, _ptr(row_offsets), _ptr(out),
                                                      _ptr(ws), ws_bytes, _stream(stream)))
    return out


def spmm(row_offsets, col_indices, values, B, K: int | None = None, row_swizzle=None, out=None,
         stream=None, seg_rows: int = 0):
    """C = A·B (fp32 out).  values and B are both fp32 or both bf16."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(col_indices, "col_indices", (torch.int32,))
    _require(values, "values", (torch.float32, torch.bfloat16))
    _require(B, "B", (values.dtype,))
    M = row_offsets.numel() - 1
    K = B.shape[0] if K is None else K
    N = B.shape[1]
    B = _tma_ready(B)
    C = out if out is not None else _new_dense_out(M, N, B.device)
    _require(C, "out", (torch.float32,))
    code = lib.csr_spmm(M, K, N, col_indices.numel(), _ptr(row_offsets), _ptr(col_indices), _ptr(values),
                        _ptr(row_swizzle), seg_rows, _ptr(B), _ld(B), _ptr(C), _ld(C), _dtype_code(values),
                        _stream(stream))
    _check("csr_spmm", code)
    return C


def spmm_row_softmax(row_offsets, col_indices, scores, B, K: int | None = None, row_swizzle=None, out=None,
                     stream=None, seg_rows: int = 0):
    """C = softmax_rows(scores)·B (fp32 out): each row's stored fp32 scores
    turned into softmax probabilities, rounded to B's element type (fp32 or
    bf16), inside the product; see csr_spmm_row_softmax."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(col_indices, "col_indices", (torch.int32,))
    _require(scores, "scores", (torch.float32,))
    _require(B, "B", (torch.float32, torch.bfloat16))
    M = row_offsets.numel() - 1
    K = B.shape[0] if K is None else K
    N = B.shape[1]
    B = _tma_ready(B)
    C = out if out is not None else _new_dense_out(M, N, B.device)
    _require(C, "out", (torch.float32,))
    code = lib.csr_spmm_row_softmax(M, K, N, col_indices.numel(), _ptr(row_offsets), _ptr(col_indices), _ptr(scores),
                                    _ptr(row_swizzle), seg_rows, _ptr(B), _ld(B), _ptr(C), _ld(C), _dtype_code(B),
                                    _stream(stream))
    _check("csr_spmm_row_softmax", code)
    return C


def sddmm(row_offsets, col_indices, X, Y, row_swizzle=None, out=None, out_dtype=None, workspace=None,
          stream=None, seg_rows: int = 0):
    """out[p] = X[r]·Y[col_p] on the mask's nonzeros (CSR order)."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(col_indices, "col_indices", (torch.int32,))
    _require(X, "X", (torch.float32, torch.bfloat16))
    _require(Y, "Y", (X.dtype,))
    M = row_offsets.numel() - 1
    K, D = Y.shape[0], Y.shape[1]
    if X.shape[1] != D:
        raise ValueError("X and Y must have the same number of columns")
    X, Y = _tma_ready(X), _tma_ready(Y)
    nnz = col_indices.numel()
    if out is None:
        od = out_dtype if out_dtype is not None else torch.float32
        out = torch.empty(nnz, dtype=od, device=X.device)
    in_code = _dtype_code(X)
    out_code = _dtype_code(out)
    ws_bytes = lib.csr_sddmm_workspace_bytes(M, K, D, nnz, in_code)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=X.device)
    code = lib.csr_sddmm(M, K, D, nnz, _ptr(row_offsets), _ptr(col_indices), _ptr(row_swizzle), seg_rows,
                         _ptr(X), _ld(X), _ptr(Y), _ld(Y), _ptr(out), in_code, out_code,
                         _ptr(workspace) if ws_bytes else None, ws_bytes, _stream(stream))
    _check("csr_sddmm", code)
    return out


def sddmm_general(row_offsets, col_indices, X, Y, values=None, y_transposed=True, row_swizzle=None, out=None,
                  out_dtype=None, stream=None, seg_rows: int = 0):
    """out[p] = (values[p] if given) · X[r]·Yop[col_p]; Yop = Y (K×D) when
    y_transposed, else Yᵀ with Y given D×K."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(col_indices, "col_indices", (torch.int32,))
    _require(X, "X", (torch.float32, torch.bfloat16))
    _require(Y, "Y", (X.dtype,))
    if values is not None:
        _require(values, "values", (X.dtype,))
    M = row_offsets.numel() - 1
    D = X.shape[1]
    K = Y.shape[0] if y_transposed else Y.shape[1]
    if (Y.shape[1] if y_transposed else Y.shape[0]) != D:
        raise ValueError("X and Y disagree on D")
    X = _tma_ready(X)
    if y_transposed:
        Y = _tma_ready(Y)
    elif Y.stride(1) != 1:
        Y = Y.contiguous()
    nnz = col_indices.numel()
    if out is None:
        out = torch.empty(nnz, dtype=out_dtype if out_dtype is not None else torch.float32, device=X.device)
    in_code = _dtype_code(X)
    ws_bytes = lib.csr_sddmm_general_workspace_bytes(M, K, D, nnz, in_code, int(bool(y_transposed)))
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=X.device)
    code = lib.csr_sddmm_general(M, K, D, nnz, _ptr(row_offsets), _ptr(col_indices), _ptr(values),
                                 _ptr(row_swizzle), seg_rows, _ptr(X), _ld(X), _ptr(Y), Y.stride(0),
                                 int(bool(y_transposed)),
                                 _ptr(out), in_code, _dtype_code(out), _ptr(ws) if ws_bytes else None, ws_bytes,
                                 _stream(stream))
    _check("csr_sddmm_general", code)
    return out


def row_softmax(row_offsets, scores, out=None, out_dtype=None, stream=None):
    """Softmax over the stored entries of each CSR row (fp32 scores in)."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(scores, "scores", (torch.float32,))
    if out is None:
        out = torch.empty_like(scores, dtype=out_dtype if out_dtype is not None else torch.float32)
    code = lib.csr_row_softmax(row_offsets.numel() - 1, scores.numel(), _ptr(row_offsets), _ptr(scores), _ptr(out),
                               _dtype_code(out), _stream(stream))
    _check("csr_row_softmax", code)
    return out


# ---------------------------------------------------------------------------
# Sparse attention: position bias, differential map, softmax gradients, and
# attention of few rows.  Every tensor of a call lies on one device, which need
# not be the current one; 1-D arrays are contiguous.  Single tokens spend most
# of such a call on the host, so a check that passes costs one expression and
# only a failing one looks for the reason.
# ---------------------------------------------------------------------------
def _on_stream(fn):
    """Gives an operation its `stream` keyword.  With a stream of the caller's,
    copies, outputs and scratch belong to that stream too (as under
    torch.cuda.stream), so none of them races the current stream's work."""
    signature = inspect.signature(fn)
    takes_device = "device" in signature.parameters

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        torch = _torch()
        for t in (*args, *kwargs.values()):
            if isinstance(t, torch.Tensor) and t.device != stream.device:
                raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
        device = signature.bind(*args, **kwargs).arguments.get("device") if takes_device else None
        if device is not None:
            device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
            if device.type != "cuda" or device.index not in (None, stream.device.index):
                raise ValueError(f"stream is on {stream.device}, the result on {device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)

    return call


class _Types:
    """Element types the operations take (filled in once torch is there)."""
    torch = i32 = f32 = real = empty = current_device = raw_stream = None


def _types():
    if _Types.torch is None:
        torch = _torch()
        _Types.i32, _Types.f32, _Types.real = (torch.int32,), (torch.float32,), (torch.float32, torch.bfloat16)
        _Types.empty, _Types.current_device = staticmethod(torch.empty), staticmethod(torch.cuda.current_device)
        # The current stream's handle; the public way builds a Stream object for it.
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _Types.raw_stream = staticmethod(raw or (lambda index: torch.cuda.current_stream(index).cuda_stream))
        _Types.torch = torch
    return _Types


def _tensor(t, name, index, dtypes, dims):
    """A tensor of the call: its type, number of dimensions and device."""
    if t is None or t.dtype not in dtypes or t.dim() != dims or t.get_device() != index or index < 0:
        if t is None:
            raise ValueError(f"{name} is required")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
        if t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimension(s), has {t.dim()}")
        raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{index}")
    return t


def _array(t, name, index, dtypes, n=None):
    """A contiguous 1-D tensor, of n elements unless None."""
    if (t is None or t.dtype not in dtypes or t.dim() != 1 or t.get_device() != index or index < 0
            or not t.is_contiguous() or (n is not None and t.numel() != n)):
        _tensor(t, name, index, dtypes, 1)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    return t


def _device_of(t, name) -> int:
    if t is None:
        raise ValueError(f"{name} is required")
    return t.get_device()


def _rows(row_offsets, index, T) -> int:
    M = _array(row_offsets, "row_offsets", index, T.i32).numel() - 1
    if not 0 <= M < 2**31:
        raise ValueError(f"row_offsets has {M + 1} elements: from 1 to 2**31 are expected")
    return M


def _entries(n: int) -> int:
    if n >= 2**31:
        raise ValueError(f"{n} entries do not fit 32 bits")
    return n


def _int32(values, names):
    for v in values:
        if not -2**31 <= v < 2**31:
            raise ValueError(f"{names[values.index(v)]} = {v} does not fit 32 bits")


def _out(out, like, n, dtype, index, T, name="out"):
    """A given 1-D output, checked, or a new one beside `like`."""
    if out is None:
        return T.empty(n, dtype=T.f32[0] if dtype is None else dtype, device=like.device)
    return _array(out, name, index, T.real if dtype is None else (dtype,), n)


def _workspace(workspace, need: int, like, T):
    """The caller's workspace, if it holds `need` bytes, or a new one."""
    if need == 0:
        return None
    if workspace is not None:
        if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the others")
        if workspace.numel() * workspace.element_size() >= need:
            return workspace
    return T.empty(need, dtype=T.torch.uint8, device=like.device)


def _bias(bucket_map, num_heads, num_buckets, seg_rows, seg_cols, q_offset, M, index, T, table=None):
    """The usm_rel_bias struct, as bytes that the call takes a pointer to."""
    _int32((seg_rows, seg_cols, num_heads, num_buckets), ("seg_rows", "seg_cols", "num_heads", "num_buckets"))
    n = _array(bucket_map, "bucket_map", index, T.i32).numel()
    if n < 3 or n % 2 == 0:
        raise ValueError("bucket_map has 2*max_distance + 1 entries")
    if q_offset is not None:
        blocks = 1 if seg_rows <= 0 or seg_rows > M else -(-M // seg_rows)
        if M == 0 and q_offset.numel() == 0:
            blocks = 0  # a batch of no sequences
        _array(q_offset, "q_offset", index, T.i32, blocks)
    if table is not None and not table.is_contiguous():
        raise ValueError("table must be contiguous")
    return _pack_bias(0 if table is None else table.data_ptr(), USM_F32 if table is None else _code(table, T), num_heads,
                      num_buckets, bucket_map.data_ptr(), n // 2, seg_cols, 0 if q_offset is None else q_offset.data_ptr())


def _code(t, T) -> int:
    """Type code of a tensor that holds fp32 or bf16."""
    d = t.dtype
    if d not in T.real:
        raise TypeError(f"unsupported element type {d} (fp32 or bf16)")
    return USM_F32 if d is T.f32[0] else USM_BF16


def _run(name, fn, index, T, *args):
    """Call the library on device `index`, on its current stream."""
    if index == T.current_device():
        code = fn(*args, T.raw_stream(index))
    else:
        with T.torch.cuda.device(index):
            code = fn(*args, T.raw_stream(index))
    if code != 0:
        raise USMError(name, code)


@_on_stream
def rel_bucket_map(num_buckets: int, max_distance: int, causal: bool = False, device=None):
    """int32[2*max_distance + 1]: the bucket of each relative position
    -max_distance..max_distance, logarithmic past num_buckets/2 (causal) or
    num_buckets/4; see rel_bucket_build."""
    T, lib = _types(), load()
    _int32((num_buckets, max_distance), ("num_buckets", "max_distance"))
    if max_distance > REL_BIAS_MAX_DISTANCE:  # no memory is taken for a map that is refused
        raise USMError("rel_bucket_build", lib.rel_bucket_build(num_buckets, max_distance, int(bool(causal)), None, None))
    out = T.torch.empty(max(2 * max_distance + 1, 1), dtype=T.i32[0], device="cuda" if device is None else device)
    index = out.get_device()
    _array(out, "bucket_map", index, T.i32)
    _run("rel_bucket_build", lib.rel_bucket_build, index, T, num_buckets, max_distance, int(bool(causal)),
         out.data_ptr())
    return out


@_on_stream
def rel_bias(row_offsets, col_indices, scores, table, bucket_map, seg_rows: int = 0, seg_cols: int = 0, q_offset=None,
             out=None):
    """out[p] = scores[p] + table[head][bucket of p's relative position]; out
    may be scores.  table: num_heads x num_buckets, fp32 or bf16; see
    csr_rel_bias."""
    T, lib = _types(), load()
    index = _device_of(row_offsets, "row_offsets")
    M = _rows(row_offsets, index, T)
    _array(scores, "scores", index, T.f32)
    nnz = _entries(scores.numel())
    _array(col_indices, "col_indices", index, T.i32, nnz)
    _tensor(table, "table", index, T.real, 2)
    heads, buckets = table.shape
    b = _bias(bucket_map, heads, buckets, seg_rows, seg_cols, q_offset, M, index, T, table)
    out = _out(out, scores, nnz, T.f32[0], index, T)
    _run("csr_rel_bias", lib.csr_rel_bias, index, T, M, _ANY_COLUMN, nnz, row_offsets.data_ptr(),
         col_indices.data_ptr(), scores.data_ptr(), seg_rows, b, out.data_ptr())
    return out


_ANY_COLUMN = 2**31 - 1  # K of calls that address nothing by column: it only says that there are columns


@_on_stream
def rel_bias_grad(row_offsets, col_indices, dscores, num_heads: int, num_buckets: int, bucket_map, seg_rows: int = 0,
                  seg_cols: int = 0, q_offset=None, out=None, workspace=None):
    """The gradient of rel_bias's table (num_heads x num_buckets fp32) from the
    scores' gradient (fp32 or bf16); see csr_rel_bias_grad."""
    T, lib = _types(), load()
    index = _device_of(row_offsets, "row_offsets")
    M = _rows(row_offsets, index, T)
    _array(dscores, "dscores", index, T.real)
    nnz = _entries(dscores.numel())
    _array(col_indices, "col_indices", index, T.i32, nnz)
    b = _bias(bucket_map, num_heads, num_buckets, seg_rows, seg_cols, q_offset, M, index, T)
    if out is None:
        out = T.empty((max(num_heads, 0), max(num_buckets, 0)), dtype=T.f32[0], device=dscores.device)
    else:
        _tensor(out, "out", index, T.f32, 2)
        if not out.is_contiguous() or tuple(out.shape) != (num_heads, num_buckets):
            raise ValueError("out must be a contiguous num_heads x num_buckets tensor")
    need = lib.csr_rel_bias_grad_workspace_bytes(M, nnz, seg_rows, num_heads, num_buckets)
    ws = _workspace(workspace, need, dscores, T)
    _run("csr_rel_bias_grad", lib.csr_rel_bias_grad, index, T, M, _ANY_COLUMN, nnz, row_offsets.data_ptr(),
         col_indices.data_ptr(), dscores.data_ptr(), _code(dscores, T), seg_rows, b, out.data_ptr(),
         _ptr(ws), need)
    return out


@_on_stream
def diff_softmax(row_offsets, scores1, scores2, lam, seg_rows: int = 0, out=None, out_dtype=None):
    """softmax_rows(scores1) - lam[head]*softmax_rows(scores2) on the stored
    entries: the value array of spmm with V; see csr_diff_softmax."""
    T, lib = _types(), load()
    index = _device_of(row_offsets, "row_offsets")
    M = _rows(row_offsets, index, T)
    _array(scores1, "scores1", index, T.f32)
    nnz = _entries(scores1.numel())
    _array(scores2, "scores2", index, T.f32, nnz)
    _array(lam, "lam", index, T.f32)
    _int32((seg_rows,), ("seg_rows",))
    out = _out(out, scores1, nnz, out_dtype, index, T)
    _run("csr_diff_softmax", lib.csr_diff_softmax, index, T, M, nnz, row_offsets.data_ptr(), scores1.data_ptr(),
         scores2.data_ptr(), lam.data_ptr(), lam.numel(), seg_rows, out.data_ptr(), _code(out, T))
    return out


@_on_stream
def diff_softmax_grad(row_offsets, scores1, scores2, lam, dout, seg_rows: int = 0, out1=None, out2=None,
                      out_dtype=None, dlam=None, workspace=None):
    """Gradients of diff_softmax: (dscores1, dscores2, dlam) from the map's
    gradient dout (fp32 or bf16); see csr_diff_softmax_grad."""
    T, lib = _types(), load()
    index = _device_of(row_offsets, "row_offsets")
    M = _rows(row_offsets, index, T)
    _array(scores1, "scores1", index, T.f32)
    nnz = _entries(scores1.numel())
    _array(scores2, "scores2", index, T.f32, nnz)
    _array(lam, "lam", index, T.f32)
    _array(dout, "dout", index, T.real, nnz)
    _int32((seg_rows,), ("seg_rows",))
    if out_dtype is None:
        given = out1 if out1 is not None else out2
        out_dtype = T.f32[0] if given is None else given.dtype
    out1 = _out(out1, scores1, nnz, out_dtype, index, T, "out1")
    out2 = _out(out2, scores1, nnz, out_dtype, index, T, "out2")
    dlam = _out(dlam, scores1, lam.numel(), T.f32[0], index, T, "dlam")
    need = lib.csr_diff_softmax_grad_workspace_bytes(M)
    ws = _workspace(workspace, need, scores1, T)
    _run("csr_diff_softmax_grad", lib.csr_diff_softmax_grad, index, T, M, nnz, row_offsets.data_ptr(),
         scores1.data_ptr(), scores2.data_ptr(), lam.data_ptr(), lam.numel(), seg_rows, dout.data_ptr(),
         _code(dout, T), out1.data_ptr(), out2.data_ptr(), _code(out1, T), dlam.data_ptr(), _ptr(ws), need)
    return out1, out2, dlam


@_on_stream
def row_softmax_grad(row_offsets, scores, dout, out=None, out_dtype=None):
    """The gradient of row_softmax's scores from the probabilities' gradient
    dout (fp32 or bf16); see csr_row_softmax_grad."""
    T, lib = _types(), load()
    index = _device_of(row_offsets, "row_offsets")
    M = _rows(row_offsets, index, T)
    _array(scores, "scores", index, T.f32)
    nnz = _entries(scores.numel())
    _array(dout, "dout", index, T.real, nnz)
    out = _out(out, scores, nnz, out_dtype, index, T)
    _run("csr_row_softmax_grad", lib.csr_row_softmax_grad, index, T, M, nnz, row_offsets.data_ptr(), scores.data_ptr(),
         dout.data_ptr(), _code(dout, T), out.data_ptr(), _code(out, T))
    return out


def _operand(t, name, index, dtypes, rows, cols):
    """A dense operand of the given shape as the library reads it, and its
    leading dimension (a copy only where rows are not 16-byte aligned)."""
    _tensor(t, name, index, dtypes, 2)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected {(rows, cols)}")
    ld, unit = t.stride()
    if unit != 1 or ld < cols or (t.data_ptr() | ld * t.element_size()) & 15:
        t = _tma_ready(t)
        ld = t.stride(0)
    return t, ld


@_on_stream
def attention(row_offsets, col_indices, Q, Km, V, scale: float = 1.0, Q2=None, K2=None, lam=None, seg_rows: int = 0,
              table=None, bucket_map=None, seg_cols: int = 0, q_offset=None, out=None, workspace=None):
    """Sparse attention of few query rows in one pass (fp32 out): softmax of
    scale*(Q[r].Km[col]) + bias over each row's entries, times V; with Q2, K2
    and lam the differential map, with table and bucket_map the relative
    position bias; see csr_attention."""
    T, lib = _types(), load()
    index = _device_of(row_offsets, "row_offsets")
    M = _rows(row_offsets, index, T)
    _array(col_indices, "col_indices", index, T.i32)
    nnz = _entries(col_indices.numel())
    _tensor(Km, "Km", index, T.real, 2)
    _tensor(V, "V", index, T.real, 2)
    K, D = Km.shape
    N = V.shape[1]
    dt = (Km.dtype,)
    Q, ldq = _operand(Q, "Q", index, dt, M, D)
    Km, ldk = _operand(Km, "Km", index, dt, K, D)
    V, ldv = _operand(V, "V", index, dt, K, N)
    _int32((seg_rows,), ("seg_rows",))
    heads, ldq2, ldk2, b = 1, 0, 0, None
    if lam is None:
        if Q2 is not None or K2 is not None:
            raise ValueError("Q2, K2 and lam come together")
    else:
        if Q2 is None or K2 is None:
            raise ValueError("Q2, K2 and lam come together")
        Q2, ldq2 = _operand(Q2, "Q2", index, dt, M, D)
        K2, ldk2 = _operand(K2, "K2", index, dt, K, D)
        heads = _array(lam, "lam", index, T.f32).numel()
    if table is not None:
        _tensor(table, "table", index, T.real, 2)
        if lam is not None and table.shape[0] != heads:
            raise ValueError("table and lam disagree on the number of heads")
        heads, buckets = table.shape
        b = _bias(bucket_map, heads, buckets, seg_rows, seg_cols, q_offset, M, index, T, table)
    elif bucket_map is not None or q_offset is not None:
        raise ValueError("bucket_map and q_offset need a table")
    if out is None:
        out = _new_dense_out(M, N, V.device) if N % 4 or N == 0 else T.empty((M, N), dtype=T.f32[0], device=V.device)
        ldc = max(out.stride(0), N)
    else:
        _tensor(out, "out", index, T.f32, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be M x N")
        ldc = _ld(out)
    code = _code(Km, T)
    need = lib.csr_attention_workspace_bytes(M, K, D, N, nnz, int(lam is not None), code)
    ws = _workspace(workspace, need, Km, T)
    _run("csr_attention", lib.csr_attention, index, T, M, K, D, N, nnz, row_offsets.data_ptr(), col_indices.data_ptr(),
         Q.data_ptr(), ldq, Km.data_ptr(), ldk, _ptr(Q2), ldq2, _ptr(K2), ldk2, V.data_ptr(), ldv, scale, _ptr(lam),
         heads, seg_rows, b, out.data_ptr(), ldc, code, _ptr(ws), need)
    return out


def csr_validate(row_offsets, col_indices, K: int, stream=None):
    """Check the CSR contract on the device: (code, index), code one of
    CSR_CHECK (0 = valid), index the first offending row or nonzero (-1 when
    valid).  Reads the two result words back, so it waits for the stream."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(col_indices, "col_indices", (torch.int32,))
    result = torch.empty(CSR_VALIDATE_INTS, dtype=torch.int32, device=row_offsets.device)
    code = lib.csr_validate(row_offsets.numel() - 1, K, col_indices.numel(), _ptr(row_offsets), _ptr(col_indices),
                            _ptr(result), _stream(stream))
    _check("csr_validate", code)
    out = result[:2].cpu()
    return int(out[0]), int(out[1])


def csr_transpose(row_offsets, col_indices, values, K: int, with_perm: bool = False, stream=None):
    """Aᵀ in CSR: (row_offsets_t, col_indices_t, values_t[, perm])."""
    torch = _torch()
    lib = load()
    _require(row_offsets, "row_offsets", (torch.int32,))
    _require(col_indices, "col_indices", (torch.int32,))
    M = row_offsets.numel() - 1
    nnz = col_indices.numel()
    dev = row_offsets.device
    ro_t = torch.empty(K + 1, dtype=torch.int32, device=dev)
    ci_t = torch.empty(nnz, dtype=torch.int32, device=dev)
    v_t = torch.empty_like(values) if values is not None else None
    perm = torch.empty(nnz, dtype=torch.int32, device=dev) if with_perm else None
    code_dt = _dtype_code(values) if values is not None else USM_F32
    ws_bytes = lib.csr_transpose_workspace_bytes(M, K, nnz)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    code = lib.csr_transpose(M, K, nnz, _ptr(row_offsets), _ptr(col_indices), _ptr(values), code_dt, _ptr(ro_t),
                             _ptr(ci_t), _ptr(v_t), _ptr(perm), _ptr(ws), ws_bytes, _stream(stream))
    _check("csr_transpose", code)
    return (ro_t, ci_t, v_t, perm) if with_perm else (ro_t, ci_t, v_t)


def csr_permute_values(perm, values, out=None, stream=None):
    """out[q] = values[perm[q]]."""
    lib = load()
    out = out if out is not None else values.new_empty(perm.numel())
    _check("csr_permute_values", lib.csr_permute_values(perm.numel(), _ptr(perm), _ptr(values), _dtype_code(values),
                                                        _ptr(out), _stream(stream)))
    return out


def poll_status(stream=None) -> int:
    return int(load().usm_poll_status(_stream(stream)))


def set_schedule_override(rows_per_warp: int = 0, tiles_per_block: int = 0, k_splits: int = 0) -> None:
    """Force the launch shape of later SpMM/SDDMM calls (0 = the library's
    choice); see usm_set_schedule_override."""
    _check("usm_set_schedule_override", load().usm_set_schedule_override(rows_per_warp, tiles_per_block, k_splits))


def status_string(code: int) -> str:
    return load().usm_status_string(code).decode()

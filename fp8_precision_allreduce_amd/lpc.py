"""Python binding of liblpc.so: one function per C entry point, same names.

Argument marshalling only: each function checks that the torch tensors it is
given are contiguous GPU tensors of the right type and large enough for the
element count it derives, turns them into device pointers, and calls the C
entry point on torch's current HIP stream (or the stream given).  Every step
of the computation runs in the library's HIP kernels; there is no fallback.
A non-LPC_OK status raises LpcError.

bfloat16 data is passed as torch.bfloat16 tensors.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblpc.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "lpc.h")
MEASURE_HEADER = os.path.join(os.path.dirname(_HERE), "include", "lpc_measure.h")
OPS_HEADER = os.path.join(os.path.dirname(_HERE), "include", "lpc_ops.h")

BLOCK = 128
MAX_RANKS = 8
MAX_ELEMS = 1 << 32
LPC_F32, LPC_BF16 = 0, 1
ALGO_AUTO, ALGO_DDA_FLAT, ALGO_DDA_TREE, ALGO_LOW_PRECISION = 0, 1, 2, 3
ALGO_NAMES = {ALGO_AUTO: "auto", ALGO_DDA_FLAT: "dda_flat", ALGO_DDA_TREE: "dda_tree",
              ALGO_LOW_PRECISION: "low_precision"}
STATUS = ["LPC_OK", "LPC_ERR_NULL", "LPC_ERR_SHAPE", "LPC_ERR_RANKS", "LPC_ERR_DTYPE",
          "LPC_ERR_ALIGN", "LPC_ERR_HIP", "LPC_ERR_SCRATCH"]
NOALLOC_SCRATCH_BYTES = 64 << 20


class LpcError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s failed: %s" % (fn, msg))
        self.status = status
        self.status_name = STATUS[status] if 0 <= status < len(STATUS) else str(status)


class _AdamwTensor(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("param", "grad", "m", "v", "m_scales", "v_scales", "copy")] + [
        ("n", ctypes.c_size_t)]


_vp, _sz, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_f32, _f64, _szp, _tp = ctypes.c_float, ctypes.c_double, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(_AdamwTensor)
_pp = ctypes.POINTER(ctypes.c_void_p)
SIGNATURES = {
    "lpc_quantize_fp8": [_vp, _int, _sz, _vp, _vp, _vp],
    "lpc_reduce_scatter_chunk": [_pp, _pp, _int, _int, _sz, _vp, _vp, _vp],
    "lpc_allgather_dequant": [_pp, _pp, _int, _sz, _vp, _int, _vp],
    "lpc_rs_ag_fused": [_pp, _pp, _int, _int, _sz, _vp, _vp, _pp, _pp, _vp, _int, _vp],
    "lpc_reduce_scatter": [_pp, _pp, _int, _int, _sz, _vp, _int, _vp],
    "dda_flat_reduce": [_pp, _int, _sz, _vp, _vp],
    "dda_tree_reduce_scatter": [_pp, _int, _int, _int, _sz, _vp, _vp],
    "dda_tree_allgather": [_pp, _int, _int, _sz, _vp, _vp],
    "lpc_a2av_route": [_vp, _sz, _int, _vp, _vp, _vp, _vp],
    "lpc_quantize_fp8_rows": [_vp, _int, _sz, _sz, _vp, _vp, _vp, _vp],
    "lpc_dequantize_fp8": [_vp, _vp, _sz, _vp, _int, _vp],
    "lpc_e4m3_encode": [_vp, _sz, _vp, _vp],
    "lpc_select_algo": [_int, _sz, _int, _int],
    "lpc_allreduce_workspace_bytes": [_int, _int, _sz, _int, ctypes.POINTER(ctypes.c_size_t)],
    "lpc_allreduce_emulated": [_pp, _int, _sz, _int, _int, _vp, _sz, _vp],
    "lpc_allreduce_emulated_noalloc": [_pp, _int, _sz, _int, _int, _vp],
    # training and serving operators (include/lpc_ops.h)
    "lpc_gemm_fp8": [_vp, _vp, _sz, _sz, _vp, _vp, _sz, _int, _vp, _vp, _int, _vp],
    "lpc_padded_rows": [_sz, _int],
    "lpc_quantize_fp8_cols": [_vp, _int, _sz, _sz, _int, _vp, _vp, _vp, _vp, _vp, _vp],
    "lpc_requantize_fp8_cols": [_vp, _vp, _sz, _sz, _int, _vp, _vp, _vp, _vp],
    "lpc_gemm_fp8_wgrad": [_vp, _vp, _sz, _vp, _vp, _sz, _sz, _int, _vp, _vp, _vp],
    "lpc_router_workspace_bytes": [_sz, _int],
    "lpc_router_forward": [_vp, _int, _sz, _int, _int, _int, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "lpc_router_backward": [_vp, _int, _sz, _int, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "lpc_adamw_plan_bytes": [_tp, _int],
    "lpc_adamw_plan": [_tp, _int, _int, _int, _vp, _sz, _szp],
    "lpc_adamw_step": [_vp, _sz, _int, _int, ctypes.c_int64, _f64, _f64, _f64, _f64, _f64, _vp, _vp],
    # reference kernels for measurement (include/lpc_measure.h)
    "lpc_measure_stream": [_vp, _sz, _vp, _sz, _int, _vp],
    "lpc_measure_empty": [ctypes.c_uint, ctypes.c_uint, ctypes.c_uint, _sz, _vp, _vp],
}

SIZES = ("lpc_padded_rows", "lpc_router_workspace_bytes", "lpc_adamw_plan_bytes")  # these return a size_t, not a status

_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded liblpc.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "liblpc.so is not built (%s); build it with "
                    "`python -m fp8_precision_allreduce_amd.build` -- there is no fallback path"
                    % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            for name, args in SIGNATURES.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = ctypes.c_size_t if name in SIZES else ctypes.c_int
            L.lpc_status_string.argtypes = [ctypes.c_int]
            L.lpc_status_string.restype = ctypes.c_char_p
            L.lpc_abi_version.argtypes = []
            L.lpc_abi_version.restype = ctypes.c_int
            _lib = L
    return _lib


def header_functions(header: str = HEADER) -> list:
    """Names of the functions a header under include/ declares (lpc.h by default)."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


def lpc_status_string(status: int) -> str:
    return lib().lpc_status_string(status).decode()


def lpc_abi_version() -> int:
    return lib().lpc_abi_version()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _call(name: str, *args):
    st = getattr(lib(), name)(*args)
    if st != 0:
        raise LpcError(name, st, lpc_status_string(st))


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, what: str, dtypes=None, min_numel: int = 0) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % what)
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (what, t.dtype, dtypes))
    if t.numel() < min_numel:
        raise ValueError("%s holds %d elements, needs %d" % (what, t.numel(), min_numel))
    return ctypes.c_void_p(t.data_ptr())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LPC_F32
    if t.dtype == torch.bfloat16:
        return LPC_BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def _ptrs(ts, what, dtypes, min_numel, skip=None):
    arr = (ctypes.c_void_p * len(ts))()
    for i, t in enumerate(ts):
        if i == skip and t is None:
            arr[i] = None
            continue
        arr[i] = _dev(t, "%s[%d]" % (what, i), dtypes, min_numel).value
    return arr


_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_FB = (torch.float32, torch.bfloat16)
_I32 = (torch.int32,)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def lpc_quantize_fp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    n = x.numel()
    _call("lpc_quantize_fp8", _dev(x, "x", _FB), _dtype(x), n, _dev(codes, "codes", _U8, n),
          _dev(scales, "scales", _F32, n // BLOCK), _stream(stream))


def lpc_reduce_scatter_chunk(codes, scales, rank: int, chunk_codes, chunk_scales, n: int = None,
                             stream=None):
    N = len(codes)
    n = codes[0].numel() if n is None else n
    _call("lpc_reduce_scatter_chunk", _ptrs(codes, "codes", _U8, n),
          _ptrs(scales, "scales", _F32, n // BLOCK), N, rank, n,
          _dev(chunk_codes, "chunk_codes", _U8, n // max(N, 1)),
          _dev(chunk_scales, "chunk_scales", _F32, n // max(N, 1) // BLOCK), _stream(stream))


def lpc_allgather_dequant(chunk_codes, chunk_scales, out: torch.Tensor, stream=None):
    N = len(chunk_codes)
    n = out.numel()
    C = n // max(N, 1)
    _call("lpc_allgather_dequant", _ptrs(chunk_codes, "chunk_codes", _U8, C),
          _ptrs(chunk_scales, "chunk_scales", _F32, C // BLOCK), N, n, _dev(out, "out", _FB),
          _dtype(out), _stream(stream))


def lpc_rs_ag_fused(codes, scales, rank: int, chunk_codes, chunk_scales, peer_chunk_codes,
                    peer_chunk_scales, out: torch.Tensor, stream=None):
    N = len(codes)
    n = out.numel()
    C = n // max(N, 1)
    _call("lpc_rs_ag_fused", _ptrs(codes, "codes", _U8, n), _ptrs(scales, "scales", _F32, n // BLOCK),
          N, rank, n, _dev(chunk_codes, "chunk_codes", _U8, C),
          _dev(chunk_scales, "chunk_scales", _F32, C // BLOCK),
          _ptrs(peer_chunk_codes, "peer_chunk_codes", _U8, C, skip=rank),
          _ptrs(peer_chunk_scales, "peer_chunk_scales", _F32, C // BLOCK, skip=rank),
          _dev(out, "out", _FB), _dtype(out), _stream(stream))


def lpc_reduce_scatter(codes, scales, rank: int, out: torch.Tensor, n: int = None, stream=None):
    N = len(codes)
    n = codes[0].numel() if n is None else n
    _call("lpc_reduce_scatter", _ptrs(codes, "codes", _U8, n), _ptrs(scales, "scales", _F32, n // BLOCK),
          N, rank, n, _dev(out, "out", _FB, n // max(N, 1)), _dtype(out), _stream(stream))


def dda_flat_reduce(bufs, out: torch.Tensor, stream=None):
    n = out.numel()
    _call("dda_flat_reduce", _ptrs(bufs, "bufs", (torch.bfloat16,), n), len(bufs), n,
          _dev(out, "out", (torch.bfloat16,)), _stream(stream))


def dda_tree_reduce_scatter(bufs, rank: int, out: torch.Tensor, stream=None):
    N = len(bufs)
    n = bufs[0].numel()
    _call("dda_tree_reduce_scatter", _ptrs(bufs, "bufs", (out.dtype,), n), _dtype(out), N, rank, n,
          _dev(out, "out", _FB, n // max(N, 1)), _stream(stream))


def dda_tree_allgather(chunks, out: torch.Tensor, stream=None):
    N = len(chunks)
    n = out.numel()
    _call("dda_tree_allgather", _ptrs(chunks, "chunks", (out.dtype,), n // max(N, 1)), _dtype(out), N, n,
          _dev(out, "out", _FB), _stream(stream))


def lpc_a2av_route(dest: torch.Tensor, nranks: int, counts, offsets, perm, stream=None):
    rows = dest.numel()
    _call("lpc_a2av_route", _dev(dest, "dest", _I32), rows, nranks,
          _dev(counts, "counts", _I32, nranks), _dev(offsets, "offsets", _I32, nranks),
          _dev(perm, "perm", _I32, rows), _stream(stream))


def lpc_quantize_fp8_rows(x: torch.Tensor, perm: torch.Tensor, codes, scales, stream=None):
    if x.dim() != 2:
        raise ValueError("x must be 2-D (rows x row_len)")
    rows, row_len = x.shape
    _call("lpc_quantize_fp8_rows", _dev(x, "x", _FB), _dtype(x), rows, row_len,
          _dev(perm, "perm", _I32, rows), _dev(codes, "codes", _U8, rows * row_len),
          _dev(scales, "scales", _F32, rows * row_len // BLOCK), _stream(stream))


def lpc_dequantize_fp8(codes, scales, out: torch.Tensor, stream=None):
    n = out.numel()
    _call("lpc_dequantize_fp8", _dev(codes, "codes", _U8, n), _dev(scales, "scales", _F32, n // BLOCK),
          n, _dev(out, "out", _FB), _dtype(out), _stream(stream))


def lpc_select_algo(nranks: int, n: int, dtype, low_precision_enabled: bool) -> int:
    """Algorithm the library picks for an allreduce of n elements per rank (no GPU call)."""
    t = LPC_BF16 if dtype == torch.bfloat16 else LPC_F32 if dtype == torch.float32 else 99
    return lib().lpc_select_algo(nranks, n, t, 1 if low_precision_enabled else 0)


def lpc_allreduce_workspace_bytes(algo: int, nranks: int, n: int, dtype) -> int:
    out = ctypes.c_size_t(0)
    t = LPC_BF16 if dtype == torch.bfloat16 else LPC_F32 if dtype == torch.float32 else 99
    _call("lpc_allreduce_workspace_bytes", algo, nranks, n, t, ctypes.byref(out))
    return out.value


def lpc_allreduce_emulated(bufs, algo: int, workspace: torch.Tensor, stream=None):
    """In-place allreduce (SUM) of the N rank buffers `bufs` (same shape and dtype)."""
    N = len(bufs)
    n = bufs[0].numel()
    dt = bufs[0].dtype
    _call("lpc_allreduce_emulated", _ptrs(bufs, "bufs", (dt,), n), N, n, _dtype(bufs[0]), algo,
          _dev(workspace, "workspace", _U8), workspace.numel(), _stream(stream))


def lpc_allreduce_emulated_noalloc(bufs, algo: int, stream=None):
    """lpc_allreduce_emulated with the library's static scratch in place of a workspace
    (allocates nothing; calls that overlap on one GPU race on the scratch)."""
    N = len(bufs)
    n = bufs[0].numel()
    dt = bufs[0].dtype
    _call("lpc_allreduce_emulated_noalloc", _ptrs(bufs, "bufs", (dt,), n), N, n, _dtype(bufs[0]), algo,
          _stream(stream))


def lpc_measure_stream(src, read_bytes: int, dst, write_bytes: int, per_lane: int = 0, stream=None):
    """Plain streaming kernel (measurement reference): reads read_bytes of src, writes write_bytes
    of dst (with write_bytes == 0, dst is a never-written sink of at least 16 bytes); per_lane 0
    is one round of resident wavefronts, 1/2/4/8 that many vectors per lane."""
    if src is not None and src.numel() * src.element_size() < read_bytes:
        raise ValueError("src holds fewer than %d bytes" % read_bytes)
    if dst is not None and dst.numel() * dst.element_size() < max(write_bytes, 16 if read_bytes else 0):
        raise ValueError("dst holds fewer than %d bytes" % max(write_bytes, 16))
    _call("lpc_measure_stream", _dev(src, "src") if src is not None else None, read_bytes,
          _dev(dst, "dst") if dst is not None else None, write_bytes, per_lane, _stream(stream))


def lpc_measure_empty(grid_x: int, grid_y: int, threads: int, kernarg_bytes: int, sink, stream=None):
    """Empty launch of the given shape (measurement reference); sink is never written."""
    _call("lpc_measure_empty", grid_x, grid_y, threads, kernarg_bytes, _dev(sink, "sink", None, 1),
          _stream(stream))


def lpc_e4m3_encode(x: torch.Tensor, codes: torch.Tensor, stream=None):
    n = x.numel()
    _call("lpc_e4m3_encode", _dev(x, "x", _F32), n, _dev(codes, "codes", _U8, n), _stream(stream))


# ---------------------------------------------------------------------------
# training and serving operators (include/lpc_ops.h)
#
# One operator call is a few microseconds of GPU work at its smallest, so these
# marshal with plain integers and run on the tensors' own device: all tensors of
# a call must be on one GPU, and the work goes to that GPU's current stream
# unless another is given.
# ---------------------------------------------------------------------------

_u8, _f4, _i4, _MASK = torch.uint8, torch.float32, torch.int32, (torch.uint8, torch.bool)


class _Args:
    """Pointers of one call's tensors, checked as _dev checks them and to be on one GPU."""

    __slots__ = ("device",)

    def __init__(self):
        self.device = None

    def __call__(self, t, what, dtypes, numel, exact=False):
        if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous():
            n, d = t.numel(), t.get_device()
            if (n == numel or (n > numel and not exact)) and (d == self.device or self.device is None):
                self.device = d
                return t.data_ptr()
        raise self.fault(t, what, dtypes, numel, exact)

    def fault(self, t, what, dtypes, numel, exact):
        """What is wrong with an argument that was refused."""
        if not isinstance(t, torch.Tensor):
            return TypeError("%s must be a torch tensor" % what)
        if not t.is_cuda:
            return ValueError("%s must be a GPU tensor" % what)
        if not t.is_contiguous():
            return ValueError("%s must be contiguous" % what)
        if t.dtype not in dtypes:
            return TypeError("%s has dtype %s, expected one of %s" % (what, t.dtype, dtypes))
        n = t.numel()
        if n < numel or (exact and n != numel):
            return ValueError("%s holds %d elements, needs %d" % (what, n, numel))
        return ValueError("%s is on cuda:%d, the other tensors on cuda:%d" % (what, t.get_device(), self.device))

    def optional(self, t, what, dtypes, numel):
        return None if t is None else self(t, what, dtypes, numel)

    def many(self, ts, what, dtypes, numels):
        """Pointers of a list's tensors, each of exactly its number of elements."""
        first = self(ts[0], what + "[0]", dtypes, numels[0], True)
        dtype, device = ts[0].dtype, ts[0].device
        out = [first]
        for i in range(1, len(ts)):
            t = ts[i]
            try:
                alike = t.dtype is dtype and t.device == device and t.numel() == numels[i] and t.is_contiguous()
            except AttributeError:
                alike = False
            out.append(t.data_ptr() if alike else self(t, "%s[%d]" % (what, i), dtypes, numels[i], True))
        return out


def _run(name, device, stream, *args):
    """Call an entry point whose last argument is the stream, with `device` current."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    f = getattr(_lib or lib(), name)
    if torch._C._cuda_getDevice() == device:
        st = f(*args, stream)
    else:
        with torch.cuda.device(device):
            st = f(*args, stream)
    if st != 0:
        raise LpcError(name, st, lpc_status_string(st))


def _torch_stream(stream, device):
    return stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)


def _scratch(size, device, stream):
    """Device memory for one call.  It comes from the pool of the stream that the call runs on: a block of another
    stream's pool may still be in use there, and nothing would order the call after that."""
    if stream is None:
        return torch.empty(size, dtype=_u8, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        return torch.empty(size, dtype=_u8, device=device)


def _shape2(t, what):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % what)
    return t.shape


def _groups(counts):
    return 1 if counts is None else counts.numel()


def _blocks(n):
    return -(-n // BLOCK)


def lpc_gemm_fp8(x, xs, w, ws, out, counts=None, stream=None):
    """out [rows, n] = x [rows, k] times w [groups, n, k] (or [n, k]) transposed, E4M3 codes with scales
    xs [rows, k/128] and ws [groups, ceil(n/128), k/128]; counts [groups] int32: rows of each group.  Sums are FP32 where
    out is; for a bf16 out the matrix instruction drops what is small beside the largest of 8 neighbouring products
    (include/lpc_ops.h gives the bound)."""
    # A small product takes less time on the GPU than its call does here, so what is usual is looked at in one expression
    # (5.9 us a call against 7.5); anything else goes through the checks below, which say what is wrong.
    try:
        (rows, k), (n, kw), device = x.shape, w.shape[-2:], x.get_device()
        groups, blocks = 1 if counts is None else counts.numel(), k // BLOCK
        usual = (stream is None and device >= 0 and kw == k and out.shape == (rows, n) and w.numel() == groups * n * k
                 and xs.numel() == rows * blocks and ws.numel() == groups * -(-n // BLOCK) * blocks
                 and x.dtype is _u8 and w.dtype is _u8 and xs.dtype is _f4 and ws.dtype is _f4
                 and x.is_contiguous() and w.is_contiguous() and xs.is_contiguous() and ws.is_contiguous()
                 and out.is_contiguous() and w.get_device() == device and xs.get_device() == device
                 and ws.get_device() == device and out.get_device() == device and w.dim() < 4
                 and (counts is None or (counts.dtype is _i4 and counts.is_contiguous() and counts.get_device() == device)))
    except (AttributeError, TypeError, ValueError):
        usual = False
    if usual:
        return _run("lpc_gemm_fp8", device, None, x.data_ptr(), xs.data_ptr(), rows, k, w.data_ptr(), ws.data_ptr(), n, groups,
                    None if counts is None else counts.data_ptr(), out.data_ptr(), _dtype(out))
    rows, k = _shape2(x, "x")
    n, kw = w.shape[-2:]
    groups = _groups(counts)
    if kw != k or w.dim() not in (2, 3) or w.numel() != groups * n * k:
        raise ValueError("w has shape %s, expected [%d, n, %d]" % (tuple(w.shape), groups, k))
    if _shape2(out, "out") != (rows, n):
        raise ValueError("out has shape %s, expected [%d, %d]" % (tuple(out.shape), rows, n))
    p = _Args()
    args = (p(x, "x", _U8, 0), p(xs, "xs", _F32, rows * (k // BLOCK), True), rows, k, p(w, "w", _U8, 0),
            p(ws, "ws", _F32, groups * _blocks(n) * (k // BLOCK), True), n, groups,
            p.optional(counts, "counts", _I32, 1), p(out, "out", _FB, 0), _dtype(out))
    _run("lpc_gemm_fp8", p.device, stream, *args)


def lpc_padded_rows(rows: int, groups: int) -> int:
    """Rows of the padded column layout for any counts (no GPU call)."""
    return lib().lpc_padded_rows(rows, groups)


def lpc_quantize_fp8_cols(y, codes_t, scales_t, codes=None, scales=None, counts=None, stream=None):
    """Column codes [n, padded] and scales [padded/128, n] of y [rows, n], and in the same pass its row
    codes [rows, n] and scales [rows, n/128] where those are given."""
    rows, n = _shape2(y, "y")
    groups = _groups(counts)
    padded = lpc_padded_rows(rows, groups)
    p = _Args()
    args = (p(y, "y", _FB, 0), _dtype(y), rows, n, groups, p.optional(counts, "counts", _I32, 1),
            p(codes_t, "codes_t", _U8, padded * n, True), p(scales_t, "scales_t", _F32, padded // BLOCK * n, True),
            p.optional(codes, "codes", _U8, rows * n), p.optional(scales, "scales", _F32, rows * n // BLOCK))
    _run("lpc_quantize_fp8_cols", p.device, stream, *args)


def lpc_requantize_fp8_cols(x, xs, codes_t, scales_t, counts=None, stream=None):
    """Column codes [k, padded] and scales [padded/128, k] of the rows that codes x [rows, k] and scales
    xs [rows, k/128] hold."""
    rows, k = _shape2(x, "x")
    groups = _groups(counts)
    padded = lpc_padded_rows(rows, groups)
    p = _Args()
    args = (p(x, "x", _U8, 0), p(xs, "xs", _F32, rows * (k // BLOCK), True), rows, k, groups,
            p.optional(counts, "counts", _I32, 1), p(codes_t, "codes_t", _U8, padded * k, True),
            p(scales_t, "scales_t", _F32, padded // BLOCK * k, True))
    _run("lpc_requantize_fp8_cols", p.device, stream, *args)


def lpc_gemm_fp8_wgrad(yt, ys, xt, xs, dw, rows: int, counts=None, stream=None):
    """dw [groups, n, k] (or [n, k]) fp32 from the column forms of the incoming gradient, yt [n, padded],
    and of the rows, xt [k, padded]."""
    n, k = dw.shape[-2:]
    groups = _groups(counts)
    if dw.dim() not in (2, 3) or dw.numel() != groups * n * k:
        raise ValueError("dw has shape %s, expected [%d, n, k]" % (tuple(dw.shape), groups))
    padded = lpc_padded_rows(rows, groups)
    p = _Args()
    args = (p(yt, "yt", _U8, n * padded, True), p(ys, "ys", _F32, n * (padded // BLOCK), True), n,
            p(xt, "xt", _U8, k * padded, True), p(xs, "xs", _F32, k * (padded // BLOCK), True), k, rows, groups,
            p.optional(counts, "counts", _I32, 1), p(dw, "dw", _F32, 0))
    _run("lpc_gemm_fp8_wgrad", p.device, stream, *args)


def lpc_router_workspace_bytes(rows: int, experts: int) -> int:
    """Device workspace of lpc_router_forward (no GPU call)."""
    return (_lib or lib()).lpc_router_workspace_bytes(rows, experts)


def lpc_router_forward(logits, experts, gates, counts, load, slope, loss, coef: float, normalize: bool = True,
                       mask=None, workspace=None, stream=None):
    """Routing of logits [rows, E]: experts (int32) and gates [rows, topk], counts (int32), load and slope [E],
    loss [1].  Without a workspace (uint8, lpc_router_workspace_bytes) one is taken from torch's allocator."""
    try:  # the usual call in one expression, as in lpc_gemm_fp8
        (rows, e), (r2, topk), device = logits.shape, experts.shape, logits.get_device()
        usual = (stream is None and workspace is None and device >= 0 and r2 == rows
                 and gates.numel() == rows * topk and counts.numel() == e and load.numel() == e and slope.numel() == e
                 and loss.numel() == 1 and (logits.dtype is _f4 or logits.dtype is torch.bfloat16)
                 and experts.dtype is _i4 and counts.dtype is _i4 and gates.dtype is _f4 and load.dtype is _f4
                 and slope.dtype is _f4 and loss.dtype is _f4 and logits.is_contiguous() and experts.is_contiguous()
                 and gates.is_contiguous() and counts.is_contiguous() and load.is_contiguous() and slope.is_contiguous()
                 and experts.get_device() == device and gates.get_device() == device and counts.get_device() == device
                 and load.get_device() == device and slope.get_device() == device and loss.get_device() == device
                 and (mask is None or (mask.dtype in _MASK and mask.numel() == rows and mask.is_contiguous()
                                       and mask.get_device() == device)))
    except (AttributeError, TypeError, ValueError):
        usual = False
    if usual:
        need = lpc_router_workspace_bytes(rows, e)
        space = torch.empty(need, dtype=_u8, device=logits.device) if need else None
        return _run("lpc_router_forward", device, None, logits.data_ptr(), LPC_F32 if logits.dtype is _f4 else LPC_BF16, rows, e,
                    topk, 1 if normalize else 0, coef, None if mask is None else mask.data_ptr(), experts.data_ptr(),
                    gates.data_ptr(), counts.data_ptr(), load.data_ptr(), slope.data_ptr(), loss.data_ptr(),
                    None if space is None else space.data_ptr(), need)
    rows, e = _shape2(logits, "logits")
    r2, topk = _shape2(experts, "experts")
    if r2 != rows:
        raise ValueError("experts has %d rows, expected %d" % (r2, rows))
    p = _Args()
    args = [p(logits, "logits", _FB, 0), _dtype(logits), rows, e, topk, 1 if normalize else 0, coef,
            p.optional(mask, "mask", _MASK, rows), p(experts, "experts", _I32, 0),
            p(gates, "gates", _F32, rows * topk, True), p(counts, "counts", _I32, e, True),
            p(load, "load", _F32, e, True), p(slope, "slope", _F32, e, True), p(loss, "loss", _F32, 1, True)]
    need = lpc_router_workspace_bytes(rows, e)
    if workspace is None and need:
        workspace = _scratch(need, logits.device, stream)
    space = (None, 0) if workspace is None else (p(workspace, "workspace", _U8, 0), workspace.numel())
    _run("lpc_router_forward", p.device, stream, *args, *space)


def lpc_router_backward(logits, experts, slope, dgates, dloss, dlogits, normalize: bool = True, mask=None, stream=None):
    """dlogits [rows, E] from dgates [rows, topk] and dloss [1], with the forward call's experts and slope."""
    try:  # the usual call in one expression, as in lpc_gemm_fp8
        (rows, e), (r2, topk), device = logits.shape, experts.shape, logits.get_device()
        usual = (stream is None and device >= 0 and r2 == rows and slope.numel() == e and dgates.numel() == rows * topk
                 and dloss.numel() == 1 and dlogits.numel() == rows * e and dlogits.dtype is logits.dtype
                 and (logits.dtype is _f4 or logits.dtype is torch.bfloat16) and experts.dtype is _i4 and slope.dtype is _f4
                 and dgates.dtype is _f4 and dloss.dtype is _f4 and logits.is_contiguous() and experts.is_contiguous()
                 and slope.is_contiguous() and dgates.is_contiguous() and dlogits.is_contiguous()
                 and experts.get_device() == device and slope.get_device() == device and dgates.get_device() == device
                 and dloss.get_device() == device and dlogits.get_device() == device
                 and (mask is None or (mask.dtype in _MASK and mask.numel() == rows and mask.is_contiguous()
                                       and mask.get_device() == device)))
    except (AttributeError, TypeError, ValueError):
        usual = False
    if usual:
        return _run("lpc_router_backward", device, None, logits.data_ptr(), LPC_F32 if logits.dtype is _f4 else LPC_BF16, rows, e,
                    topk, 1 if normalize else 0, None if mask is None else mask.data_ptr(), experts.data_ptr(),
                    slope.data_ptr(), dgates.data_ptr(), dloss.data_ptr(), dlogits.data_ptr())
    rows, e = _shape2(logits, "logits")
    r2, topk = _shape2(experts, "experts")
    if r2 != rows or dlogits.dtype != logits.dtype:
        raise ValueError("experts and dlogits do not match logits")
    p = _Args()
    args = (p(logits, "logits", _FB, 0), _dtype(logits), rows, e, topk, 1 if normalize else 0,
            p.optional(mask, "mask", _MASK, rows), p(experts, "experts", _I32, 0),
            p(slope, "slope", _F32, e, True), p(dgates, "dgates", _F32, rows * topk, True),
            p(dloss, "dloss", _F32, 1, True), p(dlogits, "dlogits", _FB, rows * e, True))
    _run("lpc_router_backward", p.device, stream, *args)


class AdamW:
    """AdamW over many tensors in one launch a step (lpc_adamw_plan, lpc_adamw_step).

    params (fp32), grads (all fp32 or all bf16) and the moments m, v are lists of contiguous tensors, checked once
    and updated in place; the tensors must stay where they are.  With m_scales and v_scales the moments are E4M3
    codes (uint8) with one fp32 scale per 128 elements, v holding the root of the second moment.  copies: bf16
    tensors that get the updated params.  A step reads no tensor's address again, so it can be captured in a graph
    (its hyperparameters are then the captured ones; the object has to live as long as the graph is replayed), and a
    gradient that a program replaces by another tensor needs a new AdamW."""

    def __init__(self, params, grads, m, v, m_scales=None, v_scales=None, copies=None):
        if (m_scales is None) != (v_scales is None):
            raise ValueError("m_scales and v_scales come together")
        self.state_bits = 32 if m_scales is None else 8
        lists = {"grads": grads, "m": m, "v": v, "m_scales": m_scales, "v_scales": v_scales, "copies": copies}
        for what, ts in lists.items():
            if ts is not None and len(ts) != len(params):
                raise ValueError("%s has %d tensors, params %d" % (what, len(ts), len(params)))
        state = _F32 if self.state_bits == 32 else _U8
        p, rows = _Args(), max(len(params), 1)
        table = (_AdamwTensor * rows)()
        columns = np.frombuffer(table, dtype=np.uint64).reshape(rows, -1)  # one 8-byte field each, in the order of _fields_
        sizes = [t.numel() if isinstance(t, torch.Tensor) else 0 for t in params]
        blocks = [_blocks(n) for n in sizes]
        states = (m, "m", state, sizes), (v, "v", state, sizes)
        scales = (m_scales, "m_scales", _F32, blocks), (v_scales, "v_scales", _F32, blocks)
        fields = ((params, "params", _F32, sizes), (grads, "grads", (grads[0].dtype,) if len(params) else _FB, sizes), *states,
                  *scales, (copies, "copies", (torch.bfloat16,), sizes))
        for column, (ts, what, dtypes, ns) in enumerate(fields):
            if ts is not None and len(ts):
                columns[:, column] = p.many(ts, what, dtypes, ns)
        if len(params):
            columns[:, len(fields)] = sizes
        self.grad_dtype = _dtype(grads[0]) if len(params) else LPC_F32
        self.device = p.device
        self._tensors = (list(params), {k: list(ts) for k, ts in lists.items() if ts is not None})  # kept alive
        size = lib().lpc_adamw_plan_bytes(table, len(params))
        host = torch.empty(size, dtype=torch.uint8)
        chunks = ctypes.c_size_t(0)
        _call("lpc_adamw_plan", table, len(params), self.grad_dtype, self.state_bits, host.data_ptr() if size else None, size,
              ctypes.byref(chunks))
        self._chunks = chunks.value
        self._plan = host.to("cuda:%d" % self.device) if self._chunks else None
        # streams after whose work the plan may be handed out again when this object goes: that of its pool, and those of steps
        self._streams = {torch._C._cuda_getCurrentRawStream(self.device)} if self._chunks else set()

    def step(self, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             weight_decay: float = 0.01, grad_scale=None, stream=None):
        """Update `step` (counted from 1); grad_scale: a GPU tensor whose first element multiplies every gradient."""
        if self._plan is None:
            return
        p = _Args()
        p.device = self.device
        handle = torch._C._cuda_getCurrentRawStream(self.device) if stream is None else getattr(stream, "cuda_stream", stream)
        if handle not in self._streams:
            self._plan.record_stream(_torch_stream(handle, self._plan.device))
            self._streams.add(handle)
        _run("lpc_adamw_step", self.device, handle, self._plan.data_ptr(), self._chunks, self.grad_dtype,
             self.state_bits, step, lr, beta1, beta2, eps, weight_decay, p.optional(grad_scale, "grad_scale", _F32, 1))

"""ctypes binding of libdiffattn (include/diffattn.h): argument marshalling only.

Every computation runs inside the library's CUDA kernels.  PyTorch supplies
device memory and the current stream; this module only checks that tensors
have the layout the C ABI documents, then passes raw pointers.  If the shared
library has not been built, the first call raises; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdiffattn.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "diffattn.h")
PAGED_HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "diffattn_paged.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_BOUNDS = 0, 1, 2, 3, 4, 5
ERR_PAGE = 6
BF16, F32, E4M3_QK = 0, 1, 2
_DTYPE_CODE = {torch.bfloat16: BF16, torch.float32: F32}


class DiffAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libdiffattn status {status}: {message}")
        self.status = status


class Desc(ctypes.Structure):
    """Mirror of `diffattn_desc` in include/diffattn.h."""
    _fields_ = [
        ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("headnorm", ctypes.c_int32), ("eps", ctypes.c_float), ("lambda_init", ctypes.c_float),
        ("status_dev", ctypes.c_void_p),
    ]


class Strides(ctypes.Structure):
    """Mirror of `diffattn_strides` (element strides of batch, head, row)."""
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


class PagedCacheStruct(ctypes.Structure):
    """Mirror of `diffpaged_cache` in include/diffattn_paged.h."""
    _fields_ = [
        ("k1", ctypes.c_void_p), ("k2", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("weights", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p),
        ("k1_strides", Strides), ("k2_strides", Strides), ("v_strides", Strides),
        ("num_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
        ("max_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libdiffattn.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        _lib = bind(ctypes.CDLL(path))
        return _lib


@contextlib.contextmanager
def using(lib):
    """Route this module's calls to another bound library (e.g. the
    bounds-checked debug build) for the duration of a `with` block."""
    global _lib
    with _lock:
        prev, _lib = _lib, lib
    try:
        yield lib
    finally:
        with _lock:
            _lib = prev


def bind(lib):
    """Declare the C signatures of include/diffattn.h on a loaded library."""
    vp, fp = ctypes.c_void_p, ctypes.c_void_p
    dp = ctypes.POINTER(Desc)
    lib.diffattn_fwd.restype = ctypes.c_int
    lib.diffattn_fwd.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp, vp]
    lib.diffattn_fwd_kv.restype = ctypes.c_int
    lib.diffattn_fwd_kv.argtypes = [dp, ctypes.c_int64, vp, vp, vp, vp, vp, fp, fp, vp,
                                    ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.diffattn_fwd_kv_plan.restype = ctypes.c_int
    lib.diffattn_fwd_kv_plan.argtypes = [dp, ctypes.c_int64, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_size_t)]
    lib.diffattn_fwd_kv_noalloc.restype = ctypes.c_int
    lib.diffattn_fwd_kv_noalloc.argtypes = [dp, ctypes.c_int64, vp, vp, vp, vp, vp, fp, fp,
                                            vp, ctypes.c_int, vp]
    lib.diffattn_train_sizes.restype = ctypes.c_int
    lib.diffattn_train_sizes.argtypes = [dp, ctypes.POINTER(ctypes.c_size_t),
                                         ctypes.POINTER(ctypes.c_size_t)]
    lib.diffattn_fwd_train.restype = ctypes.c_int
    lib.diffattn_fwd_train.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp, vp,
                                       ctypes.c_size_t, vp]
    lib.diffattn_bwd.restype = ctypes.c_int
    lib.diffattn_bwd.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp, vp, vp, vp, vp, vp, vp,
                                 fp, fp, vp, ctypes.c_size_t, vp]
    lib.diffattn_fwd_host.restype = ctypes.c_int
    lib.diffattn_fwd_host.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp, vp, ctypes.c_size_t,
                                      vp]
    lib.diffattn_fwd_host_staging_bytes.restype = ctypes.c_int
    lib.diffattn_fwd_host_staging_bytes.argtypes = [dp, ctypes.POINTER(ctypes.c_size_t)]
    lib.diffattn_fwd_strided.restype = ctypes.c_int
    lib.diffattn_fwd_strided.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp,
                                         ctypes.POINTER(Strides), vp]
    lib.diffattn_fwd_train_strided.restype = ctypes.c_int
    lib.diffattn_fwd_train_strided.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp, vp,
                                               ctypes.c_size_t, ctypes.POINTER(Strides), vp]
    lib.diffattn_bwd_strided.restype = ctypes.c_int
    lib.diffattn_bwd_strided.argtypes = [dp, vp, vp, vp, vp, vp, fp, fp, vp, vp, vp, vp, vp, vp,
                                         vp, fp, fp, vp, ctypes.c_size_t,
                                         ctypes.POINTER(Strides), vp]
    lib.diffattn_fwd_kv_strided.restype = ctypes.c_int
    lib.diffattn_fwd_kv_strided.argtypes = [dp, ctypes.c_int64, vp, vp, vp, vp, vp, fp, fp,
                                            vp, ctypes.c_int, vp, ctypes.c_size_t,
                                            ctypes.POINTER(Strides), vp]
    cp, szp, i64 = ctypes.POINTER(PagedCacheStruct), ctypes.POINTER(ctypes.c_size_t), ctypes.c_int64
    for name, args in (
            ("append", [dp, cp, vp, vp, vp, ctypes.POINTER(Strides), vp]),
            ("fwd_plan", [dp, cp, ctypes.c_int, szp]),
            ("fwd", [dp, cp, vp, vp, fp, fp, vp, ctypes.POINTER(Strides), ctypes.c_int, vp,
                     ctypes.c_size_t, vp]),
            ("evict_plan", [dp, cp, i64, szp]),
            ("evict", [dp, cp, i64, i64, vp, ctypes.c_size_t, vp])):
        fn = getattr(lib, "diffpaged_" + name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    lib.diffattn_selftest_wait.restype = ctypes.c_int
    lib.diffattn_selftest_wait.argtypes = [vp, ctypes.c_int64, vp]
    lib.diffattn_headnorm.restype = ctypes.c_int
    lib.diffattn_headnorm.argtypes = [dp, fp, fp, vp, vp]
    lib.diffattn_lambda_init.restype = ctypes.c_double
    lib.diffattn_lambda_init.argtypes = [ctypes.c_int]
    lib.diffattn_strerror.restype = ctypes.c_char_p
    lib.diffattn_strerror.argtypes = [ctypes.c_int]
    lib.diffattn_version.restype = ctypes.c_int
    lib.diffattn_version.argtypes = []
    return lib


def declared_symbols(header: str = HEADER_PATH) -> list[str]:
    """Names of the functions include/diffattn.h declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"\b(diffattn_[a-z0-9_]+)\s*\(", text)))


def strerror(status: int) -> str:
    return load().diffattn_strerror(int(status)).decode()


def lambda_init(layer: int) -> float:
    """lambda_init(l) = 0.8 - 0.6 exp(-0.3 (l - 1)), computed by the library."""
    return float(load().diffattn_lambda_init(int(layer)))


def _check(status: int):
    if status != OK:
        raise DiffAttnError(status, strerror(status))


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_desc(B, H, N, d, dtype_code, causal, headnorm, eps, lambda_init_value, status=None):
    return Desc(int(B), int(H), int(N), int(d), int(dtype_code), int(bool(causal)),
                int(headnorm), float(eps), float(lambda_init_value),
                None if status is None else status.data_ptr())


def fwd(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: int = 1, norm_w=None,
        eps: float = 1e-5, lambda_init: float = 0.0, out=None, status=None, stream=None,
        raw_status: bool = False):
    """Differential-attention head forward through `diffattn_fwd`.

    q1, k1, q2, k2: [B, H, N, d]; v: [B, H, N, 2d] (all bf16 or all fp32, CUDA,
    contiguous); lam: float32 [H]; norm_w: float32 [H, 2d] or None.  headnorm:
    0 none, 1 (or True) RMS form, 2 mean-subtracting group form.  Returns
    `out` [B, H, N, 2d] (allocated by torch when not given).  With
    raw_status=True the status code is returned instead of raising.
    """
    if q1.dim() != 4:
        raise ValueError("q1 must be [B, H, N, d]")
    B, H, N, d = q1.shape
    dtype = q1.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    for name, t, shape in (("k1", k1, (B, H, N, d)), ("q2", q2, (B, H, N, d)),
                           ("k2", k2, (B, H, N, d)), ("v", v, (B, H, N, 2 * d))):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name} must be {shape} {dtype}")
    tensors = [q1, k1, q2, k2, v, lam] + ([norm_w] if norm_w is not None else [])
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=dtype, device=q1.device)
    tensors.append(out)
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if norm_w is not None and (norm_w.dtype != torch.float32 or norm_w.numel() != H * 2 * d):
        raise ValueError("norm_w must be float32 [H, 2d]")
    if tuple(out.shape) != (B, H, N, 2 * d) or out.dtype != dtype:
        raise ValueError("out must be [B, H, N, 2d] of the input dtype")
    desc = make_desc(B, H, N, d, _DTYPE_CODE[dtype], causal, headnorm, eps, lambda_init, status)
    st = load().diffattn_fwd(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(v),
                             _ptr(lam), _ptr(norm_w), _ptr(out), _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


def fwd_host_staging_bytes(B, H, N, d, dtype=torch.bfloat16) -> int:
    """`diffattn_fwd_host_staging_bytes`: device staging bytes `fwd_host` needs."""
    desc = make_desc(B, H, N, d, _DTYPE_CODE[dtype], True, 1, 1e-5, 0.0)
    n = ctypes.c_size_t(0)
    _check(load().diffattn_fwd_host_staging_bytes(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def fwd_host(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: int = 1, norm_w=None,
             eps: float = 1e-5, lambda_init: float = 0.0, out=None, staging=None, status=None,
             stream=None, raw_status: bool = False):
    """`diffattn_fwd_host`: the forward with q1, k1, q2, k2, v and out in host memory.

    q1, k1, q2, k2, v: contiguous CPU tensors (bf16 or fp32; pinned keeps the copies
    asynchronous); lam (float32 [H]) and norm_w stay CUDA tensors; staging: a CUDA
    uint8 tensor of at least fwd_host_staging_bytes(...) bytes (allocated when not
    given).  Returns the CPU `out` [B, H, N, 2d], filled once `stream` reaches the
    end of the call.
    """
    B, H, N, d = q1.shape
    dtype = q1.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    for name, t, shape in (("q1", q1, (B, H, N, d)), ("k1", k1, (B, H, N, d)),
                           ("q2", q2, (B, H, N, d)), ("k2", k2, (B, H, N, d)),
                           ("v", v, (B, H, N, 2 * d))):
        if tuple(t.shape) != shape or t.dtype != dtype or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU {shape} {dtype} tensor")
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=dtype).pin_memory()
    if out.is_cuda or not out.is_contiguous() or tuple(out.shape) != (B, H, N, 2 * d):
        raise ValueError("out must be a contiguous CPU [B, H, N, 2d] tensor")
    if not lam.is_cuda or lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be a CUDA float32 [H] tensor")
    need = fwd_host_staging_bytes(B, H, N, d, dtype)
    if staging is None:
        staging = torch.empty(need, dtype=torch.uint8, device=lam.device)
    if not staging.is_cuda or staging.numel() < need:
        raise ValueError(f"staging must be a CUDA uint8 tensor of at least {need} bytes")
    desc = make_desc(B, H, N, d, _DTYPE_CODE[dtype], causal, headnorm, eps, lambda_init, status)
    st = load().diffattn_fwd_host(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2),
                                  _ptr(v), _ptr(lam), _ptr(norm_w), _ptr(out), _ptr(staging),
                                  staging.numel(), _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


def fwd_fp8(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: int = 1, norm_w=None,
            eps: float = 1e-5, lambda_init: float = 0.0, out=None, status=None, stream=None,
            raw_status: bool = False):
    """`diffattn_fwd` with DIFFATTN_E4M3_QK: q1, k1, q2, k2 torch.float8_e4m3fn
    [B, H, N, 64]; v bf16 [B, H, N, 128]; returns bf16 out [B, H, N, 128]."""
    B, H, N, d = q1.shape
    for t in (q1, k1, q2, k2):
        if t.dtype != torch.float8_e4m3fn or tuple(t.shape) != (B, H, N, d):
            raise ValueError("q1, k1, q2, k2 must be float8_e4m3fn [B, H, N, d]")
    if v.dtype != torch.bfloat16 or tuple(v.shape) != (B, H, N, 2 * d):
        raise ValueError("v must be bfloat16 [B, H, N, 2d]")
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=torch.bfloat16, device=q1.device)
    _cuda_contig([q1, k1, q2, k2, v, lam, norm_w, out])
    desc = make_desc(B, H, N, d, E4M3_QK, causal, headnorm, eps, lambda_init, status)
    st = load().diffattn_fwd(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(v),
                             _ptr(lam), _ptr(norm_w), _ptr(out), _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


def fwd_strided(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: int = 1, norm_w=None,
                eps: float = 1e-5, lambda_init: float = 0.0, out=None, status=None,
                stream=None, raw_status: bool = False):
    """`diffattn_fwd_strided`: the bf16 forward on [B, H, N, d]-shaped views of any
    layout whose rows are contiguous (e.g. x.permute(0, 2, 1, 3) of [B, N, H, d]
    storage); `out` may be such a view too (default: a contiguous tensor)."""
    B, H, N, d = q1.shape
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=q1.dtype, device=q1.device)
    ts = [q1, k1, q2, k2, v, out]
    arr = _view_strides(ts, [(B, H, N, d)] * 4 + [(B, H, N, 2 * d)] * 2, q1.dtype)
    _cuda_contig([lam, norm_w])
    desc = make_desc(B, H, N, d, _DTYPE_CODE.get(q1.dtype, -1), causal, headnorm, eps,
                     lambda_init, status)
    st = load().diffattn_fwd_strided(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2),
                                     _ptr(v), _ptr(lam), _ptr(norm_w), _ptr(out), arr,
                                     _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


def _view_strides(ts, shapes, dtype):
    """Checks [B, H, rows, width]-shaped CUDA views with contiguous rows and
    returns their (batch, head, row) element strides as a Strides array."""
    for t, shape in zip(ts, shapes):
        if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_cuda:
            raise ValueError(f"expected a CUDA {dtype} tensor of shape {tuple(shape)}")
        if t.stride(-1) != 1:
            raise ValueError("rows must be contiguous (last stride 1)")
    return (Strides * len(ts))(*[Strides(t.stride(0), t.stride(1), t.stride(2)) for t in ts])


def fwd_kv_plan(B, H, N, n_kv, *, causal: bool, splits: int = 0, d: int = 64,
                headnorm: bool = True, raw_status: bool = False):
    """`diffattn_fwd_kv_plan`: (split count that will run, workspace bytes)."""
    desc = make_desc(B, H, N, d, BF16, causal, headnorm, 1e-5, 0.0)
    sp, nb = ctypes.c_int(0), ctypes.c_size_t(0)
    st = load().diffattn_fwd_kv_plan(ctypes.byref(desc), int(n_kv), int(splits),
                                     ctypes.byref(sp), ctypes.byref(nb))
    if raw_status:
        return st, sp.value, nb.value
    _check(st)
    return sp.value, nb.value


def _kv_dtypes(q1):
    """(dtype code, value and output dtype) of a key/value-cache call: bf16
    throughout, or e4m3 queries/keys (DIFFATTN_E4M3_QK) with bf16 values and output."""
    if q1.dtype == torch.float8_e4m3fn:
        return E4M3_QK, torch.bfloat16
    return _DTYPE_CODE.get(q1.dtype, -1), q1.dtype


def fwd_kv(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: bool = True, norm_w=None,
           eps: float = 1e-5, lambda_init: float = 0.0, splits: int = 0, workspace=None,
           out=None, status=None, stream=None, raw_status: bool = False):
    """Forward of Nq queries against Nkv keys through `diffattn_fwd_kv` (d = 64).

    q1, q2: [B, H, Nq, 64]; k1, k2: [B, H, Nkv, 64]; v: [B, H, Nkv, 128]; the
    queries are the last Nq positions.  All bf16, or q1, k1, q2, k2
    float8_e4m3fn with bf16 v (DIFFATTN_E4M3_QK).  splits = 0 lets the library
    choose.  workspace: a CUDA tensor of at least the planned bytes, or None (a
    torch buffer of the planned size is used).  Returns bf16 out [B, H, Nq, 128].
    """
    if q1.dim() != 4 or k1.dim() != 4:
        raise ValueError("q1 and k1 must be [B, H, N, d]")
    B, H, N, d = q1.shape
    n_kv = k1.shape[2]
    code, vdtype = _kv_dtypes(q1)
    for name, t, shape, dt in (("q2", q2, (B, H, N, d), q1.dtype),
                               ("k1", k1, (B, H, n_kv, d), q1.dtype),
                               ("k2", k2, (B, H, n_kv, d), q1.dtype),
                               ("v", v, (B, H, n_kv, 2 * d), vdtype)):
        if tuple(t.shape) != shape or t.dtype != dt:
            raise ValueError(f"{name} must be {shape} {dt}")
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=vdtype, device=q1.device)
    if tuple(out.shape) != (B, H, N, 2 * d) or out.dtype != vdtype:
        raise ValueError(f"out must be [B, H, Nq, 2d] {vdtype}")
    tensors = [q1, k1, q2, k2, v, lam, out] + ([norm_w] if norm_w is not None else [])
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if norm_w is not None and (norm_w.dtype != torch.float32 or norm_w.numel() != H * 2 * d):
        raise ValueError("norm_w must be float32 [H, 2d]")
    desc = make_desc(B, H, N, d, code, causal, headnorm, eps, lambda_init, status)
    lib = load()
    if workspace is None:
        sp, nb = ctypes.c_int(0), ctypes.c_size_t(0)
        st = lib.diffattn_fwd_kv_plan(ctypes.byref(desc), int(n_kv), int(splits),
                                      ctypes.byref(sp), ctypes.byref(nb))
        if st != OK:
            if raw_status:
                return st
            _check(st)
        if nb.value:
            workspace = torch.empty(nb.value, dtype=torch.uint8, device=q1.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.diffattn_fwd_kv(ctypes.byref(desc), int(n_kv), _ptr(q1), _ptr(k1), _ptr(q2),
                             _ptr(k2), _ptr(v), _ptr(lam), _ptr(norm_w), _ptr(out), int(splits),
                             _ptr(workspace), ws_bytes, _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


def fwd_kv_strided(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: bool = True,
                   norm_w=None, eps: float = 1e-5, lambda_init: float = 0.0, splits: int = 0,
                   workspace=None, out=None, status=None, stream=None, raw_status: bool = False):
    """`diffattn_fwd_kv_strided`: `fwd_kv` (bf16, d = 64) on [B, H, rows, width]-shaped
    views of any layout whose rows are contiguous (e.g. a [B, Nkv, H, d] cache seen
    through permute(0, 2, 1, 3)); `out` may be such a view too (default: contiguous)."""
    B, H, N, d = q1.shape
    n_kv = k1.shape[2]
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=q1.dtype, device=q1.device)
    ts = [q1, k1, q2, k2, v, out]
    shapes = [(B, H, N, d), (B, H, n_kv, d), (B, H, N, d), (B, H, n_kv, d),
              (B, H, n_kv, 2 * d), (B, H, N, 2 * d)]
    for t, shape in zip(ts, shapes):
        if tuple(t.shape) != shape or t.dtype != q1.dtype or not t.is_cuda:
            raise ValueError(f"expected a CUDA {q1.dtype} tensor of shape {shape}")
        if t.stride(-1) != 1:
            raise ValueError("rows must be contiguous (last stride 1)")
    _cuda_contig([lam, norm_w])
    arr = (Strides * 6)(*[Strides(t.stride(0), t.stride(1), t.stride(2)) for t in ts])
    desc = make_desc(B, H, N, d, _DTYPE_CODE.get(q1.dtype, -1), causal, headnorm, eps,
                     lambda_init, status)
    lib = load()
    if workspace is None:
        sp, nb = ctypes.c_int(0), ctypes.c_size_t(0)
        st = lib.diffattn_fwd_kv_plan(ctypes.byref(desc), int(n_kv), int(splits),
                                      ctypes.byref(sp), ctypes.byref(nb))
        if st != OK:
            if raw_status:
                return st
            _check(st)
        if nb.value:
            workspace = torch.empty(nb.value, dtype=torch.uint8, device=q1.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.diffattn_fwd_kv_strided(ctypes.byref(desc), int(n_kv), _ptr(q1), _ptr(k1),
                                     _ptr(q2), _ptr(k2), _ptr(v), _ptr(lam), _ptr(norm_w),
                                     _ptr(out), int(splits), _ptr(workspace), ws_bytes, arr,
                                     _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


def train_sizes(B, H, N, *, d: int = 64):
    """`diffattn_train_sizes`: (saved-activation bytes, backward workspace bytes)."""
    desc = make_desc(B, H, N, d, BF16, True, True, 1e-5, 0.0)
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().diffattn_train_sizes(ctypes.byref(desc), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def _check_qkv(q1, k1, q2, k2, v):
    if q1.dim() != 4:
        raise ValueError("q1 must be [B, H, N, d]")
    B, H, N, d = q1.shape
    for name, t, shape in (("k1", k1, (B, H, N, d)), ("q2", q2, (B, H, N, d)),
                           ("k2", k2, (B, H, N, d)), ("v", v, (B, H, N, 2 * d))):
        if tuple(t.shape) != shape or t.dtype != q1.dtype:
            raise ValueError(f"{name} must be {shape} {q1.dtype}")
    return B, H, N, d


def _cuda_contig(ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")


def fwd_train(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: bool = True, norm_w=None,
              eps: float = 1e-5, lambda_init: float = 0.0, out=None, saved=None, status=None,
              stream=None):
    """`diffattn_fwd_train`: the forward plus the activations the backward needs.

    Returns (out, saved); `saved` is a uint8 CUDA tensor of train_sizes()[0] bytes.
    """
    B, H, N, d = _check_qkv(q1, k1, q2, k2, v)
    saved_bytes, _ = train_sizes(B, H, N, d=d)
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=q1.dtype, device=q1.device)
    if saved is None:
        saved = torch.empty(saved_bytes, dtype=torch.uint8, device=q1.device)
    _cuda_contig([q1, k1, q2, k2, v, lam, norm_w, out, saved])
    desc = make_desc(B, H, N, d, _DTYPE_CODE.get(q1.dtype, -1), causal, headnorm, eps,
                     lambda_init, status)
    _check(load().diffattn_fwd_train(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2),
                                     _ptr(v), _ptr(lam), _ptr(norm_w), _ptr(out), _ptr(saved),
                                     saved.numel() * saved.element_size(),
                                     _stream_handle(stream)))
    return out, saved


def bwd(q1, k1, q2, k2, v, lam, saved, dy, *, causal: bool, headnorm: bool = True,
        norm_w=None, eps: float = 1e-5, lambda_init: float = 0.0, workspace=None, grads=None,
        status=None, stream=None, raw_status: bool = False):
    """`diffattn_bwd`: gradients of sum(out * dy) given fwd_train's `saved`.

    Returns dict dq1, dk1, dq2, dk2 (bf16 [B, H, N, d]), dv (bf16 [B, H, N, 2d]),
    dlam (fp32 [H]) and dw (fp32 [H, 2d], zeros without the norm).
    """
    B, H, N, d = _check_qkv(q1, k1, q2, k2, v)
    _, ws_bytes = train_sizes(B, H, N, d=d)
    dev = q1.device
    if grads is None:
        grads = {k: torch.empty((B, H, N, d), dtype=q1.dtype, device=dev)
                 for k in ("dq1", "dk1", "dq2", "dk2")}
        grads["dv"] = torch.empty((B, H, N, 2 * d), dtype=q1.dtype, device=dev)
        grads["dlam"] = torch.empty(H, dtype=torch.float32, device=dev)
        grads["dw"] = torch.zeros((H, 2 * d), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _cuda_contig([q1, k1, q2, k2, v, lam, norm_w, saved, dy, workspace, *grads.values()])
    desc = make_desc(B, H, N, d, _DTYPE_CODE.get(q1.dtype, -1), causal, headnorm, eps,
                     lambda_init, status)
    st = load().diffattn_bwd(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(v),
                             _ptr(lam), _ptr(norm_w), _ptr(saved), _ptr(dy), _ptr(grads["dq1"]),
                             _ptr(grads["dk1"]), _ptr(grads["dq2"]), _ptr(grads["dk2"]),
                             _ptr(grads["dv"]), _ptr(grads["dlam"]), _ptr(grads["dw"]),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return grads


def fwd_train_strided(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: int = 1,
                      norm_w=None, eps: float = 1e-5, lambda_init: float = 0.0, out=None,
                      saved=None, status=None, stream=None):
    """`diffattn_fwd_train_strided`: fwd_train on [B, H, N, d]-shaped views with
    contiguous rows (`out` may be such a view too; default contiguous).
    Returns (out, saved)."""
    B, H, N, d = q1.shape
    saved_bytes, _ = train_sizes(B, H, N, d=d)
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=q1.dtype, device=q1.device)
    if saved is None:
        saved = torch.empty(saved_bytes, dtype=torch.uint8, device=q1.device)
    ts = [q1, k1, q2, k2, v, out]
    arr = _view_strides(ts, [(B, H, N, d)] * 4 + [(B, H, N, 2 * d)] * 2, q1.dtype)
    _cuda_contig([lam, norm_w, saved])
    desc = make_desc(B, H, N, d, _DTYPE_CODE.get(q1.dtype, -1), causal, headnorm, eps,
                     lambda_init, status)
    _check(load().diffattn_fwd_train_strided(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2),
                                             _ptr(k2), _ptr(v), _ptr(lam), _ptr(norm_w),
                                             _ptr(out), _ptr(saved),
                                             saved.numel() * saved.element_size(), arr,
                                             _stream_handle(stream)))
    return out, saved


def bwd_strided(q1, k1, q2, k2, v, lam, saved, dy, *, causal: bool, headnorm: int = 1,
                norm_w=None, eps: float = 1e-5, lambda_init: float = 0.0, workspace=None,
                grads=None, status=None, stream=None, raw_status: bool = False):
    """`diffattn_bwd_strided`: bwd on [B, H, N, .]-shaped views with contiguous rows;
    `grads` (dq1, dk1, dq2, dk2, dv views, plus dlam and dw) defaults to contiguous
    tensors.  Returns the grads dict as bwd does."""
    B, H, N, d = q1.shape
    _, ws_bytes = train_sizes(B, H, N, d=d)
    dev = q1.device
    if grads is None:
        grads = {k: torch.empty((B, H, N, d), dtype=q1.dtype, device=dev)
                 for k in ("dq1", "dk1", "dq2", "dk2")}
        grads["dv"] = torch.empty((B, H, N, 2 * d), dtype=q1.dtype, device=dev)
        grads["dlam"] = torch.empty(H, dtype=torch.float32, device=dev)
        grads["dw"] = torch.zeros((H, 2 * d), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ts = [q1, k1, q2, k2, v, dy, grads["dq1"], grads["dk1"], grads["dq2"], grads["dk2"],
          grads["dv"]]
    w = 2 * d
    shapes = [(B, H, N, d)] * 4 + [(B, H, N, w)] * 2 + [(B, H, N, d)] * 4 + [(B, H, N, w)]
    arr = _view_strides(ts, shapes, q1.dtype)
    _cuda_contig([lam, norm_w, saved, workspace, grads["dlam"], grads["dw"]])
    desc = make_desc(B, H, N, d, _DTYPE_CODE.get(q1.dtype, -1), causal, headnorm, eps,
                     lambda_init, status)
    st = load().diffattn_bwd_strided(ctypes.byref(desc), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2),
                                     _ptr(v), _ptr(lam), _ptr(norm_w), _ptr(saved), _ptr(dy),
                                     _ptr(grads["dq1"]), _ptr(grads["dk1"]), _ptr(grads["dq2"]),
                                     _ptr(grads["dk2"]), _ptr(grads["dv"]), _ptr(grads["dlam"]),
                                     _ptr(grads["dw"]), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), arr,
                                     _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return grads


NOALLOC_SCRATCH_BYTES = 64 << 20


def fwd_kv_noalloc(q1, k1, q2, k2, v, lam, *, causal: bool, headnorm: bool = True,
                   norm_w=None, eps: float = 1e-5, lambda_init: float = 0.0, splits: int = 0,
                   out=None, status=None, stream=None, raw_status: bool = False):
    """`diffattn_fwd_kv_noalloc`: fwd_kv on the library's own 64 MiB scratch area.

    Same arguments and result as :func:`fwd_kv` without the workspace.  Calls
    that overlap in time race on the shared scratch; the first call on a device
    must not be inside a CUDA graph capture.
    """
    B, H, N, d = q1.shape
    n_kv = k1.shape[2]
    code, vdtype = _kv_dtypes(q1)
    if out is None:
        out = torch.empty((B, H, N, 2 * d), dtype=vdtype, device=q1.device)
    for t in [q1, k1, q2, k2, v, lam, out] + ([norm_w] if norm_w is not None else []):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if tuple(k2.shape) != tuple(k1.shape) or tuple(q2.shape) != tuple(q1.shape) or \
            tuple(v.shape) != (B, H, n_kv, 2 * d) or tuple(out.shape) != (B, H, N, 2 * d):
        raise ValueError("q1, q2 [B, H, Nq, d]; k1, k2 [B, H, Nkv, d]; v [B, H, Nkv, 2d]; "
                         "out [B, H, Nq, 2d]")
    desc = make_desc(B, H, N, d, code, causal, headnorm, eps, lambda_init, status)
    st = load().diffattn_fwd_kv_noalloc(ctypes.byref(desc), int(n_kv), _ptr(q1), _ptr(k1),
                                        _ptr(q2), _ptr(k2), _ptr(v), _ptr(lam), _ptr(norm_w),
                                        _ptr(out), int(splits), _stream_handle(stream))
    if raw_status:
        return st
    _check(st)
    return out


class PagedCache:
    """A paged key/value cache (`diffpaged_cache` of include/diffattn_paged.h).

    k1, k2: [pages, kv_heads, page_size, d], bf16 or both float8_e4m3fn; v: bf16 [pages,
    kv_heads, page_size, 2d]; CUDA tensors or views of any layout with contiguous rows
    (e.g. x.permute(0, 2, 1, 3) of [pages, page_size, kv_heads, d] storage).  page_table:
    int32 [B, max_pages]; kv_len: int32 [B], the lengths with the newest tokens counted;
    weights: float32 [pages, kv_heads, page_size] or None.  All on one device.

    The tensors are checked here, once; the calls then use their addresses, so they are
    changed in place (kv_len.add_(1), page_table[b, n] = page), not replaced.
    """

    def __init__(self, k1, k2, v, page_table, kv_len, weights=None):
        if k1.dim() != 4:
            raise ValueError("k1 must be [pages, kv_heads, page_size, d]")
        pages, heads, page, d = k1.shape
        if k1.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"unsupported key dtype {k1.dtype}")
        if page_table.dim() != 2 or kv_len.dim() != 1:
            raise ValueError("page_table must be [B, max_pages] and kv_len [B]")
        B, max_pages = page_table.shape
        for name, t, shape, dtype in (
                ("k1", k1, (pages, heads, page, d), k1.dtype),
                ("k2", k2, (pages, heads, page, d), k1.dtype),
                ("v", v, (pages, heads, page, 2 * d), torch.bfloat16),
                ("page_table", page_table, (B, max_pages), torch.int32),
                ("kv_len", kv_len, (B,), torch.int32),
                ("weights", weights, (pages, heads, page), torch.float32)):
            if t is None:
                continue
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise ValueError(f"{name} must be {shape} {dtype}")
            if name in ("k1", "k2", "v"):
                if d and t.stride(-1) != 1:
                    raise ValueError("rows must be contiguous (last stride 1)")
            elif not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        for t in (k1, k2, v, page_table, kv_len, weights):
            if t is not None and (not t.is_cuda or t.device != k1.device):
                raise ValueError("all tensors must be CUDA tensors of one device")
        self.k1, self.k2, self.v = k1, k2, v
        self.page_table, self.kv_len, self.weights = page_table, kv_len, weights
        self.B, self.kv_heads, self.d, self.page_size = B, heads, d, page
        self.device, self.dtype = k1.device, k1.dtype
        self.index = k1.get_device()
        self.code = E4M3_QK if k1.dtype == torch.float8_e4m3fn else BF16
        self._calls = {}
        self._struct = PagedCacheStruct(
            k1.data_ptr(), k2.data_ptr(), v.data_ptr(),
            0 if weights is None else weights.data_ptr(), page_table.data_ptr(),
            kv_len.data_ptr(), *(_strides4(t) for t in (k1, k2, v)), pages, heads, max_pages,
            page, 0)
        self._ref = ctypes.byref(self._struct)

    # What a call's shapes and numbers come to (its descriptor, the shapes of its other tensors, its
    # workspace) is worked out and checked once, and kept under them; with a status word, each time.
    # Keys hold plain numbers: a tensor would stand for whatever value it had the first time.

    def _keep(self, key, status, call):
        if status is None:
            if len(self._calls) >= 256:
                self._calls.clear()
            self._calls[key] = call
        return call

    def _new_append(self, shape, status):
        if len(shape) != 4 or shape[0] != self.B or shape[1] != self.kv_heads or \
                shape[3] != self.d:
            raise ValueError(f"k1 and k2 must be [{self.B}, {self.kv_heads}, N, {self.d}], "
                             f"v [{self.B}, {self.kv_heads}, N, {2 * self.d}]")
        desc = make_desc(self.B, self.kv_heads, shape[2], self.d, self.code, True, 0, 0.0, 0.0,
                         status)
        return self._keep(shape, status, (ctypes.byref(desc), (*shape[:3], 2 * self.d)))

    def _new_fwd(self, key, status):
        shape, causal, headnorm, eps, lambda_init, accumulate = key
        if len(shape) != 4 or shape[0] != self.B or shape[3] != self.d:
            raise ValueError(f"q1 and q2 must be [{self.B}, H, N, {self.d}]")
        H, N = shape[1], shape[2]
        ref = ctypes.byref(make_desc(self.B, H, N, self.d, self.code, causal, headnorm, eps,
                                     lambda_init, status))
        need = ctypes.c_size_t(0)
        st = load().diffpaged_fwd_plan(ref, self._ref, int(accumulate), ctypes.byref(need))
        if st != OK:
            return st, None
        return OK, self._keep(key, status, (ref, (self.B, H, N, 2 * self.d), H, need.value))

    def _new_evict(self, keep, status):
        ref = ctypes.byref(make_desc(self.B, self.kv_heads, 0, self.d, self.code, True, 0, 0.0,
                                     0.0, status))
        need = ctypes.c_size_t(0)
        st = load().diffpaged_evict_plan(ref, self._ref, keep, ctypes.byref(need))
        if st != OK:
            return st, None
        return OK, self._keep(keep, status, (ref, need.value))


def _strides4(t):
    """(outer, head, row) element strides of a 4-D tensor with contiguous rows.  An axis of one
    element is never stepped along: it gets the stride it would have in contiguous storage."""
    s, n = t.stride(), t.shape
    row = s[2] if n[2] > 1 else n[3]
    head = s[1] if n[1] > 1 else row * n[2]
    return Strides(s[0] if n[0] > 1 else head * n[1], head, row)


def _strides_or_null(a, b, c):
    """The strides argument of a paged call: NULL when all three tensors are contiguous."""
    if a.is_contiguous() and b.is_contiguous() and c.is_contiguous():
        return None
    if a.stride(3) != 1 or b.stride(3) != 1 or c.stride(3) != 1:
        raise ValueError("rows must be contiguous (last stride 1)")
    return (Strides * 3)(_strides4(a), _strides4(b), _strides4(c))


def _stream_on(cache, stream):
    """The handle of a call's stream; refuses one of another device than the cache's, and the
    current device being another (its context would run the kernels)."""
    index = torch.cuda.current_device()
    if cache.index != index:
        raise ValueError(f"the cache is on cuda:{cache.index}, the current device is cuda:{index}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device != cache.device:
        raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
    return stream.cuda_stream


def _new_on(stream, shape, dtype, dev):
    """A torch buffer of `stream`'s memory (None: the current one's), reused only in its order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(workspace, need, cache, stream):
    """(pointer, bytes, buffer to keep) of a call's workspace: the caller's, or one of its own."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _new_on(stream, need, torch.uint8, cache.device)
    elif workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return workspace.data_ptr(), workspace.nbytes, workspace


def paged_append(cache, k1, k2, v, *, status=None, stream=None, raw_status: bool = False):
    """`diffpaged_append`: the N newest tokens' rows into the cache, at positions kv_len - N + i
    (negative ones are padding).

    k1, k2: bf16 [B, kv_heads, N, d] (rounded to e4m3 where the cache holds that); v: bf16
    [B, kv_heads, N, 2d]; views of any layout with contiguous rows.
    """
    shape = k1.shape
    call = cache._calls.get(shape) if status is None else None
    ref, v_shape = call or cache._new_append(shape, status)
    if k2.shape != shape or v.shape != v_shape:
        raise ValueError(f"k2 must be {tuple(shape)}, as k1, and v {v_shape}")
    dtype, index = torch.bfloat16, cache.index
    if k1.dtype != dtype or k2.dtype != dtype or v.dtype != dtype:
        raise ValueError("k1, k2 and v must be bfloat16")
    if k1.get_device() != index or k2.get_device() != index or v.get_device() != index:
        raise ValueError("all tensors must be on the cache's device")
    strides = _strides_or_null(k1, k2, v)
    handle = _stream_on(cache, stream)
    st = (_lib or load()).diffpaged_append(ref, cache._ref, k1.data_ptr(), k2.data_ptr(),
                                           v.data_ptr(), strides, handle)
    if raw_status:
        return st
    _check(st)


def paged_fwd_plan(cache, H: int, N: int = 1, *, accumulate: bool = False,
                   raw_status: bool = False):
    """`diffpaged_fwd_plan`: workspace bytes of paged_fwd with H query heads and N new tokens."""
    desc = make_desc(cache.B, H, N, cache.d, cache.code, True, 1, 1e-5, 0.0)
    n = ctypes.c_size_t(0)
    st = load().diffpaged_fwd_plan(ctypes.byref(desc), cache._ref, int(accumulate),
                                   ctypes.byref(n))
    if raw_status:
        return st, n.value
    _check(st)
    return n.value


def paged_fwd(cache, q1, q2, lam, *, causal: bool = True, headnorm: int = 1, norm_w=None,
              eps: float = 1e-5, lambda_init: float = 0.0, accumulate: bool = False,
              workspace=None, out=None, status=None, stream=None, raw_status: bool = False):
    """`diffpaged_fwd`: the N newest tokens of every sequence against the paged cache.

    q1, q2: [B, H, N, d] of the cache's key dtype, H a multiple of its kv_heads, N <= 16;
    lam: float32 [H]; norm_w: float32 [H, 2d] or None.  Views of any layout with contiguous
    rows (`out` too).  accumulate adds each key's sum |map1 - lam map2| to cache.weights.
    workspace: a CUDA tensor of at least paged_fwd_plan bytes (a torch buffer when None).
    Returns bf16 out [B, H, N, 2d] (of `stream`'s memory when allocated here).
    """
    key = (q1.shape, bool(causal), int(headnorm), float(eps), float(lambda_init), bool(accumulate))
    call = cache._calls.get(key) if status is None else None
    if call is None:
        st, call = cache._new_fwd(key, status)
        if st != OK:
            if raw_status:
                return st
            _check(st)
    ref, out_shape, H, need = call
    index, dtype, f32 = cache.index, cache.dtype, torch.float32
    if q2.shape != q1.shape:
        raise ValueError(f"q2 must be {tuple(q1.shape)}, as q1")
    if q1.dtype != dtype or q2.dtype != dtype:
        raise ValueError(f"q1 and q2 must be {dtype}, as the cache's keys")
    if q1.get_device() != index or q2.get_device() != index or lam.get_device() != index:
        raise ValueError("all tensors must be on the cache's device")
    if lam.dtype != f32 or lam.numel() != H or not lam.is_contiguous():
        raise ValueError("lam must be contiguous float32 [H]")
    if norm_w is not None and (norm_w.dtype != f32 or norm_w.numel() != H * out_shape[3] or
                               not norm_w.is_contiguous() or norm_w.get_device() != index):
        raise ValueError("norm_w must be contiguous float32 [H, 2d] on the cache's device")
    handle = _stream_on(cache, stream)
    if out is None:
        out = _new_on(stream, out_shape, torch.bfloat16, cache.device)
    elif out.shape != out_shape or out.dtype != torch.bfloat16 or out.get_device() != index:
        raise ValueError("out must be bfloat16 [B, H, N, 2d] on the cache's device")
    strides = _strides_or_null(q1, q2, out)
    ws, ws_bytes, _hold = _workspace(workspace, need, cache, stream)
    st = (_lib or load()).diffpaged_fwd(
        ref, cache._ref, q1.data_ptr(), q2.data_ptr(), lam.data_ptr(),
        None if norm_w is None else norm_w.data_ptr(), out.data_ptr(), strides, int(accumulate),
        ws, ws_bytes, handle)
    if raw_status:
        return st
    _check(st)
    return out


def paged_evict_plan(cache, *, keep: int, raw_status: bool = False):
    """`diffpaged_evict_plan`: workspace bytes of paged_evict."""
    desc = make_desc(cache.B, cache.kv_heads, 0, cache.d, cache.code, True, 0, 0.0, 0.0)
    n = ctypes.c_size_t(0)
    st = load().diffpaged_evict_plan(ctypes.byref(desc), cache._ref, int(keep), ctypes.byref(n))
    if raw_status:
        return st, n.value
    _check(st)
    return n.value


def paged_evict(cache, *, keep: int, recent: int = 0, workspace=None, status=None, stream=None,
                raw_status: bool = False):
    """`diffpaged_evict`: cut every sequence longer than `keep` to its last `recent` keys and
    the keep - recent of the largest weights, in place; updates cache.kv_len."""
    handle, keep = _stream_on(cache, stream), int(keep)
    call = cache._calls.get(keep) if status is None else None
    if call is None:
        st, call = cache._new_evict(keep, status)
        if st != OK:
            if raw_status:
                return st
            _check(st)
    ref, need = call
    ws, ws_bytes, _hold = _workspace(workspace, need, cache, stream)
    st = (_lib or load()).diffpaged_evict(ref, cache._ref, keep, int(recent), ws, ws_bytes,
                                          handle)
    if raw_status:
        return st
    _check(st)


def headnorm(x, *, H: int, norm_w=None, eps: float = 1e-5, lambda_init: float = 0.0,
             out_dtype=torch.bfloat16, out=None, stream=None, mode: int = 1):
    """Per-head normalisation through `diffattn_headnorm` (mode 1: RMS; mode 2:
    mean-subtracting group form).

    x: float32 [B, H, N, 2d] CUDA; returns [B, H, N, 2d] in out_dtype.
    """
    if x.dim() != 4 or x.dtype != torch.float32:
        raise ValueError("x must be float32 [B, H, N, 2d]")
    B, Hx, N, dv = x.shape
    if Hx != H or dv % 2:
        raise ValueError("x must be [B, H, N, 2d]")
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    for t in [x, out] + ([norm_w] if norm_w is not None else []):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
    desc = make_desc(B, H, N, dv // 2, _DTYPE_CODE[out.dtype], False, mode, eps, lambda_init)
    _check(load().diffattn_headnorm(ctypes.byref(desc), _ptr(x), _ptr(norm_w), _ptr(out),
                                    _stream_handle(stream)))
    return out


def selftest_wait(timeout_ns: int = 50_000_000, stream=None):
    """`diffattn_selftest_wait`: returns (status code, first wait us, second wait us)."""
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    _check(load().diffattn_selftest_wait(_ptr(st), int(timeout_ns), _stream_handle(stream)))
    torch.cuda.synchronize()
    code, w0, w1 = (int(x) for x in st.cpu())
    return code, w0, w1

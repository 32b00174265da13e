"""Python binding of libdsa.so, the GB300 (sm_103a) DSA hot path.

Argument marshalling only: each function checks dtypes/shapes, passes raw
device pointers and the current CUDA stream to the C entry point of the same
name (declared in include/dsa.h) and raises ``DsaError`` on a non-zero status.
Every step of the computation runs in the library's CUDA kernels; there is no
host or PyTorch fallback, and importing this package fails loudly when the
library has not been built.

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import os
import threading
import warnings

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK = 0
DSA_DEV_TIMEOUT = 0x1
DSA_DEV_BAD_POSITION = 0x2
DSA_DEV_BAD_PAGE = 0x4

_lib = None
_fast = None  # the native call path (csrc/fastcall.cpp), set before _lib; None where it cannot be used
_load_lock = threading.Lock()


class DsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"dsa error {code}: {msg}")
        self.code = code


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libdsa.so (built by ``sparse_attention_02_gb300.build``)."""
    global _lib, _fast
    if path is not None:
        return _open(path)
    if _lib is None:
        with _load_lock:  # a thread that comes meanwhile waits, and finds both or neither
            if _lib is None:
                lib = _open(LIB_PATH)
                _fast = _load_fastcall(LIB_PATH)
                _lib = lib
    return _lib


def _open(p: str) -> ctypes.CDLL:
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m sparse_attention_02_gb300.build` "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(p)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.dsa_last_error.restype = ctypes.c_char_p
    lib.dsa_version.restype = i32
    lib.dsa_get_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.dsa_quantize_fp8.argtypes = [P, i64, i64, i32, P, P, P]
    lib.dsa_indexer_logits.argtypes = [P, P, P, i32, i32, i32, P, P, i32, P, i32, i32, i32, P, P, i64, P]
    lib.dsa_topk.argtypes = [P, i64, i32, P, i32, P, P]
    lib.dsa_sparse_mla_prefill.argtypes = [P, P, i32, P, i32, i32, i32, f32, P, P, P]
    lib.dsa_sparse_mla_decode_paged.argtypes = [P, P, i32, i32, P, i32, P, P, i32, i32, i32, f32, P, P, P, sz, P]
    lib.dsa_sparse_mla_decode_paged_noalloc.argtypes = [P, P, i32, i32, P, i32, P, P, i32, i32, i32, f32, P, P, P]
    lib.dsa_prefill_host.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, f32, P, P, i32, P, sz, P]
    lib.dsa_prefill_host_workspace_size.restype = sz
    lib.dsa_prefill_host_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.dsa_prefill_host_trace.argtypes = [i32]
    lib.dsa_prefill_host_trace_read.argtypes = [P, P, P, i32, ctypes.POINTER(i32)]
    lib.dsa_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P]
    lib.dsa_selftest_wait_timeout.restype = i32
    lib.dsa_sparse_mla_decode_workspace_size.restype = sz
    lib.dsa_sparse_mla_decode_workspace_size.argtypes = [i32, i32, i32]
    lib.dsa_indexer_topk.argtypes = [P, P, P, i32, i32, i32, P, P, i32, P, i32, P, P, sz, P]
    lib.dsa_indexer_warmup.argtypes = [P, P, i32, f32, P, P, P, i32, i32, P, P, P, i32, i32, P, P, P, P, P, sz, P]
    lib.dsa_indexer_warmup_workspace_size.restype = sz
    lib.dsa_indexer_warmup_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.dsa_indexer_topk_workspace_size.restype = sz
    lib.dsa_indexer_topk_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.dsa_rmsnorm.argtypes = [P, i64, P, i64, P, i64, i32, i32, i32, f32, P, i64, P, i64, P, P, i32, i32, P]
    lib.dsa_rmsnorm_backward.argtypes = [P, P, P, P, i64, i32, i32, i32, f32, P, P, P, sz, P]
    lib.dsa_rmsnorm_backward_workspace_size.restype = sz
    lib.dsa_rmsnorm_backward_workspace_size.argtypes = [i64, i32]
    lib.dsa_cache_append.argtypes = [P, P, i32, P, i32, i32, i32, i32, P, P, i64, P, i32, f32, P, P, i64, i32, i32, P, P, P]
    lib.dsa_rope_queries.argtypes = [P, P, i32, P, i64, i64, i32, P, P, i32, i32, i32, P, P, P]
    lib.dsa_index_rope_backward.argtypes = [P, P, P, i32, i32, P, i32, P]
    lib.dsa_mla_decode_paged.argtypes = [P, P, i32, i32, P, i32, P, i32, i32, f32, P, P, P, sz, P]
    lib.dsa_mla_decode_workspace_size.restype = sz
    lib.dsa_mla_decode_workspace_size.argtypes = [i32, i32]
    for name in ("dsa_rmsnorm", "dsa_rmsnorm_backward", "dsa_cache_append", "dsa_rope_queries",
                 "dsa_index_rope_backward", "dsa_mla_decode_paged", "dsa_quantize_fp8", "dsa_indexer_logits", "dsa_topk", "dsa_indexer_topk", "dsa_indexer_warmup",
                 "dsa_sparse_mla_prefill",
                 "dsa_sparse_mla_decode_paged",
                 "dsa_sparse_mla_decode_paged_noalloc", "dsa_prefill_host", "dsa_prefill_host_trace",
                 "dsa_prefill_host_trace_read", "dsa_get_device_status"):
        getattr(lib, name).restype = i32
    return lib


def _load_fastcall(path: str):
    """The native call path, or None where it was not built for this interpreter and PyTorch (it reads tensors by
    PyTorch's C++ classes) or PyTorch lacks what it calls: the Python form of every call makes the same library calls, at 6
    to 12 us more host time each (one-row norm 6.1 and 12.5 us, dense decode of one row 6.2 and 17.6)."""
    from .build import fastcall_abi, fastcall_built_for

    try:
        if fastcall_built_for() != fastcall_abi():  # before its import: another PyTorch's would read the wrong fields
            raise ImportError("_fastcall.so is not there, or was built for another Python or PyTorch")
        from . import _fastcall

        _fastcall.init(path, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream,
                       torch._C._cuda_cudaCachingAllocator_raw_alloc, torch._C._cuda_cudaCachingAllocator_raw_delete)
    except (ImportError, AttributeError, OSError) as e:  # OSError: a PyTorch without the file that names its version
        warnings.warn(f"the native call path is not used ({e}): calls on few tokens take the host longer; "
                      "`python -m sparse_attention_02_gb300.build` builds it", RuntimeWarning, stacklevel=3)
        return None
    return _fastcall


def _check(rc: int):
    if rc != DSA_OK:
        raise DsaError(rc, load_library().dsa_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _same_device(t: torch.Tensor, name: str):
    # the library runs on the current device (cudaGetDevice); a tensor elsewhere would
    # hand it another GPU's pointer
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur}")


def _need(t: torch.Tensor, dtype, name: str, dim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _same_device(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name}: expected {dim} dims, got {t.dim()}")


def _need_rows(t: torch.Tensor, dtype, name: str):
    """A 2-D tensor whose rows may be strided (leading dimension >= width)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or t.dim() != 2:
        raise TypeError(f"{name}: expected a 2-D CUDA {dtype} tensor")
    _same_device(t, name)
    if t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows must be contiguous with a leading dimension >= width")


DSA_SCALE_AMAX = 0
DSA_SCALE_POW2 = 1


def dsa_quantize_fp8(x, codes, scale, mode: int = DSA_SCALE_AMAX, stream=None):
    """Per-row FP8 quantisation: x fp32 [rows, ...] -> codes uint8 (E4M3, same shape), scale fp32 [rows].

    mode DSA_SCALE_AMAX: scale = amax / 448; DSA_SCALE_POW2: the smallest power of two >= that.
    """
    _need(x, torch.float32, "x")
    _need(codes, torch.uint8, "codes")
    _need(scale, torch.float32, "scale", 1)
    if x.dim() < 1 or tuple(codes.shape) != tuple(x.shape) or scale.shape[0] != x.shape[0]:
        raise ValueError("codes must match x's shape and scale must have one entry per row")
    rows = x.shape[0]
    cols = x.numel() // rows if rows > 0 else 1
    _check(load_library().dsa_quantize_fp8(_ptr(x), rows, cols, int(mode), _ptr(codes), _ptr(scale),
                                           _stream(stream)))
    return codes, scale


def dsa_indexer_logits(q8, q_scale, w, k8, k_scale, q_pos, logits, block_table=None, stream=None):
    """Lightning-indexer scores into ``logits`` [T, ld] (fp32).

    q8 uint8 [T, H_I, d_I] (E4M3 codes), q_scale fp32 [T], w fp32 [T, H_I], q_pos int32 [T].
    Contiguous keys: k8 uint8 [S, d_I], k_scale fp32 [S].  Paged keys: k8 uint8
    [num_pages, page_size, d_I], k_scale fp32 [num_pages, page_size] and
    block_table int32 [T, max_pages].  ``logits`` rows may be strided
    (leading dimension = logits.stride(0)).
    """
    _need(q8, torch.uint8, "q8", 3)
    T, HI, dI = q8.shape
    _need(q_scale, torch.float32, "q_scale", 1)
    _need(w, torch.float32, "w", 2)
    _need(q_pos, torch.int32, "q_pos", 1)
    _need_rows(logits, torch.float32, "logits")
    _need(k8, torch.uint8, "k8")
    _need(k_scale, torch.float32, "k_scale")
    if q_scale.shape[0] != T or tuple(w.shape) != (T, HI) or q_pos.shape[0] != T or logits.shape[0] != T:
        raise ValueError("inconsistent query shapes")
    if block_table is None:
        if k8.dim() != 2 or k8.shape[1] != dI or k_scale.shape != (k8.shape[0],):
            raise ValueError("k8 must be [S, d_I] and k_scale [S]")
        S, mp, npg, ps = k8.shape[0], 0, 0, 0
    else:
        _need(block_table, torch.int32, "block_table", 2)
        if k8.dim() != 3 or k8.shape[2] != dI or tuple(k_scale.shape) != tuple(k8.shape[:2]):
            raise ValueError("paged: k8 must be [P, page, d_I] and k_scale [P, page]")
        if block_table.shape[0] != T:
            raise ValueError("block_table must have one row per query")
        S, mp, npg, ps = 0, block_table.shape[1], k8.shape[0], k8.shape[1]
    lib = load_library()
    _check(lib.dsa_indexer_logits(_ptr(q8), _ptr(q_scale), _ptr(w), T, HI, dI, _ptr(k8), _ptr(k_scale), S,
                                  _ptr(block_table), mp, npg, ps, _ptr(q_pos), _ptr(logits), logits.stride(0),
                                  _stream(stream)))
    return logits


DSA_BF16 = 0
DSA_FP32 = 1
_DTYPE = {torch.bfloat16: DSA_BF16, torch.float32: DSA_FP32}


def _device() -> int:
    try:
        return torch._C._cuda_getDevice()  # torch.cuda.current_device() without its initialisation check
    except (AttributeError, RuntimeError):
        return torch.cuda.current_device()


def _raw_stream(stream, cur: int) -> int:
    """The CUDA stream handle of ``stream``, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    try:
        return torch._C._cuda_getCurrentRawStream(cur)
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _native(name: str, *args) -> bool:
    """Makes the call natively where its arguments are plainly right; False leaves it, and what is wrong with it, to
    the Python form."""
    if _lib is None:
        load_library()
    if _fast is None:
        return False
    rc = getattr(_fast, name)(*args)
    if rc is NotImplemented:
        return False
    _check(rc)
    return True


def _refuse(t, cur: int, name: str, dtype, shape, rows: bool = False):
    """The error for an argument that is not what its call needs."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != cur:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if rows:
        raise ValueError(f"{name}: rows must be contiguous with a leading dimension >= width")
    raise ValueError(f"{name} must be contiguous")


def _address(t, name: str) -> int:
    """Address of a tensor's first element; fake tensors have none, which the library would take for no tensor."""
    p = t.data_ptr()
    if not p and t.numel():
        raise ValueError(f"{name} has no memory behind it")
    return p


# The checks below are one expression each: a call on a few tokens costs the host more than the GPU.
def _at(t, cur: int, name: str, dtype, shape) -> int:
    """Address of a contiguous CUDA tensor of the current device ``cur``."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == cur and t.shape == shape and t.is_contiguous():
        return _address(t, name)
    _refuse(t, cur, name, dtype, shape)


def _at_rows(t, cur: int, name: str, dtype, shape):
    """(address, distance of the rows) of a 2-D CUDA tensor whose rows may be apart."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == cur and t.shape == shape:
        if t.is_contiguous():
            return _address(t, name), shape[1]
        ld = t.stride(0) if shape[0] > 1 else shape[1]  # a single row's stride says nothing
        if (shape[1] == 1 or t.stride(1) == 1) and ld >= shape[1]:
            return _address(t, name), ld
    _refuse(t, cur, name, dtype, shape, True)


def _dtype_of(t, name: str):
    """bf16 or fp32."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name}: expected {_TYPES}, got {t.dtype}")
    return t.dtype


def _workspace(workspace, need: int, cur: int, stream):
    """(address, bytes, tensor to keep until the launch) of a call's workspace: the caller's, or one from
    PyTorch's allocator, taken on the stream that the call runs on."""
    if workspace is None:
        if not need:
            return None, 0, None
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=cur)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=cur)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != cur or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{cur}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


_TYPES = (torch.bfloat16, torch.float32)


def dsa_rmsnorm(x, weight, eps: float, out=None, residual=None, residual_out=None, codes=None, scale=None,
                block: int = 0, scale_mode: int = DSA_SCALE_AMAX, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, over the rows of x [rows, cols] (bf16 or fp32).

    residual_out gets h, out gets y (both of x's type); codes uint8 [rows, cols] and scale fp32 [rows] or
    [rows, n] get y as E4M3 codes with one scale per row (block = 0) or per 128 columns (block = 128,
    n = ceil(cols / 128)).  weight [cols] is bf16 or fp32.  Rows of x, residual, residual_out and out may be
    strided.  Returns (residual_out, out, codes, scale) as given."""
    if _native("rmsnorm", x, weight, eps, out, residual, residual_out, codes, scale, block, scale_mode, stream):
        return residual_out, out, codes, scale
    t = _dtype_of(x, "x")
    if x.dim() != 2:
        raise TypeError("x must be 2-D")
    cur, shape, f32 = _device(), x.shape, torch.float32
    rows, cols = shape
    wt = _dtype_of(weight, "weight")
    a_x, ldx = _at_rows(x, cur, "x", t, shape)
    a_r = a_h = a_o = a_c = a_s = None
    ldr = ldh = ldo = 0
    if residual is not None:
        a_r, ldr = _at_rows(residual, cur, "residual", t, shape)
    if residual_out is not None:
        a_h, ldh = _at_rows(residual_out, cur, "residual_out", t, shape)
    if out is not None:
        a_o, ldo = _at_rows(out, cur, "out", t, shape)
    if codes is not None:
        a_c = _at(codes, cur, "codes", torch.uint8, shape)
    if scale is not None:
        n = -(-cols // block) if block > 0 else 1
        a_s = _at(scale, cur, "scale", f32, (rows,) if n == 1 and isinstance(scale, torch.Tensor) and scale.dim() == 1 else (rows, n))
    _check((_lib or load_library()).dsa_rmsnorm(
        a_x, ldx, a_r, ldr, _at(weight, cur, "weight", wt, (cols,)), rows, cols, _DTYPE[t], _DTYPE[wt], float(eps), a_h, ldh, a_o, ldo,
        a_c, a_s, block, scale_mode, _raw_stream(stream, cur)))
    return residual_out, out, codes, scale


def dsa_rmsnorm_backward_workspace_size(rows: int, cols: int) -> int:
    return int(load_library().dsa_rmsnorm_backward_workspace_size(rows, cols))


def dsa_rmsnorm_backward(dy, h, weight, eps: float, dx, dweight, dres=None, workspace=None, stream=None):
    """Gradients of dsa_rmsnorm: dy, h, dres (or None) and dx [rows, cols] bf16 or fp32, h the saved residual_out
    (x without a residual); dx is the gradient of x and of the residual; dweight fp32 [cols].  ``workspace``: a
    CUDA tensor of at least dsa_rmsnorm_backward_workspace_size(rows, cols) bytes; taken from PyTorch when None."""
    if _native("rmsnorm_backward", dy, h, weight, eps, dx, dweight, dres, workspace, stream):
        return dx, dweight
    t = _dtype_of(h, "h")
    if h.dim() != 2:
        raise TypeError("h must be 2-D")
    cur, shape, wt = _device(), h.shape, _dtype_of(weight, "weight")
    rows, cols = shape
    lib = _lib or load_library()
    a_dy, a_h, a_w = _at(dy, cur, "dy", t, shape), _at(h, cur, "h", t, shape), _at(weight, cur, "weight", wt, (cols,))
    a_e = None if dres is None else _at(dres, cur, "dres", t, shape)
    a_dx, a_dw = _at(dx, cur, "dx", t, shape), _at(dweight, cur, "dweight", torch.float32, (cols,))
    need = 0 if workspace is not None else lib.dsa_rmsnorm_backward_workspace_size(rows, cols)
    ws, ws_bytes, keep = _workspace(workspace, need, cur, stream)
    _check(lib.dsa_rmsnorm_backward(a_dy, a_h, a_w, a_e, rows, cols, _DTYPE[t], _DTYPE[wt], float(eps), a_dx, a_dw, ws, ws_bytes,
                                    _raw_stream(stream, cur)))
    return dx, dweight


def dsa_cache_append(pos, block_table, inv_freq, kv=None, kv_pool=None, kI=None, k8_pool=None, ks_pool=None, seq=None,
                     kv_weight=None, eps: float = 1e-6, scale_mode: int = DSA_SCALE_AMAX, stream=None):
    """Writes T tokens into the paged caches, rotating them on the way.

    pos int32 [T] (negative: padding, nothing written); block_table int32 [num_seqs, max_pages]; seq int32 [T] names
    each token's block-table row (None: token t has row t); inv_freq fp64 [32] radians per position.  Latent cache:
    kv bf16 [T, 576] (rows may be strided) into kv_pool bf16 [P, page, 576], columns [0, 512) RMS-normed with
    kv_weight [512] (bf16 or fp32) when given, columns [512, 576) rotated in pairs (2i, 2i + 1).  Index cache: kI
    bf16 or fp32 [T, 128] (rows may be strided), pairs (i, i + 32) of its first 64 columns rotated, into k8_pool
    uint8 [P, page, 128] (E4M3 codes) and ks_pool fp32 [P, page].  Either cache may be left out."""
    if _native("cache_append", pos, block_table, inv_freq, kv, kv_pool, kI, k8_pool, ks_pool, seq, kv_weight, eps, scale_mode,
               stream):
        return
    if kv is None and kI is None:
        raise ValueError("kv or kI is needed")
    if not isinstance(pos, torch.Tensor) or pos.dim() != 1 or not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise TypeError("pos must be a 1-D and block_table a 2-D torch.Tensor")
    pool, name = (kv_pool, "kv_pool") if kv is not None else (k8_pool, "k8_pool")
    if not isinstance(pool, torch.Tensor) or pool.dim() != 3:
        raise TypeError(f"{name} must be a 3-D torch.Tensor")
    cur, T, i32, bf16 = _device(), pos.shape[0], torch.int32, torch.bfloat16
    P, ps, _ = pool.shape
    table = block_table.shape
    a_kv = a_pool = a_w = a_k = a_k8 = a_ks = None
    ld_kv = ld_kI = w = k = 0
    if kv is not None:
        a_kv, ld_kv = _at_rows(kv, cur, "kv", bf16, (T, 576))
        a_pool = _at(kv_pool, cur, "kv_pool", bf16, (P, ps, 576))
        if kv_weight is not None:
            w = _dtype_of(kv_weight, "kv_weight")
            a_w, w = _at(kv_weight, cur, "kv_weight", w, (512,)), _DTYPE[w]
    if kI is not None:
        k = _dtype_of(kI, "kI")
        a_k, ld_kI = _at_rows(kI, cur, "kI", k, (T, 128))
        k = _DTYPE[k]
        a_k8, a_ks = _at(k8_pool, cur, "k8_pool", torch.uint8, (P, ps, 128)), _at(ks_pool, cur, "ks_pool", torch.float32, (P, ps))
    _check((_lib or load_library()).dsa_cache_append(
        _at(pos, cur, "pos", i32, (T,)), None if seq is None else _at(seq, cur, "seq", i32, (T,)), T,
        _at(block_table, cur, "block_table", i32, table), table[0], table[1], P, ps,
        _at(inv_freq, cur, "inv_freq", torch.float64, (32,)), a_kv, ld_kv, a_w, w, float(eps), a_pool, a_k, ld_kI, k, scale_mode, a_k8,
        a_ks, _raw_stream(stream, cur)))


def dsa_rope_queries(pos, inv_freq, q_rope=None, q=None, qI=None, q8=None, q_scale=None,
                     scale_mode: int = DSA_SCALE_AMAX, stream=None):
    """Rotates the queries of T tokens: q_rope bf16 [T, H, 64] (any strides over tokens and heads) into columns
    [512, 576) of q bf16 [T, H, 576]; the index queries qI bf16 or fp32 [T, H_I, 128] into q8 uint8 (E4M3 codes) and
    q_scale fp32 [T].  pos int32 [T] (negative: padding, outputs left alone), inv_freq fp64 [32].  Either part may be
    left out; q_rope may be q[:, :, 512:]."""
    if _native("rope_queries", pos, inv_freq, q_rope, q, qI, q8, q_scale, scale_mode, stream):
        return
    if not isinstance(pos, torch.Tensor) or pos.dim() != 1:
        raise TypeError("pos must be a 1-D torch.Tensor")
    if q_rope is None and qI is None:
        raise ValueError("q_rope or qI is needed")
    cur, T, bf16 = _device(), pos.shape[0], torch.bfloat16
    a_r = a_q = a_i = a_8 = a_s = None
    st_t = st_h = H = HI = i_type = 0
    if q_rope is not None:
        if not isinstance(q_rope, torch.Tensor) or q_rope.dim() != 3:
            raise TypeError("q_rope must be a 3-D torch.Tensor")
        H = q_rope.shape[1]
        st_t, st_h, st_d = q_rope.stride()
        if q_rope.dtype is not bf16 or q_rope.get_device() != cur or q_rope.shape != (T, H, 64) or st_d != 1:
            _refuse(q_rope, cur, "q_rope", bf16, (T, H, 64), True)
        # a single token's or head's stride says nothing
        a_r, st_t, st_h = _address(q_rope, "q_rope"), st_t if T > 1 else 0, st_h if H > 1 else 0
        a_q = _at(q, cur, "q", bf16, (T, H, 576))
    if qI is not None:
        i_type = _dtype_of(qI, "qI")
        if qI.dim() != 3:
            raise TypeError("qI must be 3-D")
        HI = qI.shape[1]
        shape = (T, HI, 128)
        a_i, i_type = _at(qI, cur, "qI", i_type, shape), _DTYPE[i_type]
        a_8, a_s = _at(q8, cur, "q8", torch.uint8, shape), _at(q_scale, cur, "q_scale", torch.float32, (T,))
    _check((_lib or load_library()).dsa_rope_queries(
        _at(pos, cur, "pos", torch.int32, (T,)), _at(inv_freq, cur, "inv_freq", torch.float64, (32,)), T, a_r, st_t, st_h, H, a_q,
        a_i, HI, i_type, scale_mode, a_8, a_s, _raw_stream(stream, cur)))


def dsa_index_rope_backward(g, pos, inv_freq, dx, stream=None):
    """Gradient of the index rotation: g fp32 [T, H_I, 128] (or [T, 128], keys), the gradient of the rotated vectors
    (dsa_indexer_warmup's dq or dk), turned back by the tokens' angles into dx (bf16 or fp32, g's shape)."""
    if _native("index_rope_backward", g, pos, inv_freq, dx, stream):
        return dx
    if not isinstance(g, torch.Tensor) or g.dim() not in (2, 3):
        raise TypeError("g must be a 2-D or 3-D torch.Tensor")
    shape = g.shape
    if shape[-1] != 128:
        raise ValueError("g must be [T, H_I, 128] or [T, 128]")
    cur, T, HI, t = _device(), shape[0], shape[1] if len(shape) == 3 else 1, _dtype_of(dx, "dx")
    _check((_lib or load_library()).dsa_index_rope_backward(
        _at(g, cur, "g", torch.float32, shape), _at(pos, cur, "pos", torch.int32, (T,)),
        _at(inv_freq, cur, "inv_freq", torch.float64, (32,)), T, HI, _at(dx, cur, "dx", t, shape), _DTYPE[t],
        _raw_stream(stream, cur)))
    return dx


def dsa_topk(logits, valid_len, k: int, idx, stream=None):
    """Top-k indices (ascending, -1 padded) of each row of ``logits`` [T, >= max valid_len]
    (rows may be strided) into ``idx`` [T, k]."""
    _need_rows(logits, torch.float32, "logits")
    _need(valid_len, torch.int32, "valid_len", 1)
    _need(idx, torch.int32, "idx", 2)
    T = logits.shape[0]
    if valid_len.shape[0] != T or tuple(idx.shape) != (T, k):
        raise ValueError("inconsistent shapes")
    _check(load_library().dsa_topk(_ptr(logits), logits.stride(0), T, _ptr(valid_len), k, _ptr(idx),
                                   _stream(stream)))
    return idx


def dsa_indexer_topk_workspace_size(T: int, S: int, H_I: int, d_I: int, k: int) -> int:
    return int(load_library().dsa_indexer_topk_workspace_size(T, S, H_I, d_I, k))


def dsa_indexer_topk(q8, q_scale, w, k8, k_scale, q_pos, k: int, idx, workspace=None, stream=None):
    """Fused indexer -> top-k: the top-k key positions of each query row into ``idx`` [T, k]
    (ascending, -1 padded) without writing the index scores.  Inputs as for
    dsa_indexer_logits with contiguous keys.  ``workspace``: a uint8 CUDA tensor of at least
    dsa_indexer_topk_workspace_size(T, S, H_I, d_I, k) bytes; taken from PyTorch's
    allocator when None."""
    _need(q8, torch.uint8, "q8", 3)
    T, HI, dI = q8.shape
    _need(q_scale, torch.float32, "q_scale", 1)
    _need(w, torch.float32, "w", 2)
    _need(q_pos, torch.int32, "q_pos", 1)
    _need(k8, torch.uint8, "k8", 2)
    _need(k_scale, torch.float32, "k_scale", 1)
    _need(idx, torch.int32, "idx", 2)
    S = k8.shape[0]
    if q_scale.shape[0] != T or tuple(w.shape) != (T, HI) or q_pos.shape[0] != T or tuple(idx.shape) != (T, k) \
            or k8.shape[1] != dI or k_scale.shape[0] != S:
        raise ValueError("inconsistent shapes")
    if workspace is None:
        need = dsa_indexer_topk_workspace_size(T, S, HI, dI, k)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q8.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(workspace, "workspace")
    _check(load_library().dsa_indexer_topk(_ptr(q8), _ptr(q_scale), _ptr(w), T, HI, dI, _ptr(k8), _ptr(k_scale), S,
                                           _ptr(q_pos), k, _ptr(idx), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)))
    return idx


def dsa_indexer_warmup_workspace_size(T: int, S: int, H_I: int, d_I: int) -> int:
    return int(load_library().dsa_indexer_warmup_workspace_size(T, S, H_I, d_I))


def dsa_indexer_warmup(q, kv, sm_scale: float, q8, q_scale, w, k8, k_scale, q_pos, loss, dw, dq, dk,
                       workspace=None, stream=None):
    """Indexer warm-up: the KL loss of the index scores' softmax against the main attention's
    head-averaged dense distribution, and its gradients.  q bf16 [T, H, 576], kv bf16 [S, 576];
    indexer inputs as for dsa_indexer_logits (contiguous keys); outputs fp32 loss [T],
    dw [T, H_I], dq [T, H_I, d_I], dk [S, d_I].  ``workspace``: a uint8 CUDA tensor of at least
    dsa_indexer_warmup_workspace_size(T, S, H_I, d_I) bytes; taken from PyTorch when None."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(q8, torch.uint8, "q8", 3)
    _need(q_scale, torch.float32, "q_scale", 1)
    _need(w, torch.float32, "w", 2)
    _need(k8, torch.uint8, "k8", 2)
    _need(k_scale, torch.float32, "k_scale", 1)
    _need(q_pos, torch.int32, "q_pos", 1)
    for t, name, dim in ((loss, "loss", 1), (dw, "dw", 2), (dq, "dq", 3), (dk, "dk", 2)):
        _need(t, torch.float32, name, dim)
    T, H, D = q.shape
    S = kv.shape[0]
    _, HI, dI = q8.shape
    if D != 576 or kv.shape[1] != 576 or q8.shape[0] != T or q_scale.shape[0] != T or tuple(w.shape) != (T, HI) \
            or tuple(k8.shape) != (S, dI) or k_scale.shape[0] != S or q_pos.shape[0] != T \
            or loss.shape[0] != T or tuple(dw.shape) != (T, HI) or tuple(dq.shape) != (T, HI, dI) \
            or tuple(dk.shape) != (S, dI):
        raise ValueError("inconsistent shapes")
    if workspace is None:
        need = dsa_indexer_warmup_workspace_size(T, S, HI, dI)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(workspace, "workspace")
    _check(load_library().dsa_indexer_warmup(_ptr(q), _ptr(kv), H, float(sm_scale), _ptr(q8), _ptr(q_scale),
                                             _ptr(w), HI, dI, _ptr(k8), _ptr(k_scale), _ptr(q_pos), T, S, _ptr(loss),
                                             _ptr(dw), _ptr(dq), _ptr(dk), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream)))
    return loss, dw, dq, dk


def dsa_sparse_mla_prefill(q, kv, idx, sm_scale: float, out, lse, stream=None):
    """Sparse MQA-mode MLA: q bf16 [T, H, 576], kv bf16 [S, 576], idx int32 [T, k]
    -> out bf16 [T, H, 512], lse fp32 [T, H]."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(idx, torch.int32, "idx", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    T, H, D = q.shape
    S = kv.shape[0]
    k = idx.shape[1]
    if D != 576 or kv.shape[1] != 576 or idx.shape[0] != T or tuple(out.shape) != (T, H, 512) \
            or tuple(lse.shape) != (T, H):
        raise ValueError("inconsistent shapes (D must be 576, Dv 512)")
    _check(load_library().dsa_sparse_mla_prefill(_ptr(q), _ptr(kv), S, _ptr(idx), T, H, k, float(sm_scale),
                                                 _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


def dsa_sparse_mla_decode_workspace_size(B: int, H: int, k: int) -> int:
    return int(load_library().dsa_sparse_mla_decode_workspace_size(B, H, k))


def dsa_sparse_mla_decode_paged(q, kv_pool, block_table, ctx_len, idx, sm_scale: float, out, lse,
                                workspace=None, stream=None):
    """Paged decode attention: q bf16 [B, H, 576], kv_pool bf16 [P, page, 576],
    block_table int32 [B, max_pages], ctx_len int32 [B], idx int32 [B, k] (logical positions).
    ``workspace``: a uint8 CUDA tensor of at least dsa_sparse_mla_decode_workspace_size(B, H, k)
    bytes; when None and the call needs one, it is taken from PyTorch's allocator."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_pool, torch.bfloat16, "kv_pool", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    _need(idx, torch.int32, "idx", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    B, H, D = q.shape
    P, ps, D2 = kv_pool.shape
    k = idx.shape[1]
    if D != 576 or D2 != 576 or block_table.shape[0] != B or ctx_len.shape[0] != B or idx.shape[0] != B \
            or tuple(out.shape) != (B, H, 512) or tuple(lse.shape) != (B, H):
        raise ValueError("inconsistent shapes")
    ws_bytes = 0
    if workspace is None:
        need = dsa_sparse_mla_decode_workspace_size(B, H, k)
        if need:  # device memory from PyTorch's caching allocator (256-byte aligned)
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().dsa_sparse_mla_decode_paged(_ptr(q), _ptr(kv_pool), P, ps, _ptr(block_table),
                                                      block_table.shape[1], _ptr(ctx_len), _ptr(idx), B, H, k,
                                                      float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                                      ws_bytes, _stream(stream)))
    return out, lse


def dsa_sparse_mla_decode_paged_noalloc(q, kv_pool, block_table, ctx_len, idx, sm_scale: float, out, lse,
                                        stream=None):
    """dsa_sparse_mla_decode_paged for callers that cannot allocate device memory:
    the library's static device buffer serves as the workspace, and this wrapper
    allocates nothing either.  Same arguments, minus the workspace."""
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_pool, torch.bfloat16, "kv_pool", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    _need(idx, torch.int32, "idx", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    B, H, D = q.shape
    P, ps, D2 = kv_pool.shape
    k = idx.shape[1]
    if D != 576 or D2 != 576 or block_table.shape[0] != B or ctx_len.shape[0] != B or idx.shape[0] != B \
            or tuple(out.shape) != (B, H, 512) or tuple(lse.shape) != (B, H):
        raise ValueError("inconsistent shapes")
    _check(load_library().dsa_sparse_mla_decode_paged_noalloc(_ptr(q), _ptr(kv_pool), P, ps, _ptr(block_table),
                                                              block_table.shape[1], _ptr(ctx_len), _ptr(idx), B, H,
                                                              k, float(sm_scale), _ptr(out), _ptr(lse),
                                                              _stream(stream)))
    return out, lse


def dsa_mla_decode_workspace_size(B: int, H: int) -> int:
    return int(load_library().dsa_mla_decode_workspace_size(B, H))


def dsa_mla_decode_paged(q, kv_pool, block_table, ctx_len, sm_scale: float, out, lse, workspace=None, stream=None):
    """Dense paged decode attention over every position below ctx_len: q bf16 [B, H, 576], kv_pool bf16
    [P, page, 576], block_table int32 [B, max_pages], ctx_len int32 [B] -> out bf16 [B, H, 512], lse fp32 [B, H].
    ``workspace``: a CUDA tensor of at least dsa_mla_decode_workspace_size(B, H) bytes; taken from PyTorch's
    allocator when None."""
    if _native("mla_decode_paged", q, kv_pool, block_table, ctx_len, sm_scale, out, lse, workspace, stream):
        return out, lse
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not isinstance(kv_pool, torch.Tensor) or kv_pool.dim() != 3 \
            or not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise TypeError("q and kv_pool must be 3-D, block_table a 2-D torch.Tensor")
    cur, bf16, i32, mp = _device(), torch.bfloat16, torch.int32, block_table.shape[1]
    B, H, _ = q.shape
    P, ps, _ = kv_pool.shape
    lib = _lib or load_library()
    a_q, a_kv = _at(q, cur, "q", bf16, (B, H, 576)), _at(kv_pool, cur, "kv_pool", bf16, (P, ps, 576))
    a_bt, a_ctx = _at(block_table, cur, "block_table", i32, (B, mp)), _at(ctx_len, cur, "ctx_len", i32, (B,))
    a_out, a_lse = _at(out, cur, "out", bf16, (B, H, 512)), _at(lse, cur, "lse", torch.float32, (B, H))
    need = 0 if workspace is not None else lib.dsa_mla_decode_workspace_size(B, H)
    ws, ws_bytes, keep = _workspace(workspace, need, cur, stream)
    _check(lib.dsa_mla_decode_paged(a_q, a_kv, P, ps, a_bt, mp, a_ctx, B, H, float(sm_scale), a_out, a_lse, ws, ws_bytes,
                                    _raw_stream(stream, cur)))
    return out, lse


def _host(t: torch.Tensor, dtype, name: str, dim: int):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.is_cuda or not t.is_contiguous() or t.dim() != dim:
        raise ValueError(f"{name}: expected a contiguous {dim}-d host tensor of {dtype}")


def dsa_prefill_host_workspace_size(T: int, S: int, H_I: int, d_I: int, H: int, k: int, chunk_rows: int) -> int:
    return int(load_library().dsa_prefill_host_workspace_size(T, S, H_I, d_I, H, k, chunk_rows))


def dsa_prefill_host(q8, q_scale, w, q_pos, k8, k_scale, q, kv, sm_scale: float, k: int, out, lse,
                     chunk_rows: int = 4096, workspace=None, stream=None):
    """The whole prefill path on HOST tensors (pinned for overlapped copies): q8 uint8 [T, H_I, d_I],
    q_scale f32 [T], w f32 [T, H_I], q_pos i32 [T], k8 uint8 [S, d_I], k_scale f32 [S], q bf16 [T, H, 576],
    kv bf16 [S, 576] -> out bf16 [T, H, 512], lse f32 [T, H] (host).  ``workspace``: a uint8 CUDA tensor of
    dsa_prefill_host_workspace_size(...) bytes, taken from PyTorch's allocator when None."""
    _host(q8, torch.uint8, "q8", 3)
    _host(q_scale, torch.float32, "q_scale", 1)
    _host(w, torch.float32, "w", 2)
    _host(q_pos, torch.int32, "q_pos", 1)
    _host(k8, torch.uint8, "k8", 2)
    _host(k_scale, torch.float32, "k_scale", 1)
    _host(q, torch.bfloat16, "q", 3)
    _host(kv, torch.bfloat16, "kv", 2)
    _host(out, torch.bfloat16, "out", 3)
    _host(lse, torch.float32, "lse", 2)
    T, H_I, d_I = q8.shape
    S = k8.shape[0]
    H = q.shape[1]
    need = dsa_prefill_host_workspace_size(T, S, H_I, d_I, H, k, chunk_rows)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=torch.cuda.current_device())
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().dsa_prefill_host(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(q_pos), _ptr(k8), _ptr(k_scale),
                                           _ptr(q), _ptr(kv), T, S, H_I, d_I, H, k, float(sm_scale), _ptr(out),
                                           _ptr(lse), chunk_rows, _ptr(workspace), ws_bytes, _stream(stream)))
    return out, lse


def dsa_prefill_host_trace(max_chunks: int):
    """Start (max_chunks > 0) or end (0) the per-chunk timeline record of dsa_prefill_host calls."""
    _check(load_library().dsa_prefill_host_trace(int(max_chunks)))


def dsa_prefill_host_trace_read(max_chunks: int):
    """The recorded timeline: (ms [n, 6] float32 from the first recorded call's start to each chunk's
    input-copy begin/end, stages begin/end, output-copy begin/end; call [n]; rows [n])."""
    ms = np.full((max_chunks, 6), np.nan, dtype=np.float32)
    call = np.zeros(max_chunks, dtype=np.int32)
    rows = np.zeros(max_chunks, dtype=np.int32)
    n = ctypes.c_int(0)
    _check(load_library().dsa_prefill_host_trace_read(ms.ctypes.data, call.ctypes.data, rows.ctypes.data,
                                                       int(max_chunks), ctypes.byref(n)))
    return ms[:n.value], call[:n.value], rows[:n.value]


def dsa_selftest_wait_timeout(limit_us: int, stream=None):
    """Run one bounded pipeline wait that nothing completes; it sets DSA_DEV_TIMEOUT after limit_us."""
    _check(load_library().dsa_selftest_wait_timeout(int(limit_us), _stream(stream)))


def dsa_get_device_status(stream=None) -> int:
    """Read and clear the device status word (DSA_DEV_* bits)."""
    v = ctypes.c_uint32(0)
    _check(load_library().dsa_get_device_status(_stream(stream), ctypes.byref(v)))
    return int(v.value)

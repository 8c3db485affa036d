"""Python binding of libqmm.so (the C ABI in include/qmm.h).

Argument marshalling only: every function checks tensor devices, dtypes and
shapes, then passes raw device pointers, sizes and the current CUDA stream to
the library.  All arithmetic runs in the library's CUDA kernels; if the
library is missing, the first call raises instead of computing anything
another way.

Tensor conventions (all CUDA, contiguous):
  codes   torch.uint8  [N, K]           one code per byte (int8 bit pattern for bits=8)
  packed  torch.int32  [N, K*bits/32]   32-bit code words (bit patterns)
  scales  torch.float16 [N, K/group]
  biases  torch.float16 [N, K/group]    bits=4 only, else None
  x       torch.float32 [M, K] (gemv) or torch.bfloat16 [M, K] (gemm)
  y       torch.float32 [M, N]
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "qmm.h")

QMM_OK = 0
STATUS = {0: "QMM_OK", -1: "QMM_ERR_ARG", -2: "QMM_ERR_SHAPE", -3: "QMM_ERR_ALIGN",
          -4: "QMM_ERR_UNSUPPORTED", -5: "QMM_ERR_CUDA", -6: "QMM_ERR_DEVICE_TIMEOUT"}

_lock = threading.Lock()
_lib = None


class QmmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)}")


def declared_symbols() -> list[str]:
    """Names of the entry points declared in include/qmm.h."""
    text = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"\b(qmm_[a-z_0-9]+)\s*\(", text)))


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it first (python -m quantized_weight_gb300.build)")
            L = ctypes.CDLL(LIB_PATH)
            i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
            L.qmm_pack.argtypes = [vp, vp, i64, i64, i32, vp]
            L.qmm_unpack.argtypes = [vp, vp, i64, i64, i32, vp]
            L.qmm_dequant.argtypes = [vp, vp, vp, vp, i64, i64, i32, i32, vp]
            L.qmm_gemv.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
            L.qmm_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
            L.qmm_quantize.argtypes = [vp, vp, vp, vp, i64, i64, i32, vp]
            L.qmm_gather_dequant.argtypes = [vp, i64, vp, vp, vp, vp, i64, i64, i32, i32, vp]
            L.qmm_gemv_argmax_workspace_size.argtypes = [i64, i64]
            L.qmm_gemv_argmax_workspace_size.restype = ctypes.c_size_t
            L.qmm_gemv_argmax.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, ctypes.c_size_t, vp]
            L.qmm_gemv_argmax_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, vp]
            sz, f32 = ctypes.c_size_t, ctypes.c_float
            L.qmm_kv_cache_size.argtypes = [i64, i64, i64, i32, i32]
            L.qmm_kv_plan.argtypes = [vp, vp, vp, i64, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]
            L.qmm_kv_append.argtypes = [vp, vp, i32, i64, i64, i64, i64, vp, vp, i64, i64, i64, i64, i32, i32, vp]
            L.qmm_kv_read.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i64, i32, i32, vp]
            L.qmm_kv_attend_workspace_size.argtypes = [i64, i64, i64, i64, i64]
            L.qmm_kv_attend.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64,
                                        i32, i32, f32, i64, vp, sz, vp]
            L.qmm_kv_attend_tiles.argtypes = [i32, i64, i64, i64, i64, i64]
            L.qmm_kv_cache_size.restype = L.qmm_kv_attend_workspace_size.restype = sz
            L.qmm_mx4_scales_size.argtypes = [i64, i64]
            L.qmm_mx4_scales_size.restype = sz
            L.qmm_mx4_quantize.argtypes = [vp, i32, i64, i64, vp, vp, i64, i64, i64, vp]
            L.qmm_mx4_dequant.argtypes = [vp, vp, vp, i64, i64, i64, vp]
            L.qmm_mx4_gemm.argtypes = [vp, vp, vp, vp, vp, i32, i32, i64, i64, i64, vp]
            L.qmm_mx4_gemm_tile.argtypes = [i32, i64, i64, i64, i64, i64]
            L.qmm_moe_rows.argtypes = [i64, i64, i64]
            L.qmm_moe_rows.restype = i64
            L.qmm_moe_plan.argtypes = [vp, i32, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp]
            L.qmm_moe_quantize.argtypes = [vp, i32, i64, i32, vp, vp, vp, i64, i64, i64, i64, vp]
            L.qmm_moe_gemm.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i64, i64, i64, i64, i64, vp]
            L.qmm_moe_combine.argtypes = [vp, i32, vp, vp, vp, i32, i64, i64, i64, i64, vp]
            L.qmm_check.argtypes = [vp]
            L.qmm_test_timeout_next_decode.argtypes = L.qmm_test_timeout_next_attend.argtypes = [i64]
            L.qmm_test_timeout_next_mx4.argtypes = [i64]
            L.qmm_status_string.argtypes = [i32]
            L.qmm_status_string.restype = ctypes.c_char_p
            L.qmm_abi_version.argtypes = []
            for f in ("qmm_pack", "qmm_unpack", "qmm_dequant", "qmm_gemv", "qmm_gemm", "qmm_quantize",
                      "qmm_gather_dequant", "qmm_gemv_argmax", "qmm_gemv_argmax_noalloc", "qmm_check",
                      "qmm_test_timeout_next_decode", "qmm_test_timeout_next_attend", "qmm_abi_version", "qmm_kv_plan", "qmm_kv_append", "qmm_kv_read",
                      "qmm_kv_attend", "qmm_kv_attend_tiles", "qmm_mx4_quantize", "qmm_mx4_dequant", "qmm_mx4_gemm",
                      "qmm_mx4_gemm_tile", "qmm_test_timeout_next_mx4", "qmm_moe_plan", "qmm_moe_quantize", "qmm_moe_gemm", "qmm_moe_combine"):
                getattr(L, f).restype = i32
            _lib = L
    return _lib


def _status_string(status: int) -> str:
    try:
        return lib().qmm_status_string(int(status)).decode()
    except Exception:
        return STATUS.get(int(status), str(status))


try:                                   # the handle alone: a Stream object costs 3 us a call
    from torch._C import _cuda_getCurrentRawStream, _cuda_getDevice

    def _current_stream() -> int:
        return _cuda_getCurrentRawStream(_cuda_getDevice())
except ImportError:
    def _current_stream() -> int:
        return torch.cuda.current_stream().cuda_stream


def _stream(stream) -> int:
    return _current_stream() if stream is None else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _call(what, rc):
    if rc != QMM_OK:
        raise QmmError(rc, what)


def pack(codes: torch.Tensor, bits: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    N, K = codes.shape
    _need(codes, "codes", torch.uint8)
    if out is None:
        out = torch.empty((N, K * bits // 32), dtype=torch.int32, device=codes.device)
    _need(out, "out", torch.int32, (N, K * bits // 32))
    _call("qmm_pack", lib().qmm_pack(_ptr(codes), _ptr(out), N, K, bits, _stream(stream)))
    return out


def unpack(packed: torch.Tensor, N: int, K: int, bits: int, out=None, stream=None) -> torch.Tensor:
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    if out is None:
        out = torch.empty((N, K), dtype=torch.uint8, device=packed.device)
    _need(out, "out", torch.uint8, (N, K))
    _call("qmm_unpack", lib().qmm_unpack(_ptr(packed), _ptr(out), N, K, bits, _stream(stream)))
    return out


def _coeffs(scales, biases, N, K, bits, group):
    _need(scales, "scales", torch.float16, (N, K // group))
    if bits == 4:
        _need(biases, "biases", torch.float16, (N, K // group))
    elif biases is not None:
        raise ValueError("biases must be None unless bits == 4")


def dequant(packed, scales, biases, N, K, bits, group, out=None, stream=None) -> torch.Tensor:
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    _coeffs(scales, biases, N, K, bits, group)
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=packed.device)
    _need(out, "out", torch.float32, (N, K))
    _call("qmm_dequant", lib().qmm_dequant(_ptr(packed), _ptr(scales), _ptr(biases), _ptr(out),
                                           N, K, bits, group, _stream(stream)))
    return out


def gemv(x, packed, scales, biases, N, bits, group, out=None, stream=None) -> torch.Tensor:
    """Decode product y[M, N] = x[M, K] . dequant(W)^T, float32 x, 1 <= M <= 8."""
    M, K = x.shape
    _need(x, "x", torch.float32)
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    _coeffs(scales, biases, N, K, bits, group)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, (M, N))
    _call("qmm_gemv", lib().qmm_gemv(_ptr(x), _ptr(packed), _ptr(scales), _ptr(biases), _ptr(out),
                                     M, N, K, bits, group, _stream(stream)))
    return out


def gemm(x, packed, scales, biases, N, bits, group, out=None, stream=None) -> torch.Tensor:
    """Prefill product y[M, N] = x[M, K] . dequant(W)^T, bfloat16 x, any M, bits 4 / 8 / 1."""
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    _coeffs(scales, biases, N, K, bits, group)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, (M, N))
    _call("qmm_gemm", lib().qmm_gemm(_ptr(x), _ptr(packed), _ptr(scales), _ptr(biases), _ptr(out),
                                     M, N, K, bits, group, _stream(stream)))
    return out


def argmax_workspace(M: int, N: int, device="cuda") -> torch.Tensor:
    """A zeroed work area for gemv_argmax (reusable: every call leaves it ready)."""
    n = int(lib().qmm_gemv_argmax_workspace_size(M, N))
    return torch.zeros(((n + 15) // 16 * 16,), dtype=torch.uint8, device=device)


def gemv_argmax(x, packed, scales, biases, N, bits, group, workspace, idx=None, val=None, stream=None):
    """Greedy head: (idx int32 [M], val float32 [M]) of argmax_n (x . dequant(W)^T)[m, n]."""
    M, K = x.shape
    _need(x, "x", torch.float32)
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    _coeffs(scales, biases, N, K, bits, group)
    _need(workspace, "workspace", torch.uint8)
    if idx is None:
        idx = torch.empty((M,), dtype=torch.int32, device=x.device)
    if val is None:
        val = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(idx, "idx", torch.int32, (M,))
    _need(val, "val", torch.float32, (M,))
    _call("qmm_gemv_argmax", lib().qmm_gemv_argmax(_ptr(x), _ptr(packed), _ptr(scales), _ptr(biases), _ptr(idx),
                                                   _ptr(val), M, N, K, bits, group, _ptr(workspace),
                                                   workspace.numel(), _stream(stream)))
    return idx, val


def gemv_argmax_noalloc(x, packed, scales, biases, N, bits, group, idx=None, val=None, stream=None):
    """gemv_argmax for one token with the library's static work area (no workspace argument)."""
    M, K = x.shape
    if M != 1:
        raise ValueError("gemv_argmax_noalloc takes one token (M == 1)")
    _need(x, "x", torch.float32)
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    _coeffs(scales, biases, N, K, bits, group)
    if idx is None:
        idx = torch.empty((1,), dtype=torch.int32, device=x.device)
    if val is None:
        val = torch.empty((1,), dtype=torch.float32, device=x.device)
    _need(idx, "idx", torch.int32, (1,))
    _need(val, "val", torch.float32, (1,))
    _call("qmm_gemv_argmax_noalloc", lib().qmm_gemv_argmax_noalloc(
        _ptr(x), _ptr(packed), _ptr(scales), _ptr(biases), _ptr(idx), _ptr(val), N, K, bits, group, _stream(stream)))
    return idx, val


def quantize(w, group=64, out=None, stream=None):
    """INT4 affine quantization of float32 w [N, K]: (packed int32 [N, K/8],
    scales float16 [N, K/group], biases float16 [N, K/group])."""
    N, K = w.shape
    _need(w, "w", torch.float32)
    if out is None:
        out = (torch.empty((N, K // 8), dtype=torch.int32, device=w.device),
               torch.empty((N, K // group), dtype=torch.float16, device=w.device),
               torch.empty((N, K // group), dtype=torch.float16, device=w.device))
    packed, scales, biases = out
    _need(packed, "packed", torch.int32, (N, K // 8))
    _need(scales, "scales", torch.float16, (N, K // group))
    _need(biases, "biases", torch.float16, (N, K // group))
    _call("qmm_quantize", lib().qmm_quantize(_ptr(w), _ptr(packed), _ptr(scales), _ptr(biases), N, K, group,
                                             _stream(stream)))
    return packed, scales, biases


def gather_dequant(ids, packed, scales, biases, N, K, bits, group, out=None, stream=None) -> torch.Tensor:
    """out[t, :] = dequant(W[ids[t], :]); int32 ids [T]; an id outside [0, N) gives a NaN row."""
    _need(ids, "ids", torch.int32)
    T = ids.numel()
    _need(packed, "packed", torch.int32, (N, K * bits // 32))
    _coeffs(scales, biases, N, K, bits, group)
    if out is None:
        out = torch.empty((T, K), dtype=torch.float32, device=packed.device)
    _need(out, "out", torch.float32, (T, K))
    _call("qmm_gather_dequant", lib().qmm_gather_dequant(_ptr(ids), T, _ptr(packed), _ptr(scales), _ptr(biases),
                                                         _ptr(out), N, K, bits, group, _stream(stream)))
    return out


_I32 = torch.int32
_KV_DTYPE = {torch.float32: 0, torch.bfloat16: 1}


# The checks of the cache calls come in two steps: one test that a good argument
# passes, and _need's messages where it does not.  A decode step makes several such calls a layer.

def _i32(t, name, shape) -> int:
    """Pointer of a contiguous int32 CUDA tensor of the given shape."""
    if not (t.dtype is _I32 and t.is_cuda and t.shape == shape and t.is_contiguous()):
        _need(t, name, _I32, shape)
    return t.data_ptr()


def _kv_rows(t, name, dtype, shape):
    """Token and head strides of a [tokens, heads, head_dim] tensor whose last dimension is contiguous."""
    if not (t.is_cuda and t.dtype is dtype and t.shape == shape):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return (token if shape[0] > 1 else 0), (head if shape[1] > 1 else 0)   # a lone row has no stride to keep


def _kv_dtype(dtype) -> int:
    dt = _KV_DTYPE.get(dtype)
    if dt is None:
        raise TypeError(f"keys, values and queries are float32 or bfloat16, got {dtype}")
    return dt


def _kv_cache(cache, D, page, group):
    """(pages, kv_heads, pointer) of a cache."""
    if not (cache.dtype is torch.uint8 and cache.is_cuda and cache.is_contiguous()):
        _need(cache, "cache", torch.uint8)
    shape = cache.shape
    if len(shape) != 3 or shape[2] * 16 != page * (16 * D + 128 * (D // group)):
        raise ValueError(f"cache must be [pages, kv_heads, bytes] as kv_cache() makes it for head_dim {D}, page {page}, "
                         f"group {group}; got {tuple(shape)}")
    return shape[0], shape[1], cache.data_ptr()


def _kv_table(table, B):
    """(max_blocks, pointer) of a block table."""
    shape = table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_blocks], got {tuple(shape)}")
    return shape[1], _i32(table, "block_table", shape)


def _kv_out(t, name, dtype, shape) -> int:
    if not (t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, shape)
    return t.data_ptr()


def kv_cache(pages, kv_heads, head_dim, page, group=64, device="cuda") -> torch.Tensor:
    """The 4-bit key/value cache of one layer: uint8 [pages, kv_heads, bytes of a head's page]."""
    size = lib().qmm_kv_cache_size
    n = int(size(1, kv_heads, head_dim, page, group))
    if n == 0 or (pages != 0 and size(pages, kv_heads, head_dim, page, group) == 0):
        raise ValueError(f"no cache of head_dim {head_dim}, page {page}, group {group} with {pages} pages of {kv_heads} heads")
    return torch.zeros((pages, kv_heads, n // kv_heads), dtype=torch.uint8, device=device)


def kv_plan(cached, fresh, free_pages, block_table, tokens, page, out=None, stream=None):
    """One step's (slots [tokens], positions [tokens], cu [B + 1], lens [B], need [1]), int32, from the requests'
    lengths; block_table [B, max_blocks] is completed in place with pages from the front of free_pages."""
    shape = cached.shape
    B = cached.numel()
    pc, pf, pp = _i32(cached, "cached", shape), _i32(fresh, "fresh", (B,)), _i32(free_pages, "free_pages", free_pages.shape)
    blocks, pt = _kv_table(block_table, B)
    if out is None:
        buf = torch.empty(2 * (tokens + B + 1), dtype=_I32, device=cached.device)
        out = buf.unsafe_split_with_sizes((tokens, tokens, B + 1, B, 1))     # no views that autograd follows: 2 us less
        a = buf.data_ptr()
        outs = a, a + 4 * tokens, a + 8 * tokens, a + 8 * tokens + 4 * (B + 1), a + 8 * tokens + 4 * (2 * B + 1)
    else:
        outs = tuple(_i32(t, name, (n,)) for t, name, n in zip(out, ("slots", "positions", "cu", "lens", "need"),
                                                               (tokens, tokens, B + 1, B, 1)))
    _call("qmm_kv_plan", lib().qmm_kv_plan(pc, pf, pp, free_pages.numel(), pt, B, blocks, page, tokens, *outs,
                                           _stream(stream)))
    return out


def kv_append(k, v, slots, cache, page, group=64, stream=None) -> None:
    """Quantize k, v [T, kv_heads, head_dim] (float32 or bfloat16) into the cache's slots; a slot outside it is skipped."""
    dtype, shape = k.dtype, k.shape
    T, H, D = shape
    dt = _kv_dtype(dtype)
    kt, kh = _kv_rows(k, "k", dtype, shape)
    vt, vh = _kv_rows(v, "v", dtype, shape)
    ps = _i32(slots, "slots", (T,))
    pages, heads, pc = _kv_cache(cache, D, page, group)
    if heads != H:
        raise ValueError(f"cache has {heads} kv heads, k has {H}")
    _call("qmm_kv_append", lib().qmm_kv_append(k.data_ptr(), v.data_ptr(), dt, kt, kh, vt, vh, ps, pc, T, pages, H, D,
                                               page, group, _stream(stream)))


def kv_read(slots, cache, head_dim, page, group=64, dtype=torch.float32, out=None, stream=None):
    """The (keys, values) [T, kv_heads, head_dim] that the slots hold; a slot outside the cache gives NaN rows."""
    ps = _i32(slots, "slots", slots.shape)
    pages, H, pc = _kv_cache(cache, head_dim, page, group)
    T, dt = slots.numel(), _kv_dtype(dtype)
    shape = (T, H, head_dim)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=cache.device), torch.empty(shape, dtype=dtype, device=cache.device)
        pk, pv = out[0].data_ptr(), out[1].data_ptr()
    else:
        pk, pv = _kv_out(out[0], "k", dtype, shape), _kv_out(out[1], "v", dtype, shape)
    _call("qmm_kv_read", lib().qmm_kv_read(ps, pc, pk, pv, dt, T, pages, H, head_dim, page, group, _stream(stream)))
    return out


def kv_attend_workspace(B, heads, kv_heads, head_dim, max_fresh=1, device="cuda") -> torch.Tensor:
    """A zeroed work area for kv_attend (reusable: every call leaves it ready)."""
    n = int(lib().qmm_kv_attend_workspace_size(B, heads, kv_heads, head_dim, max_fresh))
    if n == 0:
        raise ValueError(f"no attention of {heads} heads over {kv_heads} kv heads of {head_dim}")
    return torch.zeros(((n + 15) // 16 * 16,), dtype=torch.uint8, device=device)


def kv_attend_tiles(dtype, B, heads, kv_heads, head_dim, max_fresh) -> bool:
    """Whether kv_attend takes such a call on tiles of 128 rows of q (include/qmm.h says what is rounded there)."""
    r = lib().qmm_kv_attend_tiles(_kv_dtype(dtype), B, heads, kv_heads, head_dim, max_fresh)
    _call("qmm_kv_attend_tiles", min(r, 0))
    return r == 1


def kv_attend(q, cache, block_table, lens, page, group, workspace, cu=None, max_fresh=1, scale=None, window=0, out=None,
              stream=None) -> torch.Tensor:
    """Attention of q [T, heads, head_dim] (float32 or bfloat16) over each request's cached tokens, causal, with an
    optional sliding window: request b's queries are tokens cu[b] .. cu[b + 1] - 1 (cu None: token b), the last of
    its lens[b] tokens.  scale defaults to head_dim ** -0.5."""
    dtype, shape = q.dtype, q.shape
    T, H, D = shape
    dt = _kv_dtype(dtype)
    qt, qh = _kv_rows(q, "q", dtype, shape)
    pages, heads, pc = _kv_cache(cache, D, page, group)
    pl = _i32(lens, "lens", lens.shape)
    B = lens.numel()
    blocks, pt = _kv_table(block_table, B)
    pcu = None if cu is None else _i32(cu, "cu", (B + 1,))
    if not (workspace.dtype is torch.uint8 and workspace.is_cuda and workspace.is_contiguous()):
        _need(workspace, "workspace", torch.uint8)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        po = out.data_ptr()
    else:
        po = _kv_out(out, "out", dtype, shape)
    _call("qmm_kv_attend", lib().qmm_kv_attend(
        q.data_ptr(), dt, qt, qh, pc, pt, pl, pcu, po, T, B, blocks, max_fresh, pages, H,
        heads, D, page, group, D ** -0.5 if scale is None else scale, window, workspace.data_ptr(), workspace.numel(),
        _stream(stream)))
    return out


# ---------------------------------------------------------------- microscaled 4-bit products and experts
#
# As for the cache calls, one test that a good argument passes comes first; what the call itself has made is not tested.

_F32 = torch.float32
_U8 = torch.uint8
_MX_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
try:
    _device = torch._C._cuda_getDevice
except AttributeError:
    _device = torch.cuda.current_device


def _mx_dtype(dtype) -> int:
    dt = _MX_DTYPE.get(dtype)
    if dt is None:
        raise TypeError(f"values are float32 or bfloat16, got {dtype}")
    return dt


def _here(t, name, dtype, shape) -> int:
    """Pointer of a contiguous tensor of the given type and shape on the current device (where the kernels run)."""
    if not (t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, shape)
    if t.get_device() != _device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_device()}")
    return t.data_ptr()


def _new(shape, dtype, device, stream):
    """An output of a call on `stream`: its memory belongs to that stream, so that no one else's work is in its way."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _mx_rows(x, name) -> int:
    """Stride between the rows of x [..., rows, K] on the current device, whose rows are contiguous."""
    strides, shape = x.stride(), x.shape
    if not (x.is_cuda and len(strides) > 1 and strides[-1] == 1 and x.get_device() == _device()):
        if not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if x.get_device() != _device():
            raise ValueError(f"{name} is on {x.device}, the current device is cuda:{_device()}")
        if len(strides) < 2:
            raise ValueError(f"{name} must have rows, got {tuple(shape)}")
        if shape[-1] > 1 and x.numel() > 0:
            raise ValueError(f"{name} must be contiguous in its last dimension")
    return strides[-2] if shape[-2] > 1 else 0                        # a lone row has no stride to keep


def mx4_scales_size(rows, K) -> int:
    """Bytes of the scales of a matrix [rows, K]."""
    if rows < 0 or K < 0 or K % 32 != 0 or rows >= 1 << 31 or K >= 1 << 31:
        raise ValueError(f"no microscaled matrix of {rows} rows of {K}: K is a multiple of 32, both are below 2**31")
    return ((rows + 127) // 128) * ((K + 127) // 128) * 512


def mx4_scales(plain) -> torch.Tensor:
    """Scales of a checkpoint, bytes [..., rows, K / 32], in the tiles that the products read (include/qmm.h)."""
    if plain.is_floating_point():
        raise TypeError(f"scales are bytes, got {plain.dtype}: pass their bits, .view(torch.uint8)")
    lead, (rows, blocks) = plain.shape[:-2], plain.shape[-2:]
    across, down = -(-blocks // 4), -(-rows // 128)
    full = torch.zeros((*lead, down * 128, across * 4), dtype=torch.uint8, device=plain.device)
    full[..., :rows, :blocks] = plain
    n = len(lead)
    tiles = full.view(*lead, down, 4, 32, across, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return tiles.reshape(*lead, down * across * 512)


def _mx_matrix(codes, scales, name, lead=()):
    """(rows, K, pointers) of a microscaled matrix [*lead, rows, K / 8] and its scales."""
    shape = codes.shape
    if len(shape) == 2 and not lead:
        rows, k8 = shape
        size = ((rows + 127) >> 7) * ((k8 + 15) >> 4) * 512
        if (codes.dtype is _I32 and codes.is_cuda and codes.is_contiguous() and k8 & 3 == 0 and scales.dtype is _U8
                and scales.shape == (size,) and scales.is_contiguous() and codes.get_device() == scales.get_device() == _device()):
            return rows, k8 * 8, codes.data_ptr(), scales.data_ptr()
    if len(shape) != len(lead) + 2 or shape[:-2] != lead:
        raise ValueError(f"{name} must be [{', '.join(map(str, (*lead, 'rows', 'K / 8')))}], got {tuple(shape)}")
    rows, K = shape[-2], shape[-1] * 8
    pc = _here(codes, name, _I32, shape)
    return rows, K, pc, _here(scales, "scales", _U8, (*lead, mx4_scales_size(rows, K)))


def mx4_quantize(x, out=None, stream=None):
    """float32 or bfloat16 x [..., rows, K] to microscaled 4-bit (codes int32 [..., rows, K / 8], scales uint8 [..., bytes])."""
    dt, row, shape = _mx_dtype(x.dtype), _mx_rows(x, "x"), x.shape
    if len(shape) == 2:
        (rows, K), n, matrix = shape, 1, 0
        codes, scales = (rows, K // 8), (mx4_scales_size(rows, K),)
    else:
        (*lead, rows, K), n = shape, shape[:-2].numel()
        if len(lead) > 1:
            try:
                x = x.view(n, rows, K)
            except RuntimeError:
                raise ValueError(f"the leading dimensions of x must be one after the other, got strides {x.stride()}") from None
        matrix = x.stride(0) if n > 1 else 0
        codes, scales = (*lead, rows, K // 8), (*lead, mx4_scales_size(rows, K))
    if out is None:
        out = _new(codes, _I32, x.device, stream), _new(scales, _U8, x.device, stream)
        pc, ps = out[0].data_ptr(), out[1].data_ptr()
    else:
        pc, ps = _here(out[0], "codes", _I32, codes), _here(out[1], "scales", _U8, scales)
    _call("qmm_mx4_quantize", lib().qmm_mx4_quantize(x.data_ptr(), dt, matrix, row, pc, ps, n, rows, K, _stream(stream)))
    return out


def mx4_dequant(codes, scales, out=None, stream=None) -> torch.Tensor:
    """The float32 values [..., rows, K] of a microscaled matrix."""
    lead = codes.shape[:-2]
    rows, K, pc, ps = _mx_matrix(codes, scales, "codes", lead)
    shape = (*lead, rows, K) if lead else (rows, K)
    if out is None:
        out = _new(shape, _F32, codes.device, stream)
        po = out.data_ptr()
    else:
        po = _here(out, "out", _F32, shape)
    _call("qmm_mx4_dequant", lib().qmm_mx4_dequant(pc, ps, po, lead.numel() if lead else 1, rows, K, _stream(stream)))
    return out


def _mx_out(out, shape, dtype, device, stream):
    """(output, its type's number, its pointer)."""
    if out is None:
        dt = _mx_dtype(dtype)
        out = _new(shape, dtype, device, stream)
        return out, dt, out.data_ptr()
    return out, _mx_dtype(out.dtype), _here(out, "out", out.dtype, shape)


def mx4_gemm(x_codes, x_scales, codes, scales, gated=False, dtype=torch.float32, out=None, stream=None) -> torch.Tensor:
    """y [M, N] = x . w^T of microscaled x [M, K] and w [N, K], float32 or bfloat16; gated: codes and scales hold two matrices
    [2, N, K], and y = silu(x . g^T) * (x . u^T).  With out, dtype is out's."""
    M, K, px, pxs = _mx_matrix(x_codes, x_scales, "x_codes")
    N, KW, pc, ps = _mx_matrix(codes, scales, "codes", (2,) if gated else ())
    if KW != K:
        raise ValueError(f"x has rows of {K}, the weights of {KW}")
    out, dt, po = _mx_out(out, (M, N), dtype, x_codes.device, stream)
    _call("qmm_mx4_gemm", lib().qmm_mx4_gemm(px, pxs, pc, ps, po, dt, gated, M, N, K, _stream(stream)))
    return out


def mx4_gemm_tile(M, N, K, gated=False, experts=0, routed=0) -> int:
    """Which kernel takes a call of mx4_gemm, or of moe_gemm with so many experts (M: its R): the tokens of a tile, plus 1024
    where a pair of CTAs shares it."""
    r = lib().qmm_mx4_gemm_tile(gated, routed, M, experts, N, K)
    _call("qmm_mx4_gemm_tile", min(r, 0))
    return r


def moe_rows(T, E, k) -> int:
    """Rows that T tokens, each with k of E experts, take at most once sorted by expert."""
    n = int(lib().qmm_moe_rows(T, E, k))
    if n < 0:
        raise ValueError(f"no routing of {T} tokens to {k} of {E} experts")
    return n


def moe_plan(logits, k, normalize=True, out=None, stream=None):
    """Each token's k best experts of logits [T, E] (float32 or bfloat16; -infinity masks an expert): (experts int32 [T, k],
    weights float32 [T, k], places int32 [T, k], starts int32 [E], counts int32 [E]).  Expert e's rows are starts[e] ..
    starts[e] + counts[e] - 1 of moe_rows(T, E, k); places says which is whose.  weights are the softmax over the chosen
    experts (normalize) or over all."""
    dt, row = _mx_dtype(logits.dtype), _mx_rows(logits, "logits")
    T, E = logits.shape
    if out is None:
        device, tk = logits.device, (T, k)
        out = (_new(tk, _I32, device, stream), _new(tk, _F32, device, stream), _new(tk, _I32, device, stream),
               _new((E,), _I32, device, stream), _new((E,), _I32, device, stream))
        pe, pw, pp, ps, pc = [t.data_ptr() for t in out]
    else:
        pe, pw, pp, ps, pc = [_here(t, *n) for t, n in zip(out, (
            ("experts", _I32, (T, k)), ("weights", _F32, (T, k)), ("places", _I32, (T, k)), ("starts", _I32, (E,)),
            ("counts", _I32, (E,))))]
    _call("qmm_moe_plan", lib().qmm_moe_plan(logits.data_ptr(), dt, row, T, E, k, normalize, pe, pw, pp, ps, pc,
                                             _stream(stream)))
    return out


def moe_quantize(x, places, rows, out=None, sorted=False, stream=None):
    """mx4_quantize of x [T, K], each token's row to its places [T, k]: (codes int32 [rows, K / 8], scales).  sorted: x
    [rows, K] is sorted by expert already, and the rows of the places stay where they are.  Other rows are left alone (without
    `out`: as memory happens to be; no product of another row reads them)."""
    dt, row = _mx_dtype(x.dtype), _mx_rows(x, "x")
    n, K = x.shape
    T, k = places.shape
    if n != (rows if sorted else T):
        raise ValueError(f"x must be [{rows if sorted else T}, K], got {tuple(x.shape)}")
    pp = _here(places, "places", _I32, (T, k))
    size = mx4_scales_size(rows, K)
    if out is None:
        out = _new((rows, K // 8), _I32, x.device, stream), _new((size,), _U8, x.device, stream)
        pc, ps = out[0].data_ptr(), out[1].data_ptr()
    else:
        pc, ps = _here(out[0], "codes", _I32, (rows, K // 8)), _here(out[1], "scales", _U8, (size,))
    _call("qmm_moe_quantize", lib().qmm_moe_quantize(x.data_ptr(), dt, row, sorted, pp, pc, ps, T, k, rows, K, _stream(stream)))
    return out


def moe_gemm(x_codes, x_scales, codes, scales, starts, counts, routed=None, gated=False, dtype=torch.float32, out=None,
             stream=None) -> torch.Tensor:
    """mx4_gemm of each expert's rows of x [R, K] with its matrix of codes [E, N, K / 8] (gated: [E, 2, N, K / 8]): y [R, N].
    Rows of no expert are left alone (without `out`: as memory happens to be).  routed: how many rows the experts have
    together, about; it picks the launch's shape (default: what moe_rows made R of)."""
    R, K, px, pxs = _mx_matrix(x_codes, x_scales, "x_codes")
    E = starts.shape[0]
    N, KW, pc, ps = _mx_matrix(codes, scales, "codes", (E, 2) if gated else (E,))
    if KW != K:
        raise ValueError(f"x has rows of {K}, the weights of {KW}")
    pst, pco = _here(starts, "starts", _I32, (E,)), _here(counts, "counts", _I32, (E,))
    out, dt, po = _mx_out(out, (R, N), dtype, x_codes.device, stream)
    if routed is None:
        routed = max(R // 128, R - 127 * E)                           # a row an expert, or full segments
    _call("qmm_moe_gemm", lib().qmm_moe_gemm(px, pxs, pc, ps, pst, pco, po, dt, gated, routed, R, E, N, K, _stream(stream)))
    return out


def moe_combine(y, weights, places, dtype=None, out=None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[places[t, j]] of y [R, N]; weights None: all 1.  dtype defaults to y's."""
    shape, tk, ydtype = y.shape, places.shape, y.dtype
    if len(shape) != 2 or len(tk) != 2:
        raise ValueError(f"y must be [R, N] and places [T, k], got {tuple(shape)} and {tuple(tk)}")
    dt, py, pp = _mx_dtype(ydtype), _here(y, "y", ydtype, shape), _here(places, "places", _I32, tk)
    pw = None if weights is None else _here(weights, "weights", _F32, tk)
    (R, N), (T, k) = shape, tk
    out, do, po = _mx_out(out, (T, N), ydtype if dtype is None else dtype, y.device, stream)
    _call("qmm_moe_combine", lib().qmm_moe_combine(py, dt, pw, pp, po, do, T, k, R, N, _stream(stream)))
    return out


def test_timeout_next_decode(limit_ns: int) -> None:
    """Test hook: the next tensor-core decode launch makes one wait that runs
    out after limit_ns; it writes no output and the next check() raises
    QMM_ERR_DEVICE_TIMEOUT."""
    _call("qmm_test_timeout_next_decode", lib().qmm_test_timeout_next_decode(int(limit_ns)))


def test_timeout_next_attend(limit_ns: int) -> None:
    """Test hook: the next kv_attend launch on tiles of 128 rows makes one wait a block that runs out after limit_ns; it
    writes no row that sees a key and the next check() raises QMM_ERR_DEVICE_TIMEOUT."""
    _call("qmm_test_timeout_next_attend", lib().qmm_test_timeout_next_attend(int(limit_ns)))


def test_timeout_next_mx4(limit_ns: int) -> None:
    """Test hook: the next mx4_gemm or moe_gemm launch makes one wait a block that runs out after limit_ns; it writes nothing
    and the next check() raises QMM_ERR_DEVICE_TIMEOUT."""
    _call("qmm_test_timeout_next_mx4", lib().qmm_test_timeout_next_mx4(int(limit_ns)))


def check(stream=None) -> None:
    """Synchronize the stream and raise if a kernel failed or a device wait timed out."""
    _call("qmm_check", lib().qmm_check(_stream(stream)))

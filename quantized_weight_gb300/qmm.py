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
            L.qmm_check.argtypes = [vp]
            L.qmm_test_timeout_next_decode.argtypes = L.qmm_test_timeout_next_attend.argtypes = [i64]
            L.qmm_status_string.argtypes = [i32]
            L.qmm_status_string.restype = ctypes.c_char_p
            L.qmm_abi_version.argtypes = []
            for f in ("qmm_pack", "qmm_unpack", "qmm_dequant", "qmm_gemv", "qmm_gemm", "qmm_quantize",
                      "qmm_gather_dequant", "qmm_gemv_argmax", "qmm_gemv_argmax_noalloc", "qmm_check",
                      "qmm_test_timeout_next_decode", "qmm_test_timeout_next_attend", "qmm_abi_version", "qmm_kv_plan", "qmm_kv_append", "qmm_kv_read",
                      "qmm_kv_attend", "qmm_kv_attend_tiles"):
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


def test_timeout_next_decode(limit_ns: int) -> None:
    """Test hook: the next tensor-core decode launch makes one wait that runs
    out after limit_ns; it writes no output and the next check() raises
    QMM_ERR_DEVICE_TIMEOUT."""
    _call("qmm_test_timeout_next_decode", lib().qmm_test_timeout_next_decode(int(limit_ns)))


def test_timeout_next_attend(limit_ns: int) -> None:
    """Test hook: the next kv_attend launch on tiles of 128 rows makes one wait a block that runs out after limit_ns; it
    writes no row that sees a key and the next check() raises QMM_ERR_DEVICE_TIMEOUT."""
    _call("qmm_test_timeout_next_attend", lib().qmm_test_timeout_next_attend(int(limit_ns)))


def check(stream=None) -> None:
    """Synchronize the stream and raise if a kernel failed or a device wait timed out."""
    _call("qmm_check", lib().qmm_check(_stream(stream)))

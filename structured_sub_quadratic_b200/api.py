"""Python binding of the MonarchAttention C ABI (``include/monarch_attn.h``).

Argument marshalling only: torch tensors are passed to the library as raw
device pointers plus sizes, on the caller's current CUDA stream.  Every step
of the forward pass runs in the library's CUDA kernels; there is no fallback,
and a missing library raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

import torch

from ._build import LIB_PATH

MONARCH_OK = 0
MONARCH_ERR_INVALID_ARG = -1
MONARCH_ERR_UNSUPPORTED = -2
MONARCH_ERR_CUDA = -3
MONARCH_ERR_DEVICE_TIMEOUT = -4
MONARCH_ERR_NO_MEMORY = -5
MONARCH_ERR_SCRATCH_LIMIT = -6
MONARCH_ERR_BAD_INDEX = -7
DTYPE_BF16 = 0
DTYPE_F32 = 1
LAYOUTS = {"fh,w": 0, "w,fh": 1, "f,hw": 2, "hw,f": 3, "fw,h": 4, "h,fw": 5}

# Every symbol the header declares, with its ctypes signature.
_I, _P, _Z = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_L, _F, _D = ctypes.c_longlong, ctypes.c_float, ctypes.c_double
_SIZES = [_I] * 8  # B, H, b1, b2, d, T, c1, c2
SIGNATURES = {
    "monarch_attn_fwd": (_I, [_P, _P, _P, _P, *_SIZES, _P]),
    "monarch_attn_fwd_f32": (_I, [_P, _P, _P, _P, *_SIZES, _P]),
    "monarch_attn_fwd_host": (_I, [_I, _P, _P, _P, _P, *_SIZES, _P]),
    "monarch_attn_fwd_noalloc": (_I, [_P, _P, _P, _P, *_SIZES, _P]),
    "monarch_attn_fwd_video": (_I, [_I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                    _I, _P]),
    "monarch_attn_fwd_padded": (_I, [_I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                     _I, _P]),
    "monarch_attn_bwd": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, *_SIZES, _P]),
    "monarch_attn_dense_fwd": (_I, [_I, _P, _P, _P, _P, _P, *[_I] * 6, _P, _I, _P, _F, _P, _Z,
                                    _P]),
    "monarch_attn_dense_fwd_workspace_bytes": (_Z, [_I] * 6),
    "monarch_attn_dense_bwd": (_I, [_I, *[_P] * 9, *[_I] * 6, _P, _I, _P, _F, _P, _Z, _P]),
    "monarch_attn_dense_bwd_workspace_bytes": (_Z, [_I, _I, _I]),
    "monarch_attn_dense_decode": (_I, [_I, *[_P] * 7, *[_I] * 7, _P, _F, _P, _Z, _P]),
    "monarch_attn_dense_decode_workspace_bytes": (_Z, [_I] * 7),
    "monarch_attn_rotary": (_I, [_I, *[_P] * 4, *[_I] * 5, _P, _I, _P, _P, _P, _L, _P, _D, _I,
                                 _I, _P]),
    "monarch_attn_workspace_bytes": (_Z, [*_SIZES, _I]),
    "monarch_attn_release_workspace": (None, []),
    "monarch_attn_check": (_I, [_P]),
    "monarch_attn_strerror": (ctypes.c_char_p, [_I]),
    "monarch_attn_last_launches": (_I, []),
    "monarch_attn_version": (_I, []),
    "monarch_attn_selftest_timeout": (_I, [ctypes.c_ulonglong, _P]),
    "monarch_attn_timing_enable": (_I, [_I]),
    "monarch_attn_timing_read": (_I, [_I, ctypes.c_char_p, _I,
                                      ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_long)]),
}


class MonarchError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"monarch_attn status {status}: {text}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the shared library and bind every declared symbol (raises if absent)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m structured_sub_quadratic_b200._build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int):
    if status != MONARCH_OK:
        raise MonarchError(status, load_library().monarch_attn_strerror(status).decode())


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dims(q, b1, b2):
    if q.dim() != 4:
        raise ValueError("expected (B, H, N, d) tensors")
    B, H, N, d = q.shape
    if N != b1 * b2:
        raise ValueError(f"N={N} != b1*b2={b1 * b2}")
    return B, H, d


def monarch_attn_fwd(q, k, v, b1, b2, T, c1=1, c2=1, out=None, stream=None):
    """MonarchAttention forward on device tensors (B, H, N, d), N = b1*b2.

    bf16 tensors go to ``monarch_attn_fwd`` and fp32 to
    ``monarch_attn_fwd_f32``.  Returns ``out`` (allocated if not given).
    """
    lib = load_library()
    B, H, d = _dims(q, b1, b2)
    for t in (q, k, v):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors of one shape and dtype")
    if out is None:
        out = torch.empty_like(q)
    if q.dtype == torch.bfloat16:
        fn = lib.monarch_attn_fwd
    elif q.dtype == torch.float32:
        fn = lib.monarch_attn_fwd_f32
    else:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check(fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
              B, H, b1, b2, d, T, c1, c2, _stream_ptr(stream)))
    return out


def monarch_attn_fwd_noalloc(q, k, v, b1, b2, T, c1=1, c2=1, out=None, stream=None):
    """bf16 forward pass that allocates no device memory inside the library.

    For callers that cannot allocate when they call (a real-time frame loop
    that must not stall on cudaMalloc/cudaFree, or a host that reserves all
    device memory for its own pool).  It runs the kernels of
    ``monarch_attn_fwd`` and returns bit-identical results.  Scratch is a
    static 64 MiB device array shared by all calls on a device, committed at
    the first call on that device (make it at initialisation); calls that
    overlap on the GPU race on it, so keep them on one stream.  Pass ``out``
    to avoid the one allocation this wrapper would otherwise make through
    torch.
    """
    lib = load_library()
    B, H, d = _dims(q, b1, b2)
    for t in (q, k, v):
        if t.shape != q.shape or t.dtype != torch.bfloat16 or not t.is_cuda \
                or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors of one shape")
    if out is None:
        out = torch.empty_like(q)
    _check(lib.monarch_attn_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        out.data_ptr(), B, H, b1, b2, d, T, c1, c2,
                                        _stream_ptr(stream)))
    return out


def monarch_attn_fwd_padded(q, k, v, b1, b2, T, c1=1, c2=1, pad_front=True, out=None,
                            stream=None):
    """Forward pass on (B, H, n_real, d) tensors with n_real <= b1*b2: the
    sequence is padded to the b1*b2 grid with the pad tokens before the real
    ones (``pad_front``, pre-padding) or after them; the objective covers the
    real tokens only.  Returns ``out`` (B, H, n_real, d)."""
    lib = load_library()
    if q.dim() != 4:
        raise ValueError("expected (B, H, n_real, d) tensors")
    B, H, n_real, d = q.shape
    for t in (q, k, v):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors of one shape and dtype")
    dtype = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(q.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if out is None:
        out = torch.empty_like(q)
    _check(lib.monarch_attn_fwd_padded(dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       out.data_ptr(), B, H, n_real, b1, b2,
                                       1 if pad_front else 0, d, T, c1, c2, _stream_ptr(stream)))
    return out


def monarch_attn_bwd(q, k, v, dout, b1, b2, T=1, c1=1, c2=1, stream=None):
    """Gradients (dq, dk, dv) of sum(O * dout) for the T = 1 forward pass on
    device tensors (B, H, N, d), N = b1*b2, bf16 or fp32."""
    lib = load_library()
    B, H, d = _dims(q, b1, b2)
    for t in (q, k, v, dout):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, dout must be contiguous CUDA tensors of one shape and dtype")
    dtype = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(q.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    _check(lib.monarch_attn_bwd(dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, b1, b2, d, T,
                                c1, c2, _stream_ptr(stream)))
    return dq, dk, dv


def video_blocks(f, h, w, layout):
    """(b1, b2) of an aligned layout name such as "w,fh" (see LAYOUTS)."""
    size = {"f": f, "h": h, "w": w}
    rows, cols = layout.split(",")
    b1 = 1
    for a in rows:
        b1 *= size[a]
    b2 = 1
    for a in cols:
        b2 *= size[a]
    return b1, b2


def monarch_attn_fwd_video(q, k, v, f, h, w, layout, T, c1=1, c2=1, out=None, stream=None,
                           rotary=None):
    """Forward pass on a video latent (B, H, f*h*w, d) in raster token order,
    with the Monarch blocks aligned to ``layout`` (a key of LAYOUTS).

    ``rotary``: keyword arguments of ``monarch_attn_rotary`` (``axis_dims`` of
    the three axes f, h and w, and any of ``interleaved``, ``base`` and
    ``scaling``) that q and k are rotated with first, by their place in the
    latent; q and k are left as they are."""
    lib = load_library()
    if layout not in LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}; expected one of {sorted(LAYOUTS)}")
    if q.dim() != 4 or q.shape[2] != f * h * w:
        raise ValueError("expected (B, H, f*h*w, d) tensors")
    B, H, _, d = q.shape
    for t in (q, k, v):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors of one shape and dtype")
    dtype = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(q.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if rotary is not None:
        q, k = monarch_attn_rotary(q, k, grid=(f, h, w), stream=stream, **rotary)
    if out is None:
        out = torch.empty_like(q)
    _check(lib.monarch_attn_fwd_video(dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      out.data_ptr(), B, H, f, h, w, LAYOUTS[layout], d, T, c1,
                                      c2, _stream_ptr(stream)))
    return out


def monarch_attn_fwd_host(q, k, v, out, b1, b2, T, c1=1, c2=1, stream=None):
    """Forward pass on HOST tensors (pinned for full bandwidth); synchronous."""
    lib = load_library()
    B, H, d = _dims(q, b1, b2)
    for t in (q, k, v, out):
        if t.is_cuda or not t.is_contiguous() or t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("host tensors must be contiguous CPU tensors of one shape and dtype")
    dtype = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}[q.dtype]
    _check(lib.monarch_attn_fwd_host(dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     out.data_ptr(), B, H, b1, b2, d, T, c1, c2,
                                     _stream_ptr(stream)))
    return out


_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _elsewhere(t, stream):
    """Whether t's device or `stream` is not the current one (see _at)."""
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {t.device}")
    return stream is not None or t.get_device() != torch.cuda.current_device()


@contextlib.contextmanager
def _at(t, stream):
    """t's device current and, if given, `stream` too: what a call allocates
    inside belongs to the stream that uses it."""
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield


def _current(device_index):
    """The current stream's handle (torch.cuda.current_stream without its object)."""
    return torch._C._cuda_getCurrentRawStream(device_index)


def _dense_dtype(name, like, *tensors):
    """The dtype code of `like` after checking that each tensor shares its
    dtype and CUDA device and has contiguous channels."""
    dtype, kind, device = _DTYPES.get(like.dtype), like.dtype, like.get_device()
    if dtype is None:
        raise ValueError(f"unsupported dtype {like.dtype}")
    for t in (like, *tensors):
        if t.dtype != kind or t.get_device() != device or device < 0:
            raise ValueError(f"{name} must be CUDA tensors of one dtype on one device")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name} must have contiguous channels (last stride 1)")
    return dtype


def _int_tensor(name, t, like, shape):
    if t.dtype != torch.int32 or t.get_device() != like.get_device() or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {shape} on {like.device}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _stride_array(*strides):
    """Batch, head and token strides, tensor after tensor, for the C ABI."""
    flat = [x for s in strides for x in s[:3]]
    return (_L * len(flat))(*flat)


def _strides(*tensors):
    return _stride_array(*(t.stride() for t in tensors))


@functools.lru_cache(maxsize=256)
def _workspace_need(call, device_index, *sizes):
    """Bytes of workspace of a call (a function of the sizes and the device)."""
    return getattr(load_library(), f"monarch_attn_{call}_workspace_bytes")(*sizes)


def _like(t):
    """Uninitialised, t's shape, and t's strides unless its elements repeat
    (of rows that overlap, torch may make another dimension the innermost)."""
    if 0 not in t.stride():
        y = torch.empty_like(t)
        if y.stride(-1) == 1 or t.shape[-1] == 1:
            return y
    return t.new_empty(t.shape)


def _dense_dims(q, k, v, scale):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected (B, H, Nq, d) and (B, Hkv, Nk, d) tensors")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if k.shape != (B, Hkv, Nk, d) or v.shape != k.shape:
        raise ValueError("k and v must be (B, Hkv, Nk, d) with q's B and d")
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{H} query heads cannot share {Hkv} key/value heads")
    return B, H, Hkv, Nq, Nk, d, 1.0 / math.sqrt(d) if scale is None else scale


def monarch_attn_dense_fwd(q, k, v, causal=False, k_lens=None, scale=None, out=None,
                           stream=None):
    """Exact softmax attention: (out, lse) of q (B, H, Nq, d) over k and v
    (B, Hkv, Nk, d), H a multiple of Hkv, in any strides with contiguous
    channels.

    ``causal``: query i sees the keys up to i + Nk - Nq.  ``k_lens``: int32
    (B,) on the device, the keys of each sequence that count; what lies past
    them is never used.  A row that sees no key (or only keys that score -inf)
    gets out = 0, lse = -inf.
    ``scale`` defaults to 1/sqrt(d).  lse is fp32 (B, H, Nq), for
    ``monarch_attn_dense_bwd``.
    """
    lib = load_library()
    B, H, Hkv, Nq, Nk, d, scale = _dense_dims(q, k, v, scale)
    dtype = _dense_dtype("q, k, v and out", q, k, v, *(() if out is None else (out,)))
    if out is not None and out.shape != q.shape:
        raise ValueError("out must have q's shape")
    lens = None if k_lens is None else _int_tensor("k_lens", k_lens, q, (B,))
    if _elsewhere(q, stream):
        with _at(q, stream):
            return monarch_attn_dense_fwd(q, k, v, causal, k_lens, scale, out)
    if out is None:
        out = _like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    need = _workspace_need("dense_fwd", q.get_device(), dtype, B, H, Nq, Nk, d)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _check(lib.monarch_attn_dense_fwd(
        dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H,
        Hkv, Nq, Nk, d, _strides(q, k, v, out), bool(causal), lens, scale,
        ws.data_ptr() if need else None, need, _current(q.get_device())))
    return out, lse


def monarch_attn_dense_bwd(q, k, v, out, lse, dout, causal=False, k_lens=None, scale=None,
                           stream=None):
    """Gradients (dq, dk, dv) of sum(out * dout) for the exact attention of
    ``monarch_attn_dense_fwd``, whose out and lse it takes with the same other
    arguments.  The probabilities are recomputed tile by tile; a key/value
    head's gradient sums over the query heads that share it."""
    lib = load_library()
    B, H, Hkv, Nq, Nk, d, scale = _dense_dims(q, k, v, scale)
    dtype = _dense_dtype("q, k, v, out and dout", q, k, v, out, dout)
    if out.shape != q.shape or dout.shape != q.shape:
        raise ValueError("out and dout must have q's shape")
    if lse.dtype != torch.float32 or lse.shape != (B, H, Nq) or lse.device != q.device \
            or not lse.is_contiguous():
        raise ValueError("lse must be the contiguous fp32 (B, H, Nq) tensor of the forward pass")
    lens = None if k_lens is None else _int_tensor("k_lens", k_lens, q, (B,))
    if _elsewhere(q, stream):
        with _at(q, stream):
            return monarch_attn_dense_bwd(q, k, v, out, lse, dout, causal, k_lens, scale)
    dq, dk, dv = _like(q), _like(k), _like(v)
    need = lib.monarch_attn_dense_bwd_workspace_bytes(B, H, Nq)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(lib.monarch_attn_dense_bwd(
        dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
        dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Hkv, Nq, Nk, d,
        _strides(q, k, v, out, dout, dq, dk, dv), bool(causal), lens, scale, ws.data_ptr(), need,
        _current(q.get_device())))
    return dq, dk, dv


def monarch_attn_dense_decode(q, k_cache, v_cache, page_table, lens, scale=None, out=None,
                              stream=None):
    """Exact attention of one new token per sequence over a paged cache:
    (out, lse) of q (B, H, d).

    k_cache, v_cache: (pages, Hkv, page_size, d) in any strides with
    contiguous channels (a (pages, page_size, Hkv, d) cache is passed as its
    transpose(1, 2)).  page_table: int32 (B, max_pages); key j of sequence b is
    row j % page_size of page page_table[b, j // page_size].  lens: int32
    (B,), the keys of each sequence (0: out = 0, lse = -inf).  lse is fp32
    (B, H).  Pages and lengths are checked on the device: one that lies outside
    the cache stands for zero keys and values, or counts as the nearer end, and
    ``check`` then raises MONARCH_ERR_BAD_INDEX.
    """
    lib = load_library()
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("expected q (B, H, d) and caches (pages, Hkv, page_size, d)")
    B, H, d = q.shape
    pages, Hkv, page_size, dk = k_cache.shape
    if dk != d or Hkv < 1 or H % Hkv:
        raise ValueError("the caches must have q's d and a divisor of its heads")
    dtype = _dense_dtype("q, k_cache, v_cache and out", q, k_cache, v_cache,
                         *(() if out is None else (out,)))
    if out is not None and out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if page_table.dim() != 2:
        raise ValueError("page_table must be (B, max_pages)")
    max_pages = page_table.shape[1]
    table = _int_tensor("page_table", page_table, q, (B, max_pages))
    len_ptr = _int_tensor("lens", lens, q, (B,))
    if _elsewhere(q, stream):
        with _at(q, stream):
            return monarch_attn_dense_decode(q, k_cache, v_cache, page_table, lens, scale, out)
    if out is None:
        out = _like(q)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    need = _workspace_need("dense_decode", q.get_device(), dtype, B, H, Hkv, d, page_size,
                           max_pages)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    # (a query's and an output's third stride, of one token, is not used)
    strides = _strides(q, k_cache, v_cache, out)
    _check(lib.monarch_attn_dense_decode(
        dtype, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table, len_ptr,
        out.data_ptr(), lse.data_ptr(), B, H, Hkv, d, pages, page_size, max_pages, strides,
        1.0 / math.sqrt(d) if scale is None else scale, ws.data_ptr() if need else None, need,
        _current(q.get_device())))
    return out, lse


def rotary_frequencies(axis_dims, base=10000.0, scaling=None):
    """(angular frequency of each rotated pair, magnitude), axis after axis.

    Pair r of an axis with n channels turns base^(-2r/n) radians per position.
    ``scaling`` stretches them to a longer context by a factor s:
    ``("linear", s)`` divides every frequency by s; ``("ntk", s)`` raises the
    base by s^(n/(n-2)), which leaves the fastest pair and slows the last one
    s-fold; ``("parts", s, original, slow, fast)`` keeps the pairs that turn
    more than ``fast`` times over the original context, divides by s those
    that turn less than ``slow`` times, blends linearly between, and scales
    the rotated channels by 0.1 ln(s) + 1 (s >= 1).
    """
    kind = None if scaling is None else scaling[0]
    if kind is not None and (len(scaling) != {"linear": 2, "ntk": 2, "parts": 5}.get(kind)
                             or not scaling[1] > 0):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not base > 0:
        raise ValueError("base must be positive")
    freqs = []
    for n in axis_dims:
        b = base * scaling[1] ** (n / max(n - 2, 1)) if kind == "ntk" else base
        for r in range(n // 2):
            f = b ** (-2 * r / n)
            if kind == "linear":
                f /= scaling[1]
            elif kind == "parts":
                _, s, original, slow, fast = scaling
                if not fast > slow or s < 1:
                    raise ValueError("parts scaling needs fast > slow and a factor >= 1")
                keep = min(1.0, max(0.0, (original * f / (2 * math.pi) - slow) / (fast - slow)))
                f *= keep + (1 - keep) / s
            freqs.append(f)
    return freqs, 0.1 * math.log(scaling[1]) + 1 if kind == "parts" else 1.0


@functools.lru_cache(maxsize=64)
def _rotary_args(axis_dims, base, scaling):
    """ctypes forms of axis_dims and the frequencies, and the rotated channels
    (a function of the arguments alone)."""
    if not 1 <= len(axis_dims) <= 4 or any(n < 2 or n % 2 for n in axis_dims):
        raise ValueError("axis_dims must be one to four even sizes")
    freqs, magnitude = rotary_frequencies(axis_dims, base, scaling)
    return ((_I * len(axis_dims))(*axis_dims), (_D * len(freqs))(*freqs), magnitude,
            sum(axis_dims))


def monarch_attn_rotary(q, k=None, positions=None, *, axis_dims=None, grid=None,
                        interleaved=False, base=10000.0, scaling=None, inverse=False, q_out=None,
                        k_out=None, stream=None):
    """Rotary positions: (rotated q, rotated k) of q (B, H, N, d) and k (B,
    Hkv, N, d) (k may be None), in any strides with contiguous channels.

    The first sum(axis_dims) channels are cut into one section per position
    axis (default: all d, one axis); the pairs of a section are neighbours if
    ``interleaved``, else the same place of its two halves; the other channels
    are copied.  Positions: ``grid``, one size per axis with product N (token
    n is that place in raster order: (f, h, w) for a video latent), or
    ``positions``, int32 (N,), (axes, N) or (B, axes, N) on the device.
    Frequencies: see ``rotary_frequencies``.  ``inverse`` turns the other way:
    the gradient with respect to q and k of a gradient with respect to the
    outputs.  ``q_out`` and ``k_out`` may be q and k (in place).
    """
    lib = load_library()
    if q.dim() != 4 or (k is not None and (k.dim() != 4 or k.shape[0] != q.shape[0]
                                           or k.shape[2:] != q.shape[2:])):
        raise ValueError("expected q (B, H, N, d) and k (B, Hkv, N, d)")
    B, H, N, d = q.shape
    axis_dims = (d,) if axis_dims is None else tuple(axis_dims)
    dims, freqs, magnitude, rotated = _rotary_args(
        axis_dims, base, None if scaling is None else tuple(scaling))
    if rotated > d:
        raise ValueError(f"axis_dims rotate {rotated} of {d} channels")
    given = [t for t in (k, q_out, k_out) if t is not None]
    dtype = _dense_dtype("q, k and the outputs", q, *given)
    if (q_out is not None and q_out.shape != q.shape) or \
            (k_out is not None and (k is None or k_out.shape != k.shape)):
        raise ValueError("q_out and k_out must have the shapes of q and k")
    if (grid is None) == (positions is None):
        raise ValueError("one of grid and positions is needed")
    where, step, sizes = None, 0, None
    if grid is not None:
        if len(grid) != len(axis_dims) or math.prod(grid) != N:
            raise ValueError("grid must have one size per axis, with product N")
        sizes = (_I * len(grid))(*grid)
    else:
        shape = (len(axis_dims), N)
        if positions.dim() == 1 and len(axis_dims) == 1:
            shape = (N,)
        elif positions.dim() == 3:
            shape, step = (B, *shape), len(axis_dims) * N
        where = _int_tensor("positions", positions, q, shape)
    if _elsewhere(q, stream):
        with _at(q, stream):
            return monarch_attn_rotary(q, k, positions, axis_dims=axis_dims, grid=grid,
                                       interleaved=interleaved, base=base, scaling=scaling,
                                       inverse=inverse, q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = _like(q)
    if k is None:
        heads, kp, kop, strides = 0, None, None, _strides(q, q_out, q, q_out)
    else:
        if k_out is None:
            k_out = _like(k)
        heads, kp, kop = k.shape[1], k.data_ptr(), k_out.data_ptr()
        strides = _strides(q, q_out, k, k_out)
    _check(lib.monarch_attn_rotary(
        dtype, q.data_ptr(), kp, q_out.data_ptr(), kop, B, H, heads, N, d, strides,
        len(axis_dims), dims, sizes, where, step, freqs, magnitude, bool(interleaved),
        bool(inverse), _current(q.get_device())))
    return q_out, k_out


def workspace_bytes(B, H, b1, b2, d, T, c1=1, c2=1, dtype=torch.bfloat16):
    code = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32
    return load_library().monarch_attn_workspace_bytes(B, H, b1, b2, d, T, c1, c2, code)


def release_workspace():
    load_library().monarch_attn_release_workspace()


def check(stream=None):
    _check(load_library().monarch_attn_check(_stream_ptr(stream)))


def last_launches() -> int:
    return load_library().monarch_attn_last_launches()


def timing_enable(enable: bool) -> bool:
    """Turn per-kernel CUDA-event timing on or off; returns the old setting."""
    return bool(load_library().monarch_attn_timing_enable(1 if enable else 0))


def timing_read(max_kernels: int = 32):
    """{kernel name: (total ms, launches)} since the previous read."""
    lib = load_library()
    name_len = 64
    names = ctypes.create_string_buffer(max_kernels * name_len)
    ms = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_long * max_kernels)()
    n = lib.monarch_attn_timing_read(max_kernels, names, name_len, ms, cnt)
    if n < 0:
        _check(n)
    out = {}
    for s in range(min(n, max_kernels)):
        raw = names.raw[s * name_len:(s + 1) * name_len]
        out[raw.split(b"\0", 1)[0].decode()] = (ms[s], cnt[s])
    return out


def selftest_timeout(limit_ns: int, stream=None):
    """Launch the bounded-wait self-test (see the header); check() then reports it."""
    _check(load_library().monarch_attn_selftest_timeout(limit_ns, _stream_ptr(stream)))

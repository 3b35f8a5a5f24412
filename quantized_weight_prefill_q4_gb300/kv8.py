"""ctypes binding of the 8-bit paged KV cache (include/apr_kv8.h), same names.

Like :mod:`.capi` it only marshals: tensors become device pointers, sizes are
checked against the tensors so that no call can address past an allocation,
and a nonzero status raises :class:`~.capi.AprError`. The library works on the
calling thread's current device: tensors on another than the cache's, and a
cache on another than that, are refused.
"""

from __future__ import annotations

import ctypes

import torch

from . import capi

APR_T_F32 = 0
APR_T_F16 = 1
APR_T_BF16 = 30

# Every symbol include/apr_kv8.h declares.
KV8_EXPORTS = ("apr_kv8_append", "apr_kv8_read", "apr_kv8_attention", "apr_kv8_prefill_attention", "apr_kv8_evict")

_I8, _I32, _F32, _Tensor = torch.int8, torch.int32, torch.float32, torch.Tensor
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_TYPES = {torch.float32: APR_T_F32, torch.float16: APR_T_F16, torch.bfloat16: APR_T_BF16}


class _Cache(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_void_p),
        ("V", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("page_tokens", ctypes.c_int),
        ("head_dim", ctypes.c_int),
    ]


class _Rows(ctypes.Structure):
    _fields_ = [
        ("page_table", ctypes.c_void_p),
        ("table_ld", ctypes.c_int),
        ("lens", ctypes.c_void_p),
        ("row_start", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int),
        ("num_rows", ctypes.c_int),
        ("max_rows", ctypes.c_int),
        ("max_len", ctypes.c_int),
    ]


def _bind():
    lib = capi.library()
    vp, ci, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    cache, rows = ctypes.POINTER(_Cache), ctypes.POINTER(_Rows)
    sig = {
        "apr_kv8_append": [cache, rows, ci, vp, vp, ll, vp],
        "apr_kv8_read": [cache, rows, ci, vp, vp, ll, vp],
        "apr_kv8_attention": [cache, rows, ci, vp, ll, vp, ll, ci, ctypes.c_float, vp, ll, ci, vp],
        "apr_kv8_prefill_attention": [cache, rows, ci, vp, ll, vp, ll, ci, ctypes.c_float, vp],
        "apr_kv8_evict": [cache, rows, vp, ll, ci, ci, vp, vp, vp, vp, ll, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    return lib


_lib = _bind()


def _array(x, name, dtype, dims, device=None):
    """A contiguous CUDA tensor of the type and number of dimensions on the
    device (an index), checked."""
    if isinstance(x, _Tensor) and x.get_device() == device and x.dtype is dtype and x.ndim == dims and x.is_contiguous():
        return x  # (a tensor that is not on a GPU has no device index)
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a CUDA tensor, got {type(x).__name__}")
    if not x.is_cuda:
        raise ValueError(f"{name}: tensor is on {x.device}, the library takes device memory")
    if x.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.get_device() != device:
        raise ValueError(f"{name}: tensor is on device {x.get_device()}, the cache on {device}")
    raise ValueError(f"{name}: expected a contiguous tensor of {dims} dimensions, got shape {tuple(x.shape)}")


def _stream(stream, device_index):
    """The raw stream: the given one, or torch's current one. The library takes
    scratch and status word, and launches, on the current device."""
    device = _current_device()
    if device != device_index:
        raise ValueError(f"the cache is on device {device_index}, the current device is {device}")
    return _raw_stream(device_index) if stream is None else capi._stream(stream)


class Kv8Cache:
    """The cache's arrays: codes K and V int8 [pages][kv_heads][page_tokens][head_dim],
    scales k_scale and v_scale float32 [pages][kv_heads], all contiguous."""

    __slots__ = ("_arrays", "kv_heads", "page_tokens", "head_dim", "device_index", "_c")
    # (read-only: the C structure holds their addresses)
    K = property(lambda self: self._arrays[0])
    V = property(lambda self: self._arrays[1])
    k_scale = property(lambda self: self._arrays[2])
    v_scale = property(lambda self: self._arrays[3])

    def __init__(self, K, V, k_scale, v_scale):
        device = K.get_device() if isinstance(K, _Tensor) else None
        shape = _array(K, "K", _I8, 4, device).shape
        scales = shape[:2]
        if (_array(V, "V", _I8, 4, device).shape != shape or _array(k_scale, "k_scale", _F32, 2, device).shape != scales
                or _array(v_scale, "v_scale", _F32, 2, device).shape != scales):
            raise ValueError("Kv8Cache: V, k_scale and v_scale must match K's pages, heads, tokens and head_dim")
        self._arrays = (K, V, k_scale, v_scale)
        pages, self.kv_heads, self.page_tokens, self.head_dim = shape
        self.device_index = device
        self._c = _Cache(K.data_ptr(), V.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, self.kv_heads,
                         self.page_tokens, self.head_dim)

    @classmethod
    def allocate(cls, num_pages, num_kv_heads, head_dim, page_tokens=64, device="cuda"):
        """A cache of num_pages pages (zeros)."""
        codes = (num_pages, num_kv_heads, page_tokens, head_dim)
        if torch.device(device).type != "cuda":
            raise ValueError(f"Kv8Cache: the library takes device memory, got {device}")
        return cls(torch.zeros(codes, dtype=torch.int8, device=device),
                   torch.zeros(codes, dtype=torch.int8, device=device),
                   torch.zeros(codes[:2], dtype=torch.float32, device=device),
                   torch.zeros(codes[:2], dtype=torch.float32, device=device))


def _rows(cache, page_table, lens, row_start, num_rows, max_rows, max_len):
    device = cache.device_index
    seqs, width = _array(page_table, "page_table", _I32, 2, device).shape
    if _array(lens, "lens", _I32, 1, device).numel() != seqs:
        raise ValueError(f"page_table has {seqs} rows, lens {lens.numel()} entries")
    start = None
    if row_start is not None:
        if _array(row_start, "row_start", _I32, 1, device).numel() != seqs + 1:
            raise ValueError(f"row_start: expected {seqs + 1} entries, got {row_start.numel()}")
        start = row_start.data_ptr()
    return _Rows(page_table.data_ptr(), width, lens.data_ptr(), start, seqs, num_rows, max_rows, max_len)


def _matrix(x, name, width, device=None, like=None):
    """(pointer, rows, elements from row to row) of rows of `width` elements: a
    2-D tensor, or a 3-D one of [rows][heads][head_dim], whose rows are dense."""
    if not (isinstance(x, _Tensor) and x.get_device() == device and x.dtype in _TYPES):
        if not (isinstance(x, _Tensor) and x.is_cuda and x.dtype in _TYPES):
            raise ValueError(f"{name}: expected a float32, float16 or bfloat16 CUDA tensor")
        raise ValueError(f"{name}: tensor is on device {x.get_device()}, the cache on {device}")
    shape, stride = x.shape, x.stride()
    if len(shape) == 2:
        dense = shape[1] == width and stride[1] == 1
    else:
        dense = (len(shape) == 3 and shape[1] * shape[2] == width and stride[2] == 1
                 and (shape[1] == 1 or stride[1] == shape[2]))
    if not dense:
        raise ValueError(f"{name}: expected rows of {width} consecutive elements, got shape {tuple(shape)}, "
                         f"strides {tuple(stride)}")
    rows = shape[0]
    if like is not None and (x.dtype is not like.dtype or rows != like.shape[0]):
        raise ValueError(f"{name}: expected {like.shape[0]} rows of {like.dtype}, got {rows} of {x.dtype}")
    return x.data_ptr(), rows, stride[0] if rows > 1 else width


def _k_and_v(cache, k, v):
    width = cache.kv_heads * cache.head_dim
    kp, rows, ld = _matrix(k, "k", width, cache.device_index)
    vp, _, vld = _matrix(v, "v", width, cache.device_index, like=k)
    if vld != ld and rows > 1:
        raise ValueError(f"k and v must have the same row stride, got {ld} and {vld}")
    return kp, vp, rows, ld


def apr_kv8_append(cache, page_table, lens, k, v, *, row_start=None, max_rows=0, stream=None) -> int:
    """Quantises the packed rows k and v ([rows][kv_heads * head_dim], strided
    rows allowed) into the cache, as the last positions of their sequences:
    lens counts them already. row_start None: one row a sequence."""
    kp, vp, n, ld = _k_and_v(cache, k, v)
    rows = _rows(cache, page_table, lens, row_start, n, max_rows, 0)
    return capi._check(_lib.apr_kv8_append(cache._c, rows, _TYPES[k.dtype], kp, vp, ld, _stream(stream, cache.device_index)))


def apr_kv8_read(cache, page_table, lens, k, v, *, row_start=None, max_rows=0, stream=None) -> int:
    """Writes the values of each sequence's last rows to k and v (their types
    and strides as for the append)."""
    kp, vp, n, ld = _k_and_v(cache, k, v)
    rows = _rows(cache, page_table, lens, row_start, n, max_rows, 0)
    return capi._check(_lib.apr_kv8_read(cache._c, rows, _TYPES[k.dtype], kp, vp, ld, _stream(stream, cache.device_index)))


def apr_kv8_attention(cache, page_table, lens, q, out, num_heads, *, row_start=None, max_rows=0, max_len=0, scale=0.0,
                      weights=None, accumulate=False, stream=None) -> int:
    """out[row][head] = the causal attention of each sequence's last rows q
    over its cache, which holds their own k and v; out has q's type. weights
    ([sequences][kv_heads][>= max_len] float32) receives, or with accumulate
    adds, the weight of each position. max_len bounds lens (0: the table)."""
    width = num_heads * cache.head_dim
    qp, n, ldq = _matrix(q, "q", width, cache.device_index)
    op, _, ldo = _matrix(out, "out", width, cache.device_index, like=q)
    rows = _rows(cache, page_table, lens, row_start, n, max_rows, max_len)
    wp, wld = None, 0
    if weights is not None:
        seqs, heads, wld = _array(weights, "weights", _F32, 3, cache.device_index).shape
        if seqs != rows.num_seqs or heads != cache.kv_heads:
            raise ValueError(f"weights: expected [{rows.num_seqs}][{cache.kv_heads}][...], got {tuple(weights.shape)}")
        wp = weights.data_ptr()
    return capi._check(_lib.apr_kv8_attention(cache._c, rows, _TYPES[q.dtype], qp, ldq, op, ldo, num_heads, scale, wp,
                                              wld, int(accumulate), _stream(stream, cache.device_index)))


def apr_kv8_prefill_attention(cache, page_table, lens, q, out, num_heads, *, row_start=None, max_rows=0, max_len=0,
                              scale=0.0, stream=None) -> int:
    """apr_kv8_attention without weights for chunks of rows: any number of packed rows q of each sequence."""
    width = num_heads * cache.head_dim
    qp, n, ldq = _matrix(q, "q", width, cache.device_index)
    op, _, ldo = _matrix(out, "out", width, cache.device_index, like=q)
    rows = _rows(cache, page_table, lens, row_start, n, max_rows, max_len)
    return capi._check(_lib.apr_kv8_prefill_attention(cache._c, rows, _TYPES[q.dtype], qp, ldq, op, ldo, num_heads, scale,
                                                      _stream(stream, cache.device_index)))


def apr_kv8_evict(cache, page_table, lens, weights, budget, recent, fresh_pages, table_out, lens_out, weights_out, kept,
                  *, max_len=0, stream=None) -> int:
    """Cuts every sequence of more than `budget` positions to its `recent` last
    and the others of the largest weights, moved into fresh_pages
    ([sequences][ceil(budget / page_tokens)]); table_out, lens_out, weights_out
    ([sequences][kv_heads][>= budget]) and kept ([sequences][kv_heads][budget])
    say what the sequences are afterwards."""
    rows = _rows(cache, page_table, lens, None, 0, 0, max_len)
    n, heads, device = rows.num_seqs, cache.kv_heads, cache.device_index

    def check(x, name, dtype, shape):
        if tuple(_array(x, name, dtype, len(shape), device).shape) != shape:
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(x.shape)}")
        return x.data_ptr()

    def check_weights(x, name):
        shape = _array(x, name, _F32, 3, device).shape
        if shape[0] != n or shape[1] != heads:
            raise ValueError(f"{name}: expected [{n}][{heads}][...], got {tuple(shape)}")
        return x.data_ptr(), shape[2]

    w, w_ld = check_weights(weights, "weights")
    wo, wo_ld = check_weights(weights_out, "weights_out")
    fresh = check(fresh_pages, "fresh_pages", _I32, (n, -(-budget // cache.page_tokens)))
    to = check(table_out, "table_out", _I32, (n, rows.table_ld))
    lo = check(lens_out, "lens_out", _I32, (n,))
    ko = check(kept, "kept", _I32, (n, heads, budget))
    return capi._check(_lib.apr_kv8_evict(cache._c, rows, w, w_ld, budget, recent, fresh, to, lo, wo, wo_ld, ko,
                                          _stream(stream, cache.device_index)))

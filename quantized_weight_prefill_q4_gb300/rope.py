"""ctypes binding of the rotations by position (include/apr_rope.h), same names.

Marshalling and checks as in :mod:`.kv8`: tensors become device pointers, sizes
are checked against the tensors so that no call can address past an allocation,
and a nonzero status raises :class:`~.capi.AprError`. Tensors of another device
than the table's, and a table of another than the current one, are refused.
"""

from __future__ import annotations

import ctypes

import torch

from . import capi, kv8
from .kv8 import _TYPES, _Tensor, _array, _k_and_v, _matrix, _rows, _stream

# Every symbol include/apr_rope.h declares.
ROPE_EXPORTS = ("apr_rope_table", "apr_rope_rows", "apr_rope_kv8_append")

_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


class _Rope(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("num_positions", ctypes.c_int),
        ("rot_dim", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("pair_axis", ctypes.c_void_p),
        ("num_axes", ctypes.c_int),
        ("positions", ctypes.c_void_p),
        ("positions_ld", ctypes.c_int),
    ]


def _bind():
    lib = capi.library()
    vp, ci, ll, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    cache, rows, rope = ctypes.POINTER(kv8._Cache), ctypes.POINTER(kv8._Rows), ctypes.POINTER(_Rope)
    sig = {
        "apr_rope_table": [vp, ci, ll, ll, ctypes.c_double, vp, vp],
        "apr_rope_rows": [rope, ci, vp, ll, vp, ll, ci, ci, ci, vp, cf, vp],
        "apr_rope_kv8_append": [cache, rows, rope, ci, vp, vp, ll, vp, vp, ll, vp, ll, ci, vp, cf, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    return lib


_lib = _bind()


class Rope:
    """What turns a head's pairs: table float32 [positions][rot_dim / 2][2] (cosine, sine; see apr_rope_table), the
    order of the dims (pair i is dims i and i + rot_dim / 2, or interleaved 2 i and 2 i + 1) and, where positions have
    several axes, pair_axis uint8 [rot_dim / 2], the axis that turns each pair."""

    __slots__ = ("_arrays", "device_index", "rot_dim", "interleaved")
    table = property(lambda self: self._arrays[0])
    pair_axis = property(lambda self: self._arrays[1])

    def __init__(self, table, *, interleaved=False, pair_axis=None):
        device = table.get_device() if isinstance(table, _Tensor) else None
        shape = _array(table, "table", _F32, 3, device).shape
        if shape[2] != 2:
            raise ValueError(f"table: expected [positions][pairs][2], got {tuple(shape)}")
        if pair_axis is not None and _array(pair_axis, "pair_axis", _U8, 1, device).numel() != shape[1]:
            raise ValueError(f"pair_axis: expected {shape[1]} entries, got {pair_axis.numel()}")
        self._arrays = (table, pair_axis)
        self.device_index, self.rot_dim, self.interleaved = device, 2 * shape[1], bool(interleaved)

    def _with(self, positions, rows):
        table, pair_axis = self._arrays
        axes, at, ld = 1, None, 0
        if positions is not None:
            if isinstance(positions, _Tensor) and positions.ndim == 2:
                axes = _array(positions, "positions", _I32, 2, self.device_index).shape[0]
            else:
                _array(positions, "positions", _I32, 1, self.device_index)
            if positions.shape[-1] != rows:
                raise ValueError(f"positions: expected {rows} on each axis, got {tuple(positions.shape)}")
            at, ld = positions.data_ptr(), rows
        return _Rope(table.data_ptr(), table.shape[0], self.rot_dim, int(self.interleaved),
                     None if pair_axis is None else pair_axis.data_ptr(), axes, at, ld)


def _norm(x, name, dim, device):
    if x is None:
        return None
    if _array(x, name, _F32, 1, device).numel() != dim:
        raise ValueError(f"{name}: expected {dim} weights, got {x.numel()}")
    return x.data_ptr()


def apr_rope_table(inv_freq, table, *, first=0, scale=1.0, stream=None) -> int:
    """table[p][i] = scale * (cos, sin) of (first + p) * inv_freq[i]: float32 [positions][pairs][2]."""
    device = table.get_device() if isinstance(table, _Tensor) else None
    positions, pairs, two = _array(table, "table", _F32, 3, device).shape
    if two != 2 or _array(inv_freq, "inv_freq", _F32, 1, device).numel() != pairs:
        raise ValueError(f"table: expected [positions][{inv_freq.numel()}][2], got {tuple(table.shape)}")
    return capi._check(_lib.apr_rope_table(inv_freq.data_ptr(), pairs, first, positions, scale, table.data_ptr(),
                                           _stream(stream, device)))


def apr_rope_rows(rope, positions, x, out, num_heads, head_dim, *, norm=None, eps=0.0, stream=None) -> int:
    """out = rows x ([rows][num_heads * head_dim], strided rows allowed) with each head normed (weights norm, float32
    [head_dim]) and rotated by its row's positions (int32 [rows], or [axes][rows]). out may be x."""
    width, device = num_heads * head_dim, rope.device_index
    xp, n, ldx = _matrix(x, "x", width, device)
    op, _, ldo = _matrix(out, "out", width, device, like=x)
    if positions is None:
        raise ValueError("positions: expected int32 [rows], or [axes][rows]")
    return capi._check(_lib.apr_rope_rows(rope._with(positions, n), _TYPES[x.dtype], xp, ldx, op, ldo, n, num_heads,
                                          head_dim, _norm(norm, "norm", head_dim, device), eps, _stream(stream, device)))


def apr_rope_kv8_append(cache, page_table, lens, rope, k, v, *, positions=None, k_norm=None, q=None, q_out=None,
                        num_heads=0, q_norm=None, eps=0.0, row_start=None, max_rows=0, stream=None) -> int:
    """apr_kv8_append of the normed and rotated rows k and of v; rows q ([rows][num_heads * head_dim]), if given, are
    normed and rotated into q_out (which may be q). positions None: each row's position in its sequence."""
    kp, vp, n, ld = _k_and_v(cache, k, v)
    device = cache.device_index
    if rope.device_index != device:
        raise ValueError(f"rope: table is on device {rope.device_index}, the cache on {device}")
    rows = _rows(cache, page_table, lens, row_start, n, max_rows, 0)
    qp = op = None
    ldq = ldo = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out: expected both or neither")
    if q is not None:
        qp, _, ldq = _matrix(q, "q", num_heads * cache.head_dim, device, like=k)
        op, _, ldo = _matrix(q_out, "q_out", num_heads * cache.head_dim, device, like=k)
    return capi._check(_lib.apr_rope_kv8_append(
        cache._c, rows, rope._with(positions, n), _TYPES[k.dtype], kp, vp, ld, _norm(k_norm, "k_norm", cache.head_dim, device),
        qp, ldq, op, ldo, num_heads, _norm(q_norm, "q_norm", cache.head_dim, device), eps, _stream(stream, device)))

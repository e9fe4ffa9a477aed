"""Python names of attention to states of another length (sfa_cross_*) and of a
decode step behind a shared prefix (sfa_prefix_decode).

Calls take the current stream of their tensors' device, only enqueue work, keep
nothing, and may be captured into a CUDA graph (prefix_decode with a RoPE table
made before).  include/sfa.h says what each computes.

As with the paged cache, a call whose arguments are in order and that gives no
outputs or workspace is made by csrc/cross_py.cpp; any other, or all if that could not
be built, here."""
from __future__ import annotations

import ctypes as C
import functools
import struct

import torch

from ._lib import _lib, check
from .api import _ROPE_CACHE
from .kv4 import _F32, _I32, _U8, _call, _code, _dense, _entry, _ints, _refuse, _rope, _rows

_cross_desc = struct.Struct("7i4x9q2P").pack  # the bytes of _lib.CrossDesc
_prefix_desc = struct.Struct("7i4x5qPi4x").pack  # and of _lib.PrefixDesc


@functools.cache
def _native():
    """The native calls, or None where they could not be built."""
    try:
        from . import _cross
    except ImportError:
        return None
    L = _lib()
    _cross.bind(*(C.cast(L[name], C.c_void_p).value for name in ("sfa_cross_workspace_size", "sfa_cross_forward", "sfa_cross_backward",
                                                                  "sfa_prefix_workspace_size", "sfa_prefix_decode")))
    return _cross


def _view(t, name, like=None, shape=None):
    """Strides of t [B, H, T, 64], whose rows are dense, of like's type and device."""
    if not t.is_cuda or t.dim() != 4 or t.shape[3] != 64 or (shape is not None and t.shape != shape):
        _refuse(name, t, t.dtype, shape or (None, None, None, 64))
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must be {like.dtype} on device {like.get_device()}, got {t.dtype} on {t.get_device()}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{name}: the 64 numbers of a row must be contiguous")
    for n, step in zip(t.shape, s[:3]):
        if n > 1 and (step < 64 or step * t.element_size() % 16):
            raise ValueError(f"{name}: rows must not overlap and must start at multiples of 16 bytes")
    return s[:3]


def _lengths(t, name, B, index):
    return 0 if t is None else _ints(index, B, t, name)


def _describe(q, k, v, q_len, kv_len):
    """Device index, shape of q's tensors and of k's, and the descriptor of a call."""
    qs = _view(q, "q")
    ks = _view(k, "k", q)
    vs = _view(v, "v", q, k.shape)
    at = q.get_device()
    B, Hq, Tq, _ = q.shape
    if k.shape[0] != B:
        raise ValueError(f"k must have q's {B} sequences, got {k.shape[0]}")
    d = _cross_desc(B, Tq, k.shape[2], Hq, k.shape[1], 64, _code(q.dtype), *qs, *ks, *vs, _lengths(q_len, "q_len", B, at),
                    _lengths(kv_len, "kv_len", B, at))
    return at, (B, Hq, Tq, 64), tuple(k.shape), d


def _workspace(name, at, ws, d, *args):
    """Address and bytes of a workspace: the caller's if it is large enough, else a new one, kept by the caller of this."""
    n = C.c_size_t(0)
    rc = _entry(name)(d, *args, C.byref(n))
    if rc:
        check(rc, name)
    n = n.value
    if n == 0:
        return None, 0, None
    if ws is None or ws.numel() * ws.element_size() < n:
        ws = torch.empty((n,), dtype=_U8, device=torch.device("cuda", at))
    elif ws.get_device() != at or not ws.is_contiguous():
        _refuse("ws", ws, ws.dtype, tuple(ws.shape), at)
    return ws.data_ptr(), n, ws


def _output(t, name, at, shape, dtype):
    """t, or a new tensor, and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=torch.device("cuda", at))
        return t, t.data_ptr()
    return t, _dense(at, shape, dtype, t, name)


def cross_workspace_size(q, k, v, *, backward: bool = False) -> int:
    """Scratch bytes of cross_forward or cross_backward for these shapes (of any lengths)."""
    d = _describe(q, k, v, None, None)[3]
    n = C.c_size_t(0)
    check(_entry("sfa_cross_workspace_size")(d, int(backward), C.byref(n)), "sfa_cross_workspace_size")
    return n.value


def cross_forward(q, k, v, *, q_len=None, kv_len=None, o=None, lse=None, ws=None):
    """Attention of q [B, Hq, Tq, 64] over all rows of k and v [B, Hkv, Tk, 64]
    (sfa_cross_forward; bf16 or fp32, strided views of other layouts too).  q_len
    and kv_len: int32 [B], how many rows of each sequence count (None: all); a
    query behind its length or without a key gives zeros and lse = -inf.  A single
    token a sequence is Tq = 1.  ws: scratch of cross_workspace_size bytes or more (one
    that is smaller is not used).  Returns o [B, Hq, Tq, 64] and lse fp32 [B, Hq, Tq]."""
    fast = _native()
    if fast is not None and o is None and lse is None and ws is None:
        r = fast.forward(q, k, v, q_len, kv_len)
        if type(r) is tuple:
            return r
        if r is not None:
            check(r, "sfa_cross_forward")
    at, qshape, _, d = _describe(q, k, v, q_len, kv_len)
    o, op = _output(o, "o", at, qshape, q.dtype)
    lse, lp = _output(lse, "lse", at, qshape[:3], _F32)
    wp, n, keep = _workspace("sfa_cross_workspace_size", at, ws, d, 0)
    _call("sfa_cross_forward", at, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), op, lp, wp, n)
    return o, lse


def cross_backward(q, k, v, o, lse, do, *, q_len=None, kv_len=None, dq=None, dk=None, dv=None, ws=None):
    """Gradients of sum(o * do) for cross_forward's q, k, v, from its o and lse
    (sfa_cross_backward): dq [B, Hq, Tq, 64], dk and dv [B, Hkv, Tk, 64], contiguous,
    zeros behind the lengths.  The same inputs give the same bits.  ws: scratch of
    cross_workspace_size(q, k, v, backward=True) bytes or more."""
    fast = _native()
    if fast is not None and dq is None and dk is None and dv is None and ws is None:
        r = fast.backward(q, k, v, o, lse, do, q_len, kv_len)
        if type(r) is tuple:
            return r
        if r is not None:
            check(r, "sfa_cross_backward")
    at, qshape, kshape, d = _describe(q, k, v, q_len, kv_len)
    inputs = _dense(at, qshape, q.dtype, o, "o"), _dense(at, qshape[:3], _F32, lse, "lse"), _dense(at, qshape, q.dtype, do, "do")
    dq, qp = _output(dq, "dq", at, qshape, q.dtype)
    dk, kp = _output(dk, "dk", at, kshape, q.dtype)
    dv, vp = _output(dv, "dv", at, kshape, q.dtype)
    wp, n, keep = _workspace("sfa_cross_workspace_size", at, ws, d, 1)
    _call("sfa_cross_backward", at, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), *inputs, qp, kp, vp, wp, n)
    return dq, dk, dv


def _heads(t, name, index, dtype, Hkv):
    """P and the stride between the heads of t [Hkv, P, 64], each of which is dense."""
    if not t.is_cuda or t.get_device() != index or t.dtype is not dtype or t.dim() != 3 or t.shape[0] != Hkv or t.shape[2] != 64:
        _refuse(name, t, dtype, (Hkv, None, 64), index)
    P = t.shape[1]
    s = t.stride()
    if P and (s[2] != 1 or (P > 1 and s[1] != 64) or (Hkv > 1 and (s[0] < 64 * P or s[0] * t.element_size() % 16))):
        raise ValueError(f"{name}: the rows of a head must be contiguous, heads must not overlap and must start at multiples of 16 bytes")
    return P, s[0]


def prefix_workspace_size(q, prefix_k, k_cache) -> int:
    """Scratch bytes of prefix_decode for these shapes."""
    if not k_cache.is_cuda or k_cache.dim() != 4 or not k_cache.is_contiguous() or k_cache.shape[3] != 64:
        _refuse("k_cache", k_cache, k_cache.dtype, (None, None, None, 64))
    B, Hkv, T, _ = k_cache.shape
    dtype, at = k_cache.dtype, k_cache.get_device()
    n, Hq, qs = _rows(q, "q", 0, at)
    if n != B or q.dtype is not dtype:
        raise ValueError(f"q must have the caches' {B} rows and type {dtype}, got {n} and {q.dtype}")
    P, ps = _heads(prefix_k, "prefix_k", at, dtype, Hkv)
    n = C.c_size_t(0)
    d = _prefix_desc(B, P, T, Hq, Hkv, 64, _code(dtype), qs, 64 * Hkv, 64 * Hkv, ps, ps, 0, 0)
    check(_entry("sfa_prefix_workspace_size")(d, C.byref(n)), "sfa_prefix_workspace_size")
    return n.value


def prefix_decode(q, k_new, v_new, prefix_k, prefix_v, k_cache, v_cache, pos, *, rope_theta: float = 1e4, rope=None,
                  o=None, lse=None, ws=None):
    """One decode step of a batch whose sequences all begin with the same P rows
    (sfa_prefix_decode): q [B, Hq, 64], k_new and v_new [B, Hkv, 64] (rows may be
    slices of wider ones; both None where the caches hold the step's rows already),
    prefix_k and prefix_v [Hkv, P, 64] (keys rotated: rope_keys), k_cache and v_cache
    [B, Hkv, T, 64], pos int32 [B], the row of each cache that the step stands at, at
    position P + pos.  The new key is rotated there and written with the value; then
    the query attends the prefix, read once for the whole batch, and rows 0..pos of
    its cache.  rope: a table of rope_table for P + T positions or more, else that of
    rope_theta (0: no rotation; prefix and caches then hold unrotated keys).  ws: scratch
    of prefix_workspace_size bytes or more.  Returns o [B, Hq, 64] and lse fp32 [B, Hq]."""
    fast = _native()
    if fast is not None and o is None and lse is None and ws is None:
        made = rope
        if made is None and rope_theta and prefix_k.dim() == 3 and k_cache.dim() == 4:
            made = _ROPE_CACHE.get((prefix_k.shape[1] + k_cache.shape[2], float(rope_theta), k_cache.get_device()))
        if made is not None or not rope_theta:
            r = fast.prefix(q, k_new, v_new, prefix_k, prefix_v, k_cache, v_cache, pos, made)
            if type(r) is tuple:
                return r
            if r is not None:
                check(r, "sfa_prefix_decode")
    at = k_cache.get_device() if k_cache.is_cuda else -1
    if at < 0 or k_cache.dim() != 4 or not k_cache.is_contiguous():
        _refuse("k_cache", k_cache, k_cache.dtype, (None, None, None, 64))
    B, Hkv, T, _ = k_cache.shape
    dtype = k_cache.dtype
    code = _code(dtype)
    kp, vp = _dense(at, (B, Hkv, T, 64), dtype, k_cache, "k_cache"), _dense(at, (B, Hkv, T, 64), dtype, v_cache, "v_cache")
    n, Hq, qs = _rows(q, "q", 0, at)
    news = [(t, name, *(_rows(t, name, Hkv, at) if t is not None else (B, Hkv, 64 * Hkv))) for t, name in ((k_new, "k_new"), (v_new, "v_new"))]
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new are given together, or neither")
    for t, name, rows, *_ in ((q, "q", n), *news):
        if rows != B or (t is not None and t.dtype is not dtype):
            raise ValueError(f"{name} must have the caches' {B} rows and type {dtype}, got {rows} and {t.dtype}")
    P, pks = _heads(prefix_k, "prefix_k", at, dtype, Hkv)
    P2, pvs = _heads(prefix_v, "prefix_v", at, dtype, Hkv)
    if P2 != P:
        raise ValueError(f"prefix_v must have prefix_k's {P} rows, got {P2}")
    rp, rT = _rope(rope, rope_theta, P + T, at)
    d = _prefix_desc(B, P, T, Hq, Hkv, 64, code, qs, news[0][4], news[1][4], pks, pvs, rp, rT)
    o, op = _output(o, "o", at, (B, Hq, 64), dtype)
    lse, lp = _output(lse, "lse", at, (B, Hq), _F32)
    wp, size, keep = _workspace("sfa_prefix_workspace_size", at, ws, d)
    _call("sfa_prefix_decode", at, d, q.data_ptr(), *(None if t is None else t.data_ptr() for t in (k_new, v_new)),
          prefix_k.data_ptr() if P else None, prefix_v.data_ptr() if P else None, kp, vp, _ints(at, B, pos, "pos"), op, lp, wp, size)
    return o, lse

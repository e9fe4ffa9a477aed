"""Python names of libsfa's paged 4-bit key/value cache (sfa_kv4_*).

A serving step of a layer is kv4_plan (once for all layers), kv4_append and
kv4_attend.  The cache is a uint8 CUDA tensor [pages, Hkv, 72 * page] whose
layout include/sfa.h gives; everything else is an int32 tensor on the same
device.  Calls take the current stream of that device, only enqueue work, and
may be captured into a CUDA graph.

A decode step of a small batch takes the GPU a few microseconds, less than
Python takes to look its arguments over.  So a call whose arguments are in order
is made by csrc/kv4_py.cpp.  What that does not take (arguments to be refused,
another device than the current one, a RoPE table yet to be made, a workspace of
the caller's), or all if it could not be built, is done here.
"""
from __future__ import annotations

import ctypes as C
import functools
import struct

import torch

from ._lib import SFA_BF16, SFA_F32, SIGNATURES, _lib, check, i32_array
from .api import _ROPE_CACHE, _kept_rope_table, rope_table

ROW_BYTES = 72  # one (row, head): 32 + 32 bytes of codes, 8 of scales
PAGES = {ROW_BYTES * page: page for page in (16, 32, 64, 128)}
MAX_OWN_POSITIONS = 1 << 20  # longest RoPE table (256 bytes a position) that a call makes by itself
CODES = {torch.bfloat16: SFA_BF16, torch.float32: SFA_F32}

_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
_MAX = 3.4e38  # of the stored numbers' scales
# the bytes of _lib.Kv4Desc (0.2 us; filling in the structure takes 0.8)
_desc = struct.Struct("9i4x3q2fPi4xPi4x").pack
_OFFSETS: dict = {}
_current_device = torch.cuda.current_device
# the current stream's handle: the direct getter takes 0.1 us, the Stream object 2
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _refuse(name, t, dtype, shape, index=None):
    """Say why t is not a contiguous CUDA tensor of this type and shape (None: any size) on device `index`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libsfa has no CPU path)")
    if t.dtype != dtype or t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        want = ", ".join("any" if n is None else str(n) for n in shape)
        raise ValueError(f"{name} must be {dtype} [{want}], got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on device {t.get_device()}, expected {index}")


def _ints(index, n, t, name):
    """Address of t, int32 [n] on device `index`."""
    if not (t.dtype is _I32 and t.get_device() == index and t.shape == (n,) and t.is_contiguous()):
        _refuse(name, t, _I32, (n,), index)
    return t.data_ptr()


def _dense(index, shape, dtype, t, name):
    """Address of t, contiguous, of this shape and type, on device `index`."""
    if not (t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous()):
        _refuse(name, t, dtype, shape, index)
    return t.data_ptr()


def _pool(cache):
    """Device index, pages, KV heads and rows a page of a cache."""
    if not (cache.dtype is _U8 and cache.is_cuda and cache.dim() == 3 and cache.is_contiguous()):
        _refuse("cache", cache, _U8, (None, None, None))
    P, H, width = cache.shape
    page = PAGES.get(width)
    if page is None:
        raise ValueError(f"cache must be [pages, Hkv, {ROW_BYTES} * page] with page 16, 32, 64 or 128, "
                         f"got {tuple(cache.shape)}")
    return cache.get_device(), P, H, page


def _code(dtype) -> int:
    code = CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _rows(t, name, heads, index):
    """Rows, heads and the stride between the rows of t [N, heads, 64], whose rows are dense."""
    if t.get_device() != index or t.dim() != 3:
        _refuse(name, t, t.dtype, (None, heads or None, 64), index)
    n, h, d = t.shape
    if d != 64 or (heads and h != heads):
        raise ValueError(f"{name} must be [rows, {heads or 'Hq'}, 64], got {tuple(t.shape)}")
    if t.is_contiguous():
        return n, h, 64 * h
    s = t.stride()
    if s[2] != 1 or (s[1] != 64 and h > 1):
        raise ValueError(f"{name}: the [heads, 64] part of a row must be contiguous")
    if n <= 1:
        return n, h, 64 * h
    if s[0] < 64 * h or s[0] * t.element_size() % 16:
        raise ValueError(f"{name}: rows must not overlap and must start at multiples of 16 bytes")
    return n, h, s[0]


def _scales(kscale, vscale):
    raise ValueError(f"kscale and vscale must be positive and finite, got {kscale}, {vscale}")


def _rope(rope, rope_theta, T, index):
    """Pointer and positions of the RoPE table: the caller's, or the cached one of rope_theta for T positions."""
    if rope is None:
        if not rope_theta or rope_theta <= 0:
            return 0, 0
        if T > MAX_OWN_POSITIONS:
            raise ValueError(f"a RoPE table for {T} positions is not made on the side: pass rope=rope_table(positions)")
        rope = _kept_rope_table(T, rope_theta, index)
        if rope is None:
            with torch.cuda.device(index):
                capturing = torch.cuda.is_current_stream_capturing()
            if capturing:  # (only the cache keeps a table alive behind its address)
                raise ValueError("make the RoPE table before the capture: rope_table(T, rope_theta), passed as rope=")
            rope = rope_table(T, rope_theta, torch.device("cuda", index))
    n = rope.shape[0]
    if not (rope.dtype is _F32 and rope.get_device() == index and rope.shape == (n, 32, 2) and rope.is_contiguous()):
        _refuse("rope", rope, _F32, (None, 32, 2), index)
    return rope.data_ptr(), n


def _made_rope(rope_theta, cache, t, axis):
    """The RoPE table that an earlier call made for as many pages as t has along axis, if one did."""
    page = PAGES.get(cache.shape[-1]) if cache.dim() and t.dim() else None
    return page and _ROPE_CACHE.get((t.shape[axis] * page, float(rope_theta), cache.get_device()))


def _offsets(dist: tuple):
    """Address, number and array of host offsets, kept by the values of Python ints."""
    found = _OFFSETS.get(dist)
    if found is None:
        arr, n = i32_array(dist)
        found = C.addressof(arr), n, arr
        if all(type(s) is int for s in dist):  # (a tensor's element is found by its identity, whatever it holds now)
            if len(_OFFSETS) >= 64:
                _OFFSETS.clear()
            _OFFSETS[dist] = found
    return found


@functools.cache
def _entry(name):
    """The entry point, its descriptor given as bytes."""
    fn = _lib()[name]
    fn.argtypes = [C.c_char_p] + SIGNATURES[name][1:]
    return fn


def _call(name, index, *args):
    """Entry point `name`(*args, the device's current stream), with that device current."""
    fn = _entry(name)
    if index == _current_device():
        rc = fn(*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream_of(index))
    if rc:
        check(rc, name)


@functools.cache
def _native():
    """The native calls, or None where they could not be built."""
    try:
        from . import _kv4
    except ImportError:
        return None
    L = _lib()
    _kv4.bind(*(C.cast(L["sfa_kv4_" + name], C.c_void_p).value for name in ("plan", "append", "read", "workspace_size", "attend")))
    return _kv4


def kv4_cache(n_pages: int, Hkv: int, page: int = 64, device=None):
    """A pool of n_pages pages, every row zero."""
    n = C.c_size_t(0)
    check(_lib().sfa_kv4_cache_bytes(n_pages, page, Hkv, C.byref(n)), "sfa_kv4_cache_bytes")
    return torch.zeros((n_pages, Hkv, ROW_BYTES * page), dtype=_U8, device=device or "cuda")


def kv4_plan(n_new, seq_lens, block_table, free_pages, n_free, *, page: int, rows: int,
             seq_lens_out=None, n_free_out=None):
    """Block tables and slot maps of one step, built on the GPU (sfa_kv4_plan).

    n_new int32 [R]: new rows of each request, -1 to end it; seq_lens [R];
    block_table [R, max_pages] and free_pages [pages] (a stack of n_free[0] page
    ids) are updated in place.  rows: the capacity of the row maps.  Returns
    cu_q [R + 1], slots [rows], pos [rows], and the lengths and the number of
    free pages after the step (seq_lens_out=seq_lens and n_free_out=n_free
    update those in place, as a captured step wants).  What is not given is made
    as slices of one allocation: keeping or saving one of them keeps or saves
    all (clone what should live on alone).  A step that does not fit changes
    nothing and sets the device status."""
    fast = _native()
    if fast is not None:
        r = fast.plan(n_new, seq_lens, block_table, free_pages, n_free, page, rows, seq_lens_out, n_free_out)
        if type(r) is tuple:
            return r
        if r is not None:
            check(r, "sfa_kv4_plan")
    if not (block_table.dtype is _I32 and block_table.is_cuda and block_table.dim() == 2 and block_table.is_contiguous()):
        _refuse("block_table", block_table, _I32, (None, None))
    if rows < 0:
        raise ValueError("rows must not be negative")
    at = block_table.get_device()
    R, width = block_table.shape
    P = free_pages.shape[0]
    own = torch.empty((2 * R + 2 + 2 * rows,), dtype=_I32, device=block_table.device)
    cu_q, slots, pos, lens, left = own.split_with_sizes((R + 1, rows, rows, R, 1))
    p = own.data_ptr()
    p_lens = p + 4 * (R + 1 + 2 * rows)
    p_left = p_lens + 4 * R
    if seq_lens_out is not None:
        lens, p_lens = seq_lens_out, _ints(at, R, seq_lens_out, "seq_lens_out")
    if n_free_out is not None:
        left, p_left = n_free_out, _ints(at, 1, n_free_out, "n_free_out")
    _call("sfa_kv4_plan", at, _desc(P, page, 0, 0, R, width, rows, 0, 0, 0, 0, 0, 0.0, 0.0, 0, 0, 0, 0), _ints(at, R, n_new, "n_new"),
          _ints(at, R, seq_lens, "seq_lens"), block_table.data_ptr(), _ints(at, P, free_pages, "free_pages"),
          _ints(at, 1, n_free, "n_free"), p, p + 4 * (R + 1), p + 4 * (R + 1 + rows), p_lens, p_left)
    return cu_q, slots, pos, lens, left


def kv4_append(k, v, cache, slots, pos, *, rope_theta: float = 1e4, rope=None, kscale: float = 1.0,
               vscale: float = 1.0):
    """Rotate, quantise and store new rows (sfa_kv4_append): k, v [N, Hkv, 64]
    (bf16 or fp32; rows may be slices of wider ones) at slots [N] (distinct;
    negative: skipped) and positions pos [N].  rope: a table of rope_table that
    covers the positions; else one of rope_theta for as many positions as the
    pool has rows, up to 2^20 (0: no rotation).  The first call that wants a
    longer one than is there makes it, and waits for it, as rope_table does."""
    fast = _native()
    made = rope if rope is not None or not rope_theta else _made_rope(rope_theta, cache, cache, 0)
    if fast is not None and (made is not None or not rope_theta):
        r = fast.append(k, v, cache, slots, pos, made, kscale, vscale)
        if r is not None:
            return check(r, "sfa_kv4_append") if r else None
    at, P, H, page = _pool(cache)
    N, _, ks = _rows(k, "k", H, at)
    n, _, vs = _rows(v, "v", H, at)
    dtype = k.dtype
    if n != N or v.dtype is not dtype:
        raise ValueError(f"k and v must have the same rows and type, got {tuple(k.shape)} {dtype}, {tuple(v.shape)} {v.dtype}")
    if not (0.0 < kscale <= _MAX and 0.0 < vscale <= _MAX):
        _scales(kscale, vscale)
    rp, rT = _rope(rope, rope_theta, P * page, at)
    _call("sfa_kv4_append", at, _desc(P, page, H, 64, 0, 0, N, 0, _code(dtype), 0, ks, vs, kscale, vscale, rp, rT, 0, 0),
          k.data_ptr(), v.data_ptr(),
          cache.data_ptr(), _ints(at, N, slots, "slots"), _ints(at, N, pos, "pos"))


def kv4_read(cache, slots, *, dtype=None, kscale: float = 1.0, vscale: float = 1.0, k=None, v=None):
    """Rows of the cache as numbers (sfa_kv4_read): k, v [N, Hkv, 64], the
    rotated keys and the values stored at slots [N] (negative: zeros)."""
    fast = _native()
    if fast is not None and k is None and v is None and (dtype is None or dtype in CODES):
        r = fast.read(cache, slots, kscale, vscale, dtype is not _F32)
        if type(r) is tuple:
            return r
        if r is not None:
            check(r, "sfa_kv4_read")
    at, P, H, page = _pool(cache)
    if dtype is None:
        dtype = k.dtype if k is not None else torch.bfloat16
    code = _code(dtype)
    N = slots.shape[0]
    if not (0.0 < kscale <= _MAX and 0.0 < vscale <= _MAX):
        _scales(kscale, vscale)
    shape = (N, H, 64)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache.device)
        kp = k.data_ptr()
    else:
        kp = _dense(at, shape, dtype, k, "k")
    if v is None:
        v = torch.empty_like(k)
        vp = v.data_ptr()
    else:
        vp = _dense(at, shape, dtype, v, "v")
    _call("sfa_kv4_read", at, _desc(P, page, H, 64, 0, 0, N, 0, code, 0, 0, 0, kscale, vscale, 0, 0, 0, 0),
          cache.data_ptr(), _ints(at, N, slots, "slots"), kp, vp)
    return k, v


def _attend_desc(q, cache, block_table, dist, rope_theta, rope, kscale, vscale):
    at, P, H, page = _pool(cache)
    N, Hq, qs = _rows(q, "q", 0, at)
    if not (block_table.dtype is _I32 and block_table.get_device() == at and block_table.dim() == 2 and block_table.is_contiguous()):
        _refuse("block_table", block_table, _I32, (None, None), at)
    R, width = block_table.shape
    if not (0.0 < kscale <= _MAX and 0.0 < vscale <= _MAX):
        _scales(kscale, vscale)
    rp, rT = _rope(rope, rope_theta, width * page, at)
    offsets = arr, nd, _ = _offsets(tuple(dist)) if dist is not None else (0, 0, None)
    return at, R, N, Hq, offsets, _desc(P, page, H, 64, R, width, N, Hq, _code(q.dtype), qs, 0, 0, kscale, vscale, rp, rT, arr, nd)


def kv4_workspace_size(q, cache, block_table, *, dist=None) -> int:
    """Scratch bytes of kv4_attend for these shapes."""
    n = C.c_size_t(0)
    *_, keep, d = _attend_desc(q, cache, block_table, dist, 0, None, 1.0, 1.0)
    check(_entry("sfa_kv4_workspace_size")(d, C.byref(n)), "sfa_kv4_workspace_size")
    return n.value


def kv4_attend(q, cache, block_table, seq_lens, *, cu_q=None, dist=None, rope_theta: float = 1e4, rope=None,
               kscale: float = 1.0, vscale: float = 1.0, o=None, lse=None, ws=None):
    """Attention over the cached rows (sfa_kv4_attend): q [N, Hq, 64] (unrotated;
    rows may be slices of wider ones).  cu_q None: one row a request, at its last
    position (seq_lens - 1); else rows cu_q[r] .. cu_q[r + 1] - 1 are the last
    positions of request r, and rows behind cu_q[R] are left as they were.
    dist: offsets as for decode_int (0 required), None for every earlier row.
    rope: as in kv4_append (without it, for the block table's width).  o and lse
    overlap none of the inputs.  Returns o [N, Hq, 64] and lse fp32 [N, Hq]."""
    fast = _native()
    made = rope if rope is not None or not rope_theta else _made_rope(rope_theta, cache, block_table, -1)
    if fast is not None and (made is not None or not rope_theta):
        r = fast.attend(q, cache, block_table, seq_lens, cu_q, None if dist is None else _offsets(tuple(dist)), made, kscale, vscale,
                        o, lse, ws)
        if type(r) is tuple:
            return r
        if r is not None:
            check(r, "sfa_kv4_attend")
    at, R, N, Hq, keep, d = _attend_desc(q, cache, block_table, dist, rope_theta, rope, kscale, vscale)
    if cu_q is None and N != R:
        raise ValueError(f"without cu_q, q has one row for each of the {R} requests, got {N}")
    if o is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = o.data_ptr()
    else:
        op = _dense(at, (N, Hq, 64), q.dtype, o, "o")
    if lse is None:
        lse = torch.empty((N, Hq), dtype=_F32, device=q.device)
        lp = lse.data_ptr()
    else:
        lp = _dense(at, (N, Hq), _F32, lse, "lse")
    n = C.c_size_t(0)
    rc = _entry("sfa_kv4_workspace_size")(d, C.byref(n))
    if rc:
        check(rc, "sfa_kv4_workspace_size")
    n = n.value
    if n == 0:
        w = None
    else:
        if ws is None or ws.numel() * ws.element_size() < n:
            ws = torch.empty((n,), dtype=_U8, device=q.device)
        elif ws.get_device() != at or not ws.is_contiguous():
            _refuse("ws", ws, ws.dtype, tuple(ws.shape), at)
        w = ws.data_ptr()
    _call("sfa_kv4_attend", at, d, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
          _ints(at, R, seq_lens, "seq_lens"), None if cu_q is None else _ints(at, R + 1, cu_q, "cu_q"), op, lp, w, n)
    return o, lse

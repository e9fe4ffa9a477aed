"""Python names of libsfa's paged 4-bit key/value cache (sfa_kv4_*).

A serving step of a layer is kv4_plan (once for all layers), kv4_append and
kv4_attend.  The cache is a uint8 CUDA tensor [pages, Hkv, 72 * page] whose
layout include/sfa.h gives; everything else is an int32 tensor on the same
device.  Calls take the current stream of that device, only enqueue work, and
may be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes as C
import functools
import math

from ._lib import SFA_BF16, SFA_F32, Kv4Desc, _lib, check, i32_array
from .api import _ROPE_CACHE, _torch, rope_table

ROW_BYTES = 72  # one (row, head): 32 + 32 bytes of codes, 8 of scales


def _need(t, name, dtype, dim, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libsfa has no CPU path)")
    if t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name} must be {dtype} with {dim} dimension(s), got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache's device is {device}")


def _ints(device, **tensors):
    i32 = _torch().int32
    for name, t in tensors.items():
        _need(t, name, i32, 1, device)


def _page(cache) -> int:
    _need(cache, "cache", _torch().uint8, 3)
    page, rest = divmod(cache.shape[2], ROW_BYTES)
    if rest or page not in (16, 32, 64, 128):
        raise ValueError(f"cache must be [pages, Hkv, {ROW_BYTES} * page] with page 16, 32, 64 or 128, "
                         f"got {tuple(cache.shape)}")
    return page


def _code(dtype) -> int:
    torch = _torch()
    if dtype == torch.bfloat16:
        return SFA_BF16
    if dtype == torch.float32:
        return SFA_F32
    raise TypeError(f"unsupported dtype {dtype}")


def _rows(t, name, heads, device, dtype=None):
    """Stride between the rows of t [N, heads, 64], whose rows are dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libsfa has no CPU path)")
    if t.dim() != 3 or t.shape[2] != 64 or (heads and t.shape[1] != heads):
        raise ValueError(f"{name} must be [rows, {heads or 'Hq'}, 64], got {tuple(t.shape)}")
    if t.device != device or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype or t.dtype} on {device}, got {t.dtype} on {t.device}")
    s = t.stride()
    width = t.shape[1] * 64
    if s[2] != 1 or (s[1] != 64 and t.shape[1] > 1):
        raise ValueError(f"{name}: the [heads, 64] part of a row must be contiguous")
    if t.shape[0] <= 1:
        return width
    if s[0] < width or s[0] * t.element_size() % 16:
        raise ValueError(f"{name}: rows must not overlap and must start at multiples of 16 bytes")
    return s[0]


def _scales(kscale, vscale):
    for name, x in (("kscale", kscale), ("vscale", vscale)):
        if not (0.0 < x < math.inf):
            raise ValueError(f"{name} must be positive and finite")


def _rope(rope, rope_theta, T, device):
    """The table's (pointer, positions, tensor): the caller's, or the cached one of rope_theta."""
    torch = _torch()
    if rope is None:
        if not rope_theta or rope_theta <= 0:
            return None, 0, None
        key = (int(T), float(rope_theta), device.index)
        if key not in _ROPE_CACHE:
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("make the RoPE table before the capture: rope_table(T, rope_theta), passed as rope=")
            rope_table(T, rope_theta, device)
            # the table is shared by later calls on any stream
            torch.cuda.current_stream(device).synchronize()
        rope = _ROPE_CACHE[key]
    _need(rope, "rope", torch.float32, 3, device)
    if rope.shape[1:] != (32, 2):
        raise ValueError(f"rope must be [positions, 32, 2], got {tuple(rope.shape)}")
    return rope.data_ptr(), rope.shape[0], rope


@functools.lru_cache(maxsize=64)
def _offsets(dist: tuple):
    return i32_array(dist)


def _call(fn, name, device, desc, *args):
    torch = _torch()
    if device.index == torch.cuda.current_device():
        check(fn(desc, *args, torch.cuda.current_stream(device).cuda_stream), name)
        return
    with torch.cuda.device(device):
        check(fn(desc, *args, torch.cuda.current_stream(device).cuda_stream), name)


def kv4_cache(n_pages: int, Hkv: int, page: int = 64, device=None):
    """A pool of n_pages pages, every row zero."""
    n = C.c_size_t(0)
    check(_lib().sfa_kv4_cache_bytes(n_pages, page, Hkv, C.byref(n)), "sfa_kv4_cache_bytes")
    torch = _torch()
    return torch.zeros((n_pages, Hkv, ROW_BYTES * page), dtype=torch.uint8, device=device or "cuda")


def kv4_plan(n_new, seq_lens, block_table, free_pages, n_free, *, page: int, rows: int,
             seq_lens_out=None, n_free_out=None):
    """Block tables and slot maps of one step, built on the GPU (sfa_kv4_plan).

    n_new int32 [R]: new rows of each request, -1 to end it; seq_lens [R];
    block_table [R, max_pages] and free_pages [pages] (a stack of n_free[0] page
    ids) are updated in place.  rows: the capacity of the row maps.  Returns
    cu_q [R + 1], slots [rows], pos [rows], and the lengths and the number of
    free pages after the step (seq_lens_out=seq_lens and n_free_out=n_free
    update those in place, as a captured step wants).  A step that does not fit
    changes nothing and sets the device status."""
    torch = _torch()
    dev = block_table.device
    _need(block_table, "block_table", torch.int32, 2)
    _ints(dev, n_new=n_new, seq_lens=seq_lens, free_pages=free_pages, n_free=n_free)
    R = block_table.shape[0]
    if n_new.shape[0] != R or seq_lens.shape[0] != R or n_free.shape[0] != 1:
        raise ValueError("kv4_plan: n_new and seq_lens [R], block_table [R, max_pages], n_free [1]")
    if rows < 0:
        raise ValueError("rows must not be negative")
    for name, t, n in (("seq_lens_out", seq_lens_out, R), ("n_free_out", n_free_out, 1)):
        if t is not None:
            _ints(dev, **{name: t})
            if t.shape[0] != n:
                raise ValueError(f"{name} must have {n} element(s)")
    own = torch.empty((2 * R + 2 + 2 * rows,), dtype=torch.int32, device=dev).split([R + 1, rows, rows, R, 1])
    out = (*own[:3], own[3] if seq_lens_out is None else seq_lens_out, own[4] if n_free_out is None else n_free_out)
    d = Kv4Desc(n_pages=free_pages.shape[0], page=page, R=R, max_pages=block_table.shape[1], N=rows)
    _call(_lib().sfa_kv4_plan, "sfa_kv4_plan", dev, d, n_new.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
          free_pages.data_ptr(), n_free.data_ptr(), *[t.data_ptr() for t in out])
    return out


def kv4_append(k, v, cache, slots, pos, *, rope_theta: float = 1e4, rope=None, kscale: float = 1.0,
               vscale: float = 1.0):
    """Rotate, quantise and store new rows (sfa_kv4_append): k, v [N, Hkv, 64]
    (bf16 or fp32; rows may be slices of wider ones) at slots [N] (distinct;
    negative: skipped) and positions pos [N].  rope: a table of rope_table; else
    the one of rope_theta for the pool's rows (0: no rotation)."""
    page = _page(cache)
    dev, H = cache.device, cache.shape[1]
    ks, vs = _rows(k, "k", H, dev), _rows(v, "v", H, dev, k.dtype)
    _ints(dev, slots=slots, pos=pos)
    N = k.shape[0]
    if v.shape[0] != N or slots.shape[0] != N or pos.shape[0] != N:
        raise ValueError("kv4_append: k and v [N, Hkv, 64], slots and pos [N]")
    _scales(kscale, vscale)
    rp, rT, keep = _rope(rope, rope_theta, min(cache.shape[0] * page, 1 << 24), dev)
    d = Kv4Desc(cache.shape[0], page, H, 64, 0, 0, N, 0, _code(k.dtype), 0, ks, vs, kscale, vscale, rp, rT)
    _call(_lib().sfa_kv4_append, "sfa_kv4_append", dev, d, k.data_ptr(), v.data_ptr(), cache.data_ptr(), slots.data_ptr(),
          pos.data_ptr())


def kv4_read(cache, slots, *, dtype=None, kscale: float = 1.0, vscale: float = 1.0, k=None, v=None):
    """Rows of the cache as numbers (sfa_kv4_read): k, v [N, Hkv, 64], the
    rotated keys and the values stored at slots [N] (negative: zeros)."""
    torch = _torch()
    page = _page(cache)
    dev, H = cache.device, cache.shape[1]
    _ints(dev, slots=slots)
    dtype = dtype or (k.dtype if k is not None else torch.bfloat16)
    code = _code(dtype)
    N = slots.shape[0]
    _scales(kscale, vscale)
    if k is None:
        k = torch.empty((N, H, 64), dtype=dtype, device=dev)
    if v is None:
        v = torch.empty((N, H, 64), dtype=dtype, device=dev)
    for name, t in (("k", k), ("v", v)):
        _need(t, name, dtype, 3, dev)
        if t.shape != (N, H, 64):
            raise ValueError(f"{name} must be {(N, H, 64)}, got {tuple(t.shape)}")
    d = Kv4Desc(cache.shape[0], page, H, 64, 0, 0, N, 0, code, 0, 0, 0, kscale, vscale)
    _call(_lib().sfa_kv4_read, "sfa_kv4_read", dev, d, cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr())
    return k, v


def _attend_desc(q, cache, block_table, dist, rope_theta, rope, kscale, vscale):
    page = _page(cache)
    dev, H = cache.device, cache.shape[1]
    qs = _rows(q, "q", 0, dev)
    _need(block_table, "block_table", _torch().int32, 2, dev)
    _scales(kscale, vscale)
    rp, rT, keep = _rope(rope, rope_theta, min(block_table.shape[1] * page, 1 << 24), dev)
    arr, nd = _offsets(tuple(dist)) if dist is not None else (None, 0)
    d = Kv4Desc(cache.shape[0], page, H, 64, block_table.shape[0], block_table.shape[1], q.shape[0], q.shape[1],
                _code(q.dtype), qs, 0, 0, kscale, vscale, rp, rT, C.cast(arr, C.c_void_p) if arr is not None else None, nd)
    d._keep = (arr, keep)
    return d


def kv4_workspace_size(q, cache, block_table, *, dist=None) -> int:
    """Scratch bytes of kv4_attend for these shapes."""
    n = C.c_size_t(0)
    d = _attend_desc(q, cache, block_table, dist, 0, None, 1.0, 1.0)
    check(_lib().sfa_kv4_workspace_size(d, C.byref(n)), "sfa_kv4_workspace_size")
    return n.value


def kv4_attend(q, cache, block_table, seq_lens, *, cu_q=None, dist=None, rope_theta: float = 1e4, rope=None,
               kscale: float = 1.0, vscale: float = 1.0, o=None, lse=None, ws=None):
    """Attention over the cached rows (sfa_kv4_attend): q [N, Hq, 64] (unrotated;
    rows may be slices of wider ones).  cu_q None: one row a request, at its last
    position (seq_lens - 1); else rows cu_q[r] .. cu_q[r + 1] - 1 are the last
    positions of request r, and rows behind cu_q[R] are left as they were.
    dist: offsets as for decode_int (0 required), None for every earlier row.
    Returns o [N, Hq, 64] and lse fp32 [N, Hq]."""
    torch = _torch()
    d = _attend_desc(q, cache, block_table, dist, rope_theta, rope, kscale, vscale)
    dev, (N, Hq, _) = cache.device, q.shape
    _ints(dev, seq_lens=seq_lens)
    R = block_table.shape[0]
    if seq_lens.shape[0] != R:
        raise ValueError("kv4_attend: seq_lens [R], block_table [R, max_pages]")
    if cu_q is None:
        if N != R:
            raise ValueError(f"kv4_attend: without cu_q, q has a row for each of the {R} requests, got {N}")
    else:
        _ints(dev, cu_q=cu_q)
        if cu_q.shape[0] != R + 1:
            raise ValueError("kv4_attend: cu_q [R + 1]")
    if o is None:
        o = torch.empty((N, Hq, 64), dtype=q.dtype, device=dev)
    else:
        _need(o, "o", q.dtype, 3, dev)
    if lse is None:
        lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", torch.float32, 2, dev)
    if o.shape != (N, Hq, 64) or lse.shape != (N, Hq):
        raise ValueError(f"kv4_attend: o {(N, Hq, 64)} and lse {(N, Hq)}")
    L = _lib()
    n = C.c_size_t(0)
    check(L.sfa_kv4_workspace_size(d, C.byref(n)), "sfa_kv4_workspace_size")
    if n.value and (ws is None or ws.numel() < n.value):
        ws = torch.empty((n.value,), dtype=torch.uint8, device=dev)
    _call(L.sfa_kv4_attend, "sfa_kv4_attend", dev, d, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
          seq_lens.data_ptr(), cu_q.data_ptr() if cu_q is not None else None, o.data_ptr(), lse.data_ptr(),
          ws.data_ptr() if n.value else None, n.value)
    return o, lse

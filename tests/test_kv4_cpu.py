"""The paged 4-bit cache without a GPU: refusals of the C ABI and of the Python names, and the plain
definitions that the GPU tests use."""
import ctypes as C

import numpy as np
import pytest

import kv4_ref as ref


def _desc(**kw):
    from static_offset_sparse_gb300._lib import Kv4Desc

    d = dict(n_pages=4, page=16, Hkv=2, D=64, R=3, max_pages=2, N=3, Hq=8, dtype=1, q_stride=512, k_stride=128,
             v_stride=128, kscale=1.0, vscale=1.0)
    d.update(kw)
    return Kv4Desc(**d)


P, ODD = 4096, 4098  # never dereferenced: every call below is refused first


def test_cache_bytes(sfa_lib):
    n = C.c_size_t(0)
    assert sfa_lib.sfa_kv4_cache_bytes(7, 64, 3, C.byref(n)) == 0 and n.value == 7 * 3 * 64 * 72
    assert sfa_lib.sfa_kv4_cache_bytes(0, 64, 3, C.byref(n)) == 1
    assert sfa_lib.sfa_kv4_cache_bytes(7, 24, 3, C.byref(n)) == 2
    assert sfa_lib.sfa_kv4_cache_bytes(1 << 27, 16, 3, C.byref(n)) == 2
    assert sfa_lib.sfa_kv4_cache_bytes(7, 64, 3, None) == 1


@pytest.mark.parametrize("kw,rc", [(dict(n_pages=0), 1), (dict(page=48), 2), (dict(page=-16), 1), (dict(N=-1), 1), (dict(R=0), 1),
                                   (dict(R=8193), 2), (dict(max_pages=0), 1), (dict(max_pages=1 << 24), 2)])
def test_plan_refusals(sfa_lib, kw, rc):
    assert sfa_lib.sfa_kv4_plan(_desc(**kw), *[P] * 10, None) == rc


def test_plan_pointer_refusals(sfa_lib):
    for i in range(10):
        for bad in (None, ODD):
            args = [P] * 10
            args[i] = bad
            assert sfa_lib.sfa_kv4_plan(_desc(), *args, None) == 1, i


@pytest.mark.parametrize("kw,rc", [(dict(D=128), 2), (dict(dtype=2), 1), (dict(Hkv=0), 1), (dict(kscale=0.0), 1), (dict(vscale=-1.0), 1),
                                   (dict(kscale=float("nan")), 1), (dict(vscale=float("inf")), 1), (dict(rope=P, rope_T=0), 1),
                                   (dict(rope=ODD, rope_T=4), 1), (dict(N=1 << 27), 2), (dict(page=8), 2), (dict(n_pages=1 << 26, Hkv=2), 2)])
def test_row_refusals(sfa_lib, kw, rc):
    d = _desc(**kw)
    assert sfa_lib.sfa_kv4_append(d, P, P, P, P, P, None) == rc
    assert sfa_lib.sfa_kv4_read(d, P, P, P, P, None) == rc
    assert sfa_lib.sfa_kv4_attend(d, P, P, P, P, None, P, P, None, 0, None) == rc
    n = C.c_size_t(0)
    assert sfa_lib.sfa_kv4_workspace_size(d, C.byref(n)) == rc


@pytest.mark.parametrize("kw,rc", [(dict(Hq=6), 2), (dict(Hq=7), 2), (dict(Hq=128), 2), (dict(Hq=0), 1), (dict(R=0), 1), (dict(R=4), 1),
                                   (dict(max_pages=0), 1), (dict(max_pages=1 << 21), 2), (dict(q_stride=504), 1), (dict(q_stride=513), 1), (dict(R=1 << 20, N=1 << 20, Hkv=8, max_pages=1 << 20), 2)])
def test_attend_refusals(sfa_lib, kw, rc):
    assert sfa_lib.sfa_kv4_attend(_desc(**kw), P, P, P, P, None, P, P, P, 1 << 30, None) == rc


def test_stride_and_pointer_refusals(sfa_lib):
    for kw in (dict(k_stride=64), dict(v_stride=120), dict(k_stride=130), dict(v_stride=132)):
        assert sfa_lib.sfa_kv4_append(_desc(**kw), P, P, P, P, P, None) == 1
    for i in range(5):
        for bad in (None, ODD):
            args = [P] * 5
            args[i] = bad
            assert sfa_lib.sfa_kv4_append(_desc(), *args, None) == 1
            if i < 4:
                assert sfa_lib.sfa_kv4_read(_desc(), *args[:4], None) == 1
    for i in range(7):
        args = [P] * 7 + [P, 1 << 30]
        args[i] = ODD
        assert sfa_lib.sfa_kv4_attend(_desc(), *args, None) == 1, i


@pytest.mark.parametrize("dist,rc", [([1, 2], 1), ([0, -1], 1), ([], 1), (list(range(0, 600, 2)), 2)])
def test_offset_refusals(sfa_lib, dist, rc):
    arr = (C.c_int32 * max(1, len(dist)))(*dist)
    d = _desc(dist=C.cast(arr, C.c_void_p), n_dist=len(dist))
    n = C.c_size_t(0)
    assert sfa_lib.sfa_kv4_workspace_size(d, C.byref(n)) == rc


def test_nothing_to_do(sfa_lib):
    """No rows: nothing is launched, whatever the pointers."""
    assert sfa_lib.sfa_kv4_append(_desc(N=0), None, None, None, None, None, None) == 0
    assert sfa_lib.sfa_kv4_read(_desc(N=0), None, None, None, None, None) == 0
    assert sfa_lib.sfa_kv4_attend(_desc(N=0), P, P, P, P, P, P, P, None, 0, None) == 0
    assert sfa_lib.sfa_kv4_attend(_desc(N=0, R=0), P, P, P, P, None, P, P, None, 0, None) == 0
    n = C.c_size_t(1)
    assert sfa_lib.sfa_kv4_workspace_size(_desc(N=0, R=0), C.byref(n)) == 0 and n.value == 0


def test_python_refuses_cpu_tensors(sfa_lib):
    import torch

    import static_offset_sparse_gb300 as sfa

    cache = torch.zeros((2, 2, 72 * 16), dtype=torch.uint8)
    i = torch.zeros((3,), dtype=torch.int32)
    k = torch.zeros((3, 2, 64))
    for call in (lambda: sfa.kv4_append(k, k, cache, i, i), lambda: sfa.kv4_read(cache, i),
                 lambda: sfa.kv4_attend(torch.zeros((3, 8, 64)), cache, i[None], i[:1]),
                 lambda: sfa.kv4_plan(i, i, i[:, None], i, i[:1], page=16, rows=3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_plain_codec():
    """e4m3's and e2m1's numbers, roundings to nearest even, and the codec's error."""
    assert ref.E4M3[0x7e] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[0x38] == 1.0 and np.isnan(ref.E4M3[0x7f])
    assert (np.diff(ref.E4M3[:127]) > 0).all()
    assert ref.E2M1[ref.nearest(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, 6.0]), ref.E2M1[:8])].tolist() == [0, 1, 1, 2, 2, 4, 4, 0.5, 6]
    import torch

    b = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(b.float().numpy(), ref.E4M3[:127].astype(np.float32))
    x = np.random.default_rng(0).standard_normal((200, 3, 64)).astype(np.float32)
    c, s = ref.quantise(x)
    s_t = (torch.from_numpy(np.abs(x).reshape(200, 3, 4, 16).max(-1)) / torch.tensor([6.0])).to(torch.float8_e4m3fn)
    assert np.array_equal(s_t.view(torch.uint8).numpy(), s)
    big = np.abs(x).reshape(200, 3, 4, 16).max(-1, keepdims=True).repeat(16, -1).reshape(x.shape)
    # half of e2m1's widest step (1 of 6), and the scale's rounding (2^-4) of the largest
    assert (np.abs(ref.values(c, s) - x) <= big * (1 / 6 + 2.0 ** -4)).all()


def test_plain_pool():
    pool = ref.Pool(np.full((2, 4), -1), [0, 1, 2, 3], [0, 0], 16)
    assert pool.step([17, 1], 20) == ([0, 17, 18], [3 * 16 + i for i in range(16)] + [2 * 16, 16] + [-1] * 2, list(range(17)) + [0] + [-1] * 2)
    assert pool.step([-1, 0], 1) == ([0, 0, 0], [-1], [-1]) and pool.free == [0, 3, 2] and pool.lens == [0, 1]


def _workspace(lib, **kw):
    n = C.c_size_t(0)
    assert lib.sfa_kv4_workspace_size(_desc(**kw), C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("R,N", [(8, 4000), (3, 64), (16, 17), (5, 5), (1, 1), (300, 300)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 1), (32, 1), (4, 4)])
@pytest.mark.parametrize("page,max_pages", [(64, 256), (16, 33), (128, 8192)])
def test_workspace_holds_the_split_rows(sfa_lib, R, N, Hq, Hkv, page, max_pages):
    """Room for what the kernels leave there.  Prompts (64 columns and more a request on average): two
    parts for each of 152 CTAs, 256 columns of m, l and 64 sums.  Other rows: two parts at least of every
    row and head if any scratch is wanted, within a bound that the block table's width does not move, and
    none for prefixes of one chunk (2048 keys; 256 for more than 8 columns of a few requests)."""
    kw = dict(n_pages=1 << 14, R=R, N=N, Hq=Hq, Hkv=Hkv, page=page, max_pages=max_pages, q_stride=Hq * 64)
    n = _workspace(sfa_lib, **kw)
    prompts = 2 * 152 * 256 * 66 * 4
    if page * max_pages <= 2048 and (8 * N * Hkv <= (608 if Hq // Hkv <= 8 else 304) or Hq // Hkv * -(-N // R) <= 8):
        assert n == 0
        return
    if Hq // Hkv * -(-N // R) >= 64:
        assert prompts < n <= prompts + 8 * (N + R) * Hkv
        return
    assert n >= 2 * N * Hq * 66 * 4 or (n == 0 and N > 2000)  # enough rows: none is split
    assert n <= 16 * 608 * 8 * 66 * 4 + 16 * 304 * 16 * 66 * 4
    assert _workspace(sfa_lib, **{**kw, "max_pages": 256 // page}) == 0


def test_descriptor_bytes():
    """The Python calls' descriptor, packed by hand, is the C structure."""
    pytest.importorskip("torch")
    from static_offset_sparse_gb300 import kv4
    from static_offset_sparse_gb300._lib import Kv4Desc

    values = [*range(101, 110), 2 ** 40, 2 ** 41, 2 ** 42, 0.75, 1.5, 2 ** 47 - 16, 7, 2 ** 46, 9]
    assert bytes(Kv4Desc(*values)) == kv4._desc(*values) and len(values) == len(Kv4Desc._fields_)


def test_only_rope_tables_are_read_as_read_only_data():
    """Kernels are launched early: they live while the one before them writes what they will read, and only
    ordinary loads are ordered by their wait for it.  So __ldg, and __restrict__ on what is read (which makes the
    compiler use the same loads), are for RoPE tables alone."""
    import os
    import re

    import static_offset_sparse_gb300 as pkg

    csrc = os.path.join(os.path.dirname(pkg.__file__), "csrc")
    reads = []
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        reads += [(name, m.group(0)) for m in re.finditer(r"__ldg\([^;]*;|[^,(]*__restrict__[^,)]*|ld\.global\.nc", text)]
    assert len(reads) >= 5
    for name, text in reads:
        assert "rope" in text, (name, text)


@pytest.mark.parametrize("R,N", [(2 ** 31 - 1, 3), (2 ** 31 - 1, 1 << 20), (2 ** 31 - 100, 101)])
def test_requests_beyond_32_bits(sfa_lib, R, N):
    """Rows and requests whose number passes 32 bits are refused, not counted from below zero."""
    n = C.c_size_t(0)
    assert sfa_lib.sfa_kv4_workspace_size(_desc(R=R, N=N, max_pages=4096), C.byref(n)) == 2
    assert sfa_lib.sfa_kv4_attend(_desc(R=R, N=N, max_pages=4096), P, P, P, P, P, P, P, None, 0, None) == 2


@pytest.mark.parametrize("n_pages,page,Hkv,rc", [(1 << 20, 128, 14, 0), (1 << 20, 128, 15, 2), (1 << 24, 16, 8, 2), (3, 16, 1 << 24, 0), (3, 16, 1 << 30, 2)])
def test_cache_bytes_of_caches_that_are_too_large(sfa_lib, n_pages, page, Hkv, rc):
    """A cache that every other call would refuse has no size (128 GiB and more)."""
    n = C.c_size_t(0)
    assert sfa_lib.sfa_kv4_cache_bytes(n_pages, page, Hkv, C.byref(n)) == rc
    assert sfa_lib.sfa_kv4_append(_desc(n_pages=n_pages, page=page, Hkv=Hkv, N=0, k_stride=64 * Hkv % 2 ** 31, v_stride=64 * Hkv % 2 ** 31), P, P, P, P, P, None) == rc
    if rc == 0:
        assert n.value == 72 * n_pages * page * Hkv < 2 ** 37


def test_offset_lists_are_kept_by_value():
    """Offsets in tensors may change between calls; lists of Python ints are converted once."""
    torch = pytest.importorskip("torch")
    from static_offset_sparse_gb300 import kv4

    dist = [torch.tensor(0), torch.tensor(3)]
    assert list(kv4._offsets(tuple(dist))[2]) == [0, 3]
    dist[1].fill_(5)
    assert list(kv4._offsets(tuple(dist))[2]) == [0, 5]
    assert kv4._offsets((0, 1, 7)) is kv4._offsets((0, 1, 7)) and list(kv4._offsets((0, 1, 7))[2]) == [0, 1, 7]
    assert list(kv4._offsets(tuple(np.array([0, 1, 7])))[2]) == [0, 1, 7]
    for i in range(200):  # a bounded number of them
        assert kv4._offsets((0, i + 1))[1] == 2
    assert len(kv4._OFFSETS) <= 64

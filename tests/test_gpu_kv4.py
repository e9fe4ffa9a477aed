"""The paged 4-bit key/value cache on the GPU against plain definitions in 64 bits.

Bookkeeping, stored bytes and read-back are exact; attention is held to the
bound that its roundings give (kv4_ref.bounds).
"""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu

FIB = sorted(set(range(9)) | {1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233, 377, 610, 987})
CHRIST = sorted({0} | {j for j in range(1024) if (j + 1) * 128 // 1024 - j * 128 // 1024})


@pytest.fixture(scope="module")
def sfa(sfa_lib):
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import static_offset_sparse_gb300 as s

    return s


def _cuda(x, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(dtype) if dtype is not None else t


def _i32(x):
    return _cuda(np.asarray(x, np.int32))


def _dt(name):
    import torch

    return torch.bfloat16 if name == "bf16" else torch.float32


# ------------------------------------------------------------------ plan


def _pool(rng, lens, page, spare, width):
    held = [-(-n // page) for n in lens]
    P = sum(held) + spare
    order = rng.permutation(P)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = order[at:at + h]
        at += h
    free = np.full(P, -5, np.int32)
    free[:P - at] = order[at:]
    return table, free, P - at


@pytest.mark.parametrize("R,page,rows,most", [(1, 16, 1, 1), (3, 32, 40, 20), (257, 64, 300, 1), (1000, 16, 4096, 9),
                                              (1025, 128, 4097, 4), (2500, 16, 9000, 6), (5000, 64, 5000, 1),
                                              (400, 16, 2048, 9), (400, 16, 2049, 9), (8192, 32, 8192, 1)])
def test_plan_steps(sfa, R, page, rows, most):
    """Several steps in a row: some requests grow, some idle, some end and start again."""
    import torch

    rng = np.random.default_rng(R)
    lens = [int(x) for x in rng.integers(0, 5 * page, R)]
    width = 5 + -(-6 * most // page) + 1
    table, free, nf = _pool(rng, lens, page, R + 40, width)
    pool = ref.Pool(table.copy(), free[:nf], lens, page)
    d_table, d_free, d_lens, d_nf = _cuda(table), _cuda(free), _i32(lens), _i32([nf])
    for step in range(5):
        new = [int(x) for x in rng.integers(0, most + 1, R)]
        new = [-1 if rng.random() < 0.1 else x for x in new]
        while sum(max(0, x) for x in new) > rows:
            new[int(rng.integers(0, R))] = 0
        before_free = d_free.cpu().numpy()
        nf0 = int(d_nf)
        cu, slots, pos = pool.step(new, rows)
        if step % 2:  # in place
            g = sfa.kv4_plan(_i32(new), d_lens, d_table, d_free, d_nf, page=page, rows=rows, seq_lens_out=d_lens, n_free_out=d_nf)
            assert g[3] is d_lens and g[4] is d_nf
        else:
            keep = d_lens.clone()
            g = sfa.kv4_plan(_i32(new), d_lens, d_table, d_free, d_nf, page=page, rows=rows)
            assert torch.equal(keep, d_lens) and int(d_nf) == nf0
        d_lens, d_nf = g[3], g[4]
        assert sfa.get_device_status() == 0
        assert g[0].tolist() == cu and g[1].tolist() == slots and g[2].tolist() == pos
        assert d_lens.tolist() == pool.lens and d_nf.tolist() == [len(pool.free)]
        assert np.array_equal(d_table.cpu().numpy(), pool.table)
        f = d_free.cpu().numpy()
        n = len(pool.free)
        assert f[:n].tolist() == pool.free
        assert np.array_equal(f[max(n, nf0):], before_free[max(n, nf0):])  # behind the stack: untouched


@pytest.mark.parametrize("what,status", [("pages", 3), ("rows", 3), ("new", 6), ("len", 6), ("wide", 6), ("stack", 6)])
@pytest.mark.parametrize("rows", [50, 5000])
def test_plan_that_does_not_fit(sfa, what, status, rows):
    """Nothing changes, and the status says why."""
    rng = np.random.default_rng(3)
    lens, page, width = [5, 16, 40], 16, 9
    new = [120, 0, -1] if what == "pages" else [2, 3, 1]  # 7 pages for 3 free and 3 given back
    rows = 5 if what == "rows" else rows
    table, free, nf = _pool(rng, lens, page, 3, width)
    if what == "new":
        new[1] = -2
    if what == "len":
        lens[1] = -1
    if what == "wide":
        new[0] = width * page
    if what == "stack":
        nf = len(free) + 1
    t, f, l, n = _cuda(table), _cuda(free), _i32(lens), _i32([nf])
    cu, slots, pos, lo, no = sfa.kv4_plan(_i32(new), l, t, f, n, page=page, rows=rows)
    assert sfa.get_device_status() == status
    assert cu.tolist() == [0] * 4 and set(slots.tolist()) == {-1} and set(pos.tolist()) == {-1}
    assert lo.tolist() == lens and no.tolist() == [nf]
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(f.cpu().numpy(), free)
    # a freed page id outside the pool: its row is not given a slot
    bad = free.copy()
    bad[:] = 10 ** 6
    good = sfa.kv4_plan(_i32([1, 0, 0]), _i32([0, 0, 0]), _cuda(table), _cuda(bad), _i32([1]), page=page, rows=2)
    assert good[1].tolist() == [-1, -1] and sfa.get_device_status() == 6


# ------------------------------------------------------------------ append and read


def _rows(rng, N, H, dtype):
    import torch

    x = rng.standard_normal((N, H, 64)) * np.exp(rng.standard_normal((1, H, 64)))
    return torch.from_numpy(x).to(_dt(dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,page,ks,vs,theta", [(1, 1, 16, 1.0, 1.0, 1e4), (33, 2, 64, 1.0, 0.5, 1e4), (100, 5, 32, 0.7, 1.3, 1e4),
                                                  (517, 3, 128, 1.0, 1.0, 0.0), (129, 8, 16, 2.0 ** -9, 1e3, 5e5)])
def test_append_bytes_and_read(sfa, dtype, N, H, page, ks, vs, theta):
    """Stored bytes and the numbers read back, exactly; other rows untouched; skipped rows skipped."""
    import torch

    rng = np.random.default_rng(N)
    P = -(-N // page) + 2
    slots = rng.permutation(P * page)[:N].astype(np.int32)
    T = 900
    pos = rng.integers(0, T, N).astype(np.int32)
    k, v = _rows(rng, N, H, dtype), _rows(rng, N, H, dtype)
    k[0, 0, :16] = 0  # a block of zeros, one too small for a scale, one beyond the largest
    v[0, 0, 16:32] *= 1e-6
    v[-1, -1, :16] *= 3e5
    if N > 3:
        slots[3] = -1
    table = torch.from_numpy(ref.rope(T, theta)).cuda() if theta else None
    old = rng.integers(0, 256, (P, H, 72 * page)).astype(np.uint8)
    want = old.copy()
    k32, v32 = k.float().numpy(), v.float().numpy()
    if theta:
        k32 = ref.rotate32(k32, ref.rope(T, theta)[pos])
    kq, vq = ref.quantise(k32 / np.float32(ks)), ref.quantise(v32 / np.float32(vs))
    for n in range(N):
        if slots[n] >= 0:
            ref.pack(want, page, int(slots[n]), (kq[0][n], kq[1][n]), (vq[0][n], vq[1][n]))
    cache = _cuda(old)
    sfa.kv4_append(k.cuda(), v.cuda(), cache, _i32(slots), _i32(pos), rope=table, rope_theta=0, kscale=ks, vscale=vs)
    assert sfa.get_device_status() == 0
    assert np.array_equal(cache.cpu().numpy(), want)
    for out in ("f32", "bf16"):
        gk, gv = sfa.kv4_read(cache, _i32(slots), dtype=_dt(out), kscale=ks, vscale=vs)
        wk, wv = ref.unpack(want, page, np.maximum(slots, 0))
        for g, w, s in ((gk, wk, ks), (gv, wv, vs)):
            w = torch.from_numpy((w.astype(np.float32) * np.float32(s)) * (slots >= 0)[:, None, None]).to(_dt(out))
            assert torch.equal(g.cpu(), w)


def test_append_special_numbers(sfa):
    """NaN poisons its block of 16, infinity saturates, signs and ties are kept."""
    import torch

    k = torch.zeros((1, 1, 64))
    k[0, 0, 0], k[0, 0, 5] = float("nan"), 3.0
    k[0, 0, 16], k[0, 0, 17] = float("inf"), 1.0
    k[0, 0, 32:48] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
    k[0, 0, 48:] = torch.tensor([6 * 2.0 ** -9] + [2.0 ** -9] * 15)
    cache = sfa.kv4_cache(1, 1, 16)
    sfa.kv4_append(k.cuda(), k.cuda(), cache, _i32([3]), _i32([0]), rope_theta=0)
    gk, gv = (x.cpu()[0, 0] for x in sfa.kv4_read(cache, _i32([3]), dtype=torch.float32))
    assert torch.equal(gk, gv) or torch.equal(gk.isnan(), gv.isnan())
    assert gk[:16].isnan().all()
    assert gk[16] == 448 * 6 and gk[17] == 0
    assert gk[32:48].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6, 0, -1, -1, -2, -2, -4, -4]
    assert gk[48:].tolist() == [6 * 2.0 ** -9] + [2.0 ** -9] * 15
    assert not gk[16:].isnan().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_strided_rows(sfa, dtype):
    """Keys and values as slices of one projection's rows."""
    import torch

    rng = np.random.default_rng(9)
    N, H, page = 50, 2, 16
    wide = torch.from_numpy(rng.standard_normal((N, 3 * H + 1, 64))).to(_dt(dtype)).cuda()
    k, v = wide[:, 1:1 + H], wide[:, 1 + H:1 + 2 * H]
    a, b = sfa.kv4_cache(5, H, page), sfa.kv4_cache(5, H, page)
    s, p = _i32(rng.permutation(80)[:N]), _i32(rng.integers(0, 70, N))
    sfa.kv4_append(k, v, a, s, p)
    sfa.kv4_append(k.contiguous(), v.contiguous(), b, s, p)
    assert torch.equal(a, b) and a.any()


def test_append_and_read_bad_index(sfa):
    """A slot or position out of range is reported and skipped."""
    import torch

    k = torch.ones((3, 1, 64), device="cuda")
    for slots, pos in (([0, 64, 2], [0, 1, 2]), ([0, 1, 2], [0, 64, 2]), ([0, 2 ** 31 - 1, 2], [0, 1, 2]), ([0, 1, 2], [0, -1, 2])):
        cache = sfa.kv4_cache(4, 1, 16)
        sfa.kv4_append(k, k, cache, _i32(slots), _i32(pos))
        assert sfa.get_device_status() == 6
        gk, gv = sfa.kv4_read(cache, _i32([0, 1, 2]), dtype=torch.float32)
        assert gv[0].all() and gv[2].all() and not gv[1].any() and not gk[1].any()
    gk, gv = sfa.kv4_read(cache, _i32([64, 0]), dtype=torch.float32)
    assert sfa.get_device_status() == 6 and not gk[0].any() and not gv[0].any() and gv[1].all()


# ------------------------------------------------------------------ attend


def make_cache(rng, lens, page, H, spare=2, garbage=True):
    """A pool whose requests' rows are quantised normal numbers; every other byte is what comes along
    (NaN scales among it)."""
    width = max([1] + [-(-n // page) for n in lens]) + 1
    table, _, _ = _pool(rng, lens, page, spare, width)
    P = sum(-(-n // page) for n in lens) + spare
    cache = rng.integers(0, 256, (P, H, 72 * page)).astype(np.uint8) if garbage else np.zeros((P, H, 72 * page), np.uint8)
    wide = np.exp(0.5 * rng.standard_normal((2, H, 64)))
    for r, n in enumerate(lens):
        x = rng.standard_normal((2, n, H, 64)) * wide[:, None]
        (kc, ks), (vc, vs) = ref.quantise(x[0].astype(np.float32)), ref.quantise(x[1].astype(np.float32))
        for p in range(n):
            ref.pack(cache, page, int(table[r, p // page]) * page + p % page, (kc[p], ks[p]), (vc[p], vs[p]))
    return cache, table


def stored(cache, table, r, n, page):
    return ref.unpack(cache, page, [int(table[r, p // page]) * page + p % page for p in range(n)])


def check_rows(o, lse, q, cache, table, lens, cu, page, dist, cs, ks, vs, bf16):
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    qn = q.double().cpu().numpy()
    for r, n in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        if b == a:
            continue
        if n == 0:
            assert not o[a:b].any() and np.isneginf(lse[a:b]).all()
            continue
        k, v = stored(cache, table, r, n, page)
        pos = np.arange(n - (b - a), n)
        wo, wl, av, sz = ref.attend(qn[a:b], k, v, pos, dist, ks, vs, cs)
        bo, bl = ref.bounds(wo, wl, av, sz, bf16)
        eo, el = np.abs(o[a:b] - wo), np.abs(lse[a:b] - wl)
        assert (eo <= bo).all(), (r, float((eo / bo).max()))
        assert (el <= bl).all(), (r, float((el / bl).max()))


CASES = [  # lens, new rows (None: one each), Hq, Hkv, page, dist
    ([1], None, 8, 2, 16, None),
    ([0, 1, 17, 0, 300], None, 8, 2, 16, None),
    ([64, 65, 63, 128, 1], None, 4, 4, 64, None),
    ([700, 5, 129], None, 16, 2, 128, None),
    ([257, 31], None, 32, 1, 32, None),
    ([50, 333], None, 16, 1, 16, None),
    ([1100, 3, 0, 988], None, 8, 2, 64, FIB),
    ([1500, 12], None, 6, 3, 16, CHRIST),
    ([700, 100], None, 8, 1, 32, list(range(300))),
    ([90, 40], None, 32, 1, 128, [0, 7, 30]),
    ([40, 9, 200], [40, 1, 33], 8, 2, 16, None),
    ([70, 33, 5, 300], [0, 33, 2, 7], 16, 2, 64, None),
    ([130, 260], [129, 70], 4, 4, 32, None),
    ([45, 80], [9, 17], 32, 1, 128, None),
    ([1200, 60], [50, 60], 8, 2, 64, FIB),
    ([400, 90], [21, 90], 16, 1, 16, list(range(0, 150))),
    ([333], [100], 2, 2, 16, [0, 1, 2, 64]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend(sfa, dtype, case):
    import torch

    lens, new, Hq, Hkv, page, dist = CASES[case]
    rng = np.random.default_rng(100 + case)
    cache, table = make_cache(rng, lens, page, Hkv)
    cu = np.concatenate([[0], np.cumsum(new if new else [1] * len(lens))])
    q = torch.from_numpy(1.5 * rng.standard_normal((cu[-1], Hq, 64))).to(_dt(dtype))
    cs = ref.rope(table.shape[1] * page) if case % 4 else None
    ks, vs = (1.0, 1.0) if case % 3 else (0.7, 1.3)
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu) if new else None, dist=dist,
                            rope=_cuda(cs) if cs is not None else None, rope_theta=0, kscale=ks, vscale=vs)
    assert sfa.get_device_status() == 0
    check_rows(o, lse, q, cache, table, lens, cu, page, dist, cs, ks, vs, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dist", [None, FIB])
def test_attend_long(sfa, dtype, dist):
    """Long and ragged prefixes: many pieces of one row, and rows that need none."""
    import torch

    rng = np.random.default_rng(7)
    lens, page, Hq, Hkv = [20011, 9, 3, 5000, 64], 64, 8, 2
    cache, table = make_cache(rng, lens, page, Hkv)
    q = torch.from_numpy(2 * rng.standard_normal((len(lens), Hq, 64))).to(_dt(dtype))
    cs = ref.rope(table.shape[1] * page)
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), dist=dist, rope=_cuda(cs))
    assert sfa.get_device_status() == 0
    check_rows(o, lse, q, cache, table, lens, list(range(6)), page, dist, cs, 1.0, 1.0, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 1), (32, 1), (4, 4)])
@pytest.mark.parametrize("new", [None, [3, 0, 4, 1, 2], [9, 0, 6, 1, 2]])
@pytest.mark.parametrize("dist", [None, list(range(700)), list(range(520)) + [530, 600, 1200]])
def test_attend_block_tables(sfa, dtype, Hq, Hkv, new, dist):
    """Few rows of up to 1400 keys under block tables of 1500, 3500 and 6500 rows, whose width and not the
    requests' lengths chooses how a row's keys are shared out."""
    import torch

    rng = np.random.default_rng(21)
    lens, page = [1400, 0, 513, 1, 90], 32
    cache, table = make_cache(rng, lens, page, Hkv)
    cu = np.concatenate([[0], np.cumsum(new if new else [1] * len(lens))])
    q = torch.from_numpy(1.5 * rng.standard_normal((cu[-1], Hq, 64))).to(_dt(dtype))
    c, cs = _cuda(cache), ref.rope(table.shape[1] * page)
    for rows in (1500, 3500, 6500):
        t = np.full((len(lens), rows // page), -1, np.int32)
        t[:, :table.shape[1]] = table
        o, lse = sfa.kv4_attend(q.cuda(), c, _cuda(t), _i32(lens), cu_q=_i32(cu) if new else None, dist=dist,
                                rope=_cuda(cs), rope_theta=0, vscale=1.3)
        assert sfa.get_device_status() == 0
        check_rows(o, lse, q, cache, table, lens, cu, page, dist, cs, 1.0, 1.3, dtype == "bf16")


@pytest.mark.parametrize("width", [60, 500])
@pytest.mark.parametrize("dist", [None, list(range(600)) + [640]])
def test_attend_few_rows_padded_nan_bad_pages(sfa, width, dist):
    """A few rows over more keys than a step sees: rows behind the last request stay as they were, NaN reaches
    its own rows only, pages outside the pool are reported and left out."""
    import torch

    rng = np.random.default_rng(24)
    lens, new, page = [900, 20, 7], [10, 0, 7], 16
    cache, table = make_cache(rng, lens, page, 2, garbage=False)
    t = np.full((3, width), -1, np.int32)
    t[:, :table.shape[1]] = table
    cu = _i32([0, 10, 10, 17])
    q = torch.from_numpy(rng.standard_normal((24, 8, 64))).float().cuda()
    o, lse = torch.full((24, 8, 64), 7.0, device="cuda"), torch.full((24, 8), 7.0, device="cuda")
    sfa.kv4_attend(q, _cuda(cache), _cuda(t), _i32(lens), cu_q=cu, dist=dist, rope_theta=0, o=o, lse=lse)
    assert sfa.get_device_status() == 0
    check_rows(o[:17], lse[:17], q[:17], cache, table, lens, [0, 10, 10, 17], page, dist, None, 1.0, 1.0, False)
    assert (o[17:] == 7).all() and (lse[17:] == 7).all()
    # a NaN in a value of the first request's key 895 (KV head 1, dims 16 .. 31): rows at 895 and later
    bad = cache.copy()
    bad[table[0, 895 // page], 1, 64 * page + 8 * (895 % page) + 4 + 1] = 127
    q2 = q.clone()
    q2[12, 3, 0] = float("nan")  # and in a query
    o2, l2 = sfa.kv4_attend(q2, _cuda(bad), _cuda(t), _i32(lens), cu_q=cu, dist=dist, rope_theta=0)
    want = torch.zeros((17, 8, 64), dtype=torch.bool)
    want[5:10, 4:, 16:32] = True
    want[12, 3] = True
    assert torch.equal(o2[:17].isnan().cpu(), want) and torch.equal(o2[:17][~want.cuda()], o[:17][~want.cuda()])
    # the first request's page of rows 320 .. 335 is nowhere: its rows without those keys
    t2 = t.copy()
    t2[0, 20] = cache.shape[0]
    o3, l3 = sfa.kv4_attend(q, _cuda(cache), _cuda(t2), _i32(lens), cu_q=cu, dist=dist, rope_theta=0)
    assert sfa.get_device_status() == 6 and torch.equal(o3[10:17], o[10:17]) and torch.equal(l3[10:17], lse[10:17])
    k, v = stored(cache, table, 0, 900, page)
    for row in (0, 9):
        p = 890 + row
        j = np.array([x for x in (range(p + 1) if dist is None else p - np.array(dist)) if x >= 0 and x // page != 20])
        wo, wl, av, sz = ref.attend(q[row:row + 1].double().cpu().numpy(), k, v, np.array([p]), sorted((p - j).tolist()), 1.0, 1.0, None)
        bo, bl = ref.bounds(wo, wl, av, sz, False)
        assert (np.abs(o3[row:row + 1].double().cpu().numpy() - wo) <= bo).all()
        assert (np.abs(l3[row:row + 1].double().cpu().numpy() - wl) <= bl).all()


@pytest.mark.parametrize("Hq,Hkv,dtype", [(8, 2, "f32"), (16, 1, "bf16"), (32, 1, "bf16")])
def test_attend_rows_do_not_depend_on_their_batch(sfa, Hq, Hkv, dtype):
    """One row a request: its bits are its own, whatever the other requests' lengths, block table of some
    chunks."""
    import torch

    rng = np.random.default_rng(25)
    lens, page = [5000, 6900, 2100, 300], 64
    cache, table = make_cache(rng, lens, page, Hkv)
    q = torch.from_numpy(rng.standard_normal((4, Hq, 64))).to(_dt(dtype)).cuda()
    args = (_cuda(cache), _cuda(table))
    rope = _cuda(ref.rope(table.shape[1] * page))
    o, lse = sfa.kv4_attend(q, *args, _i32(lens), rope=rope)
    for other in ([5000, 1, 0, 0], [5000, 6900, 2099, 299], [5000, 64, 2100, 17]):
        o2, l2 = sfa.kv4_attend(q, *args, _i32(other), rope=rope)
        for r in range(4):
            if other[r] == lens[r]:
                assert torch.equal(o[r], o2[r]) and torch.equal(lse[r], l2[r])
    assert sfa.get_device_status() == 0


def test_attend_sizes_of_queries(sfa):
    """Queries from the smallest to the largest: scaled by powers of two the result of a scaled
    kscale, bit for bit; zero queries average the values."""
    import torch

    rng = np.random.default_rng(8)
    lens, page = [130, 40], 16
    cache, table = make_cache(rng, lens, page, 2)
    args = (_cuda(cache), _cuda(table), _i32(lens))
    q = torch.from_numpy(rng.standard_normal((2, 8, 64))).float().cuda()
    o, lse = sfa.kv4_attend(q, *args)
    for e in (-100, -20, 20, 100):
        o2, l2 = sfa.kv4_attend(q * 2.0 ** e, *args, kscale=2.0 ** -e)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    o, lse = sfa.kv4_attend(q * 0, *args)
    for r, n in enumerate(lens):
        v = stored(cache, table, r, n, page)[1].mean(0)
        want = np.repeat(v, 4, axis=0)
        assert np.abs(o[r].double().cpu().numpy() - want).max() <= 2.0 ** -20 * np.abs(stored(cache, table, r, n, page)[1]).mean(0).max() * 2
        assert np.abs(lse[r].double().cpu().numpy() - np.log(n)).max() <= 2.0 ** -20
    assert sfa.get_device_status() == 0


@pytest.mark.parametrize("dist", [None, [0, 1, 2, 30]])
def test_attend_nan_stays_in_its_row(sfa, dist):
    """A NaN query or a NaN key reaches the rows that attend it and no others."""
    import torch

    rng = np.random.default_rng(11)
    lens, page = [100, 60, 31], 16
    cache, table = make_cache(rng, lens, page, 2, garbage=False)
    q = torch.from_numpy(rng.standard_normal((3, 4, 64))).float().cuda()
    clean, _ = sfa.kv4_attend(q, _cuda(cache), _cuda(table), _i32(lens), dist=dist)
    q2 = q.clone()
    q2[0, 1, 5] = float("nan")
    bad = cache.copy()
    bad[table[1, 59 // 16], 1, 64 * page + 8 * (59 % 16)] = 127  # a key's scale, KV head 1, last row
    o, lse = sfa.kv4_attend(q2, _cuda(bad), _cuda(table), _i32(lens), dist=dist)
    nan = torch.zeros((3, 4), dtype=torch.bool)
    nan[0, 1] = True
    nan[1, 2:] = True
    assert torch.equal(o.isnan().any(-1).cpu(), nan) and torch.equal(lse.isnan().cpu(), nan)
    assert torch.equal(o[~nan.cuda()], clean[~nan.cuda()])


@pytest.mark.parametrize("dist", [None, FIB])
def test_attend_padded_rows_and_strides(sfa, dist):
    """Rows behind the last request stay as they were; q may be slices of wider rows."""
    import torch

    rng = np.random.default_rng(12)
    lens, new, page = [90, 20, 7], [30, 0, 7], 16
    cache, table = make_cache(rng, lens, page, 2)
    cu = _i32([0, 30, 30, 37])
    wide = torch.from_numpy(rng.standard_normal((64, 14, 64))).to(torch.bfloat16).cuda()
    q = wide[:, 3:11]
    o = torch.full((64, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((64, 8), 7.0, device="cuda")
    sfa.kv4_attend(q, _cuda(cache), _cuda(table), _i32(lens), cu_q=cu, dist=dist, o=o, lse=lse)
    # the same capacity: the variant is chosen by the rows that a request brings on average
    o2, l2 = sfa.kv4_attend(q.contiguous(), _cuda(cache), _cuda(table), _i32(lens), cu_q=cu, dist=dist)
    assert torch.equal(o[:37], o2[:37]) and torch.equal(lse[:37], l2[:37])
    o3, l3 = sfa.kv4_attend(q[:37], _cuda(cache), _cuda(table), _i32(lens), cu_q=cu, dist=dist)
    cs = ref.rope(table.shape[1] * page)
    for got in ((o[:37], lse[:37]), (o3, l3)):
        check_rows(*got, q[:37], cache, table, lens, [0, 30, 30, 37], page, dist, cs, 1.0, 1.0, True)
    assert (o[37:] == 7).all() and (lse[37:] == 7).all()
    assert sfa.get_device_status() == 0


@pytest.mark.parametrize("dist", [None, [0, 5]])
def test_attend_bad_index(sfa, dist):
    """Lengths beyond the block table or the RoPE table, more rows than the length, page ids outside
    the pool: reported, and the other requests' rows are right."""
    import torch

    rng = np.random.default_rng(13)
    lens, page = [40, 33], 16
    cache, table = make_cache(rng, lens, page, 2)
    q = torch.from_numpy(rng.standard_normal((2, 8, 64))).float().cuda()
    c, good = _cuda(cache), sfa.kv4_attend(q, _cuda(cache), _cuda(table), _i32(lens), dist=dist)
    assert sfa.get_device_status() == 0
    for n in (-1, table.shape[1] * page + 1, 2 ** 31 - 1):
        o, lse = sfa.kv4_attend(q, c, _cuda(table), _i32([n, 33]), dist=dist)
        assert sfa.get_device_status() == 6
        assert torch.equal(o[1], good[0][1]) and not o[0].any() and torch.isneginf(lse[0]).all()
    o, lse = sfa.kv4_attend(q, c, _cuda(table), _i32(lens), dist=dist, rope=_cuda(ref.rope(39)))
    assert sfa.get_device_status() == 6 and torch.equal(o[1], good[0][1]) and not o[0].any()
    o, lse = sfa.kv4_attend(q, c, _cuda(table), _i32([1, 33]), cu_q=_i32([0, 2, 2]), dist=dist)
    assert sfa.get_device_status() == 6 and not o[0].any()
    for page_id in (-1, cache.shape[0], 2 ** 31 - 1):
        t2 = table.copy()
        t2[0, 2] = page_id
        o, lse = sfa.kv4_attend(q, c, _cuda(t2), _i32(lens), dist=dist)
        assert sfa.get_device_status() == 6 and torch.equal(o[1], good[0][1])


def test_offsets_past_32_bits(sfa):
    """Rows whose bytes lie beyond 4 GiB of the pool."""
    import torch

    H, page, P = 8, 128, 70000  # 5.2 GB
    cache = sfa.kv4_cache(P, H, page)
    k = torch.randn((2, H, 64), device="cuda")
    v = torch.randn((2, H, 64), device="cuda")
    slots = _i32([(P - 1) * page + 5, (P - 1) * page + 6])
    with pytest.raises(ValueError, match="rope_table"):
        sfa.kv4_append(k, v, cache, slots, _i32([5, 6]))
    sfa.kv4_append(k, v, cache, slots, _i32([5, 6]), rope=sfa.rope_table(64))
    gk, gv = sfa.kv4_read(cache, slots, dtype=torch.float32)
    assert (gv - v).abs().max() <= v.abs().max() / 6 * 1.0625 + 1e-6  # half of the widest step, and the scale's rounding
    small = sfa.kv4_cache(2, H, page)
    small[1] = cache[P - 1]
    q = torch.randn((1, 16, 64), device="cuda")
    for dist in (None, [0, 1]):
        a = sfa.kv4_attend(q, cache, _i32([P - 1])[None], _i32([7]), dist=dist)
        b = sfa.kv4_attend(q, small, _i32([1])[None], _i32([7]), dist=dist)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert sfa.get_device_status() == 0


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("dist", [None, FIB])
def test_serving_steps_together(sfa, dist):
    """A run as a server makes it: prompts, tokens, requests that end and others that start, each layer
    step plan -> append -> attend on a stream of its own, checked against plain code step by step."""
    import torch

    rng = np.random.default_rng(21)
    R, page, Hq, Hkv, width, P = 4, 16, 8, 2, 9, 24
    cs = ref.rope(width * page)
    rope = _cuda(cs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache = sfa.kv4_cache(P, Hkv, page)
    mirror = np.zeros(tuple(cache.shape), np.uint8)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    free = _i32(np.arange(P))
    lens, nf = _i32([0] * R), _i32([P])
    pool = ref.Pool(np.full((R, width), -1, np.int32), range(P), [0] * R, page)
    steps = [[40, 0, 17, 1], [1, 30, 1, 1], [1, 1, -1, 1], [1, 1, 60, 1], [-1, 3, 1, 0], [100, 1, 1, 1]]
    torch.cuda.synchronize()
    for new in steps:
        rows = sum(max(0, x) for x in new) + 3
        qkv = torch.from_numpy(rng.standard_normal((rows, Hq + 2 * Hkv, 64))).to(torch.bfloat16)
        cu, slots, pos = pool.step(new, rows)
        with torch.cuda.stream(side):
            d = qkv.cuda()
            g = sfa.kv4_plan(_i32(new), lens, table, free, nf, page=page, rows=rows, seq_lens_out=lens, n_free_out=nf)
            sfa.kv4_append(d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cache, g[1], g[2], rope=rope)
            o, lse = sfa.kv4_attend(d[:, :Hq], cache, table, lens, cu_q=g[0], dist=dist, rope=rope)
            side.synchronize()
            assert sfa.get_device_status() == 0
        assert g[0].tolist() == cu and g[1].tolist() == slots and lens.tolist() == pool.lens
        live = cu[-1]
        k32 = ref.rotate32(qkv[:live, Hq:Hq + Hkv].float().numpy(), cs[pos[:live]])
        kq, vq = ref.quantise(k32), ref.quantise(qkv[:live, Hq + Hkv:].float().numpy())
        for n in range(live):
            ref.pack(mirror, page, slots[n], (kq[0][n], kq[1][n]), (vq[0][n], vq[1][n]))
        assert np.array_equal(cache.cpu().numpy(), mirror)
        check_rows(o[:live], lse[:live], qkv[:live, :Hq], mirror, pool.table, pool.lens, cu, page, dist, cs, 1.0, 1.0, True)


@pytest.mark.parametrize("dist", [None, FIB])
def test_captured_decode_steps(sfa, dist):
    """One captured step (plan, append, attend), replayed: lengths, pages and results move on as in
    eager steps, bit for bit."""
    import torch

    rng = np.random.default_rng(22)
    R, page, Hq, Hkv, width, P = 5, 16, 8, 2, 8, 40
    rope = _cuda(ref.rope(width * page))
    start = [int(x) for x in rng.integers(1, 60, R)]
    xs = torch.from_numpy(rng.standard_normal((20, R, Hq + 2 * Hkv, 64))).to(torch.bfloat16).cuda()
    prompt = torch.from_numpy(rng.standard_normal((sum(start), Hq + 2 * Hkv, 64))).to(torch.bfloat16).cuda()

    def state():
        s = dict(cache=sfa.kv4_cache(P, Hkv, page), table=torch.full((R, width), -1, dtype=torch.int32, device="cuda"),
                 free=_i32(np.arange(P)), lens=_i32([0] * R), nf=_i32([P]), x=torch.zeros_like(xs[0]), new=_i32([1] * R))
        g = sfa.kv4_plan(_i32(start), s["lens"], s["table"], s["free"], s["nf"], page=page, rows=len(prompt), seq_lens_out=s["lens"], n_free_out=s["nf"])
        sfa.kv4_append(prompt[:, Hq:Hq + Hkv], prompt[:, Hq + Hkv:], s["cache"], g[1], g[2], rope=rope)
        return s

    def step(s):
        x = s["x"]
        g = sfa.kv4_plan(s["new"], s["lens"], s["table"], s["free"], s["nf"], page=page, rows=R, seq_lens_out=s["lens"], n_free_out=s["nf"])
        sfa.kv4_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], s["cache"], g[1], g[2], rope=rope)
        return sfa.kv4_attend(x[:, :Hq], s["cache"], s["table"], s["lens"], dist=dist, rope=rope)

    a, b = state(), state()
    torch.cuda.synchronize()
    step(state())  # first use outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            go, gl = step(b)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(20):
        a["x"].copy_(xs[i])
        b["x"].copy_(xs[i])
        o, lse = step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, go) and torch.equal(lse, gl)
        for n in ("cache", "table", "free", "lens", "nf"):
            assert torch.equal(a[n], b[n]), n
    assert sfa.get_device_status() == 0
    assert a["lens"].tolist() == [n + 20 for n in start]


@pytest.mark.parametrize("rows", [1, 40])
def test_attend_wait_that_runs_out(sfa, sfa_lib, rows):
    """A tile whose copies are never started: its wait runs out, the status says so, the call ends, and
    the next call is right (one row a request, and prompts)."""
    import torch

    rng = np.random.default_rng(14)
    lens, page = [3000, 700], 16
    cache, table = make_cache(rng, lens, page, 2)
    q = torch.from_numpy(rng.standard_normal((2 * rows, 8, 64))).float().cuda()
    args = (q, _cuda(cache), _cuda(table), _i32(lens))
    cu = _i32([0, rows, 2 * rows])
    good = sfa.kv4_attend(*args, cu_q=cu)
    torch.cuda.synchronize()
    try:
        for tile in (0, 1):
            assert sfa_lib.sfa_debug_inject(2000000, tile) == 0
            sfa.kv4_attend(*args, cu_q=cu)
            assert sfa.get_device_status() == 5  # SFA_ERR_TIMEOUT (the warp has two tiles)
    finally:
        sfa_lib.sfa_debug_inject(0, -1)
    again = sfa.kv4_attend(*args, cu_q=cu)
    assert sfa.get_device_status() == 0 and torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


def test_attend_wait_that_runs_out_before_other_units(sfa, sfa_lib):
    """A wait that runs out in the first of a CTA's pieces of prompts: those behind it are still told to the
    join, in a workspace that holds anything before."""
    import torch

    rng = np.random.default_rng(22)
    lens, new, page = [400] * 200, 70, 16
    cache, table = make_cache(rng, [400], page, 2)
    q = torch.from_numpy(rng.standard_normal((200 * new, 8, 64))).float().cuda()
    args = (q, _cuda(cache), _cuda(np.repeat(table, 200, 0)), _i32(lens))
    cu = _i32(np.arange(201) * new)
    n = sfa.kv4_workspace_size(*args[:3])
    good = sfa.kv4_attend(*args, cu_q=cu)
    torch.cuda.synchronize()
    try:
        assert sfa_lib.sfa_debug_inject(2000000, 0) == 0
        sfa.kv4_attend(*args, cu_q=cu, ws=torch.full((n,), 1, dtype=torch.uint8, device="cuda"))
        assert sfa.get_device_status() == 5  # SFA_ERR_TIMEOUT
    finally:
        sfa_lib.sfa_debug_inject(0, -1)
    again = sfa.kv4_attend(*args, cu_q=cu, ws=torch.full((n,), 1, dtype=torch.uint8, device="cuda"))
    assert sfa.get_device_status() == 0 and torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,new,Hq,Hkv,page,dist", [
    ([700, 300, 64], [200, 129, 64], 8, 2, 64, None),
    ([1000, 31, 500, 77], [33, 31, 500, 1], 16, 1, 16, None),
    ([2500, 900], [300, 64], 4, 4, 128, None),
    ([900, 70], [40, 70], 32, 1, 32, None),
    ([1500, 130, 600], [100, 130, 64], 8, 2, 32, list(range(200))),
    ([1, 300, 128], [1, 300, 128], 8, 1, 16, list(range(65))),
])
def test_attend_prompts(sfa, dtype, lens, new, Hq, Hkv, page, dist):
    """Pieces of prompts, long enough for the tensor memory kernel: columns that fill their items and
    do not, prefixes that are split and are not, windows."""
    import torch

    rng = np.random.default_rng(len(lens) + page)
    cache, table = make_cache(rng, lens, page, Hkv)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = torch.from_numpy(2 * rng.standard_normal((cu[-1], Hq, 64))).to(_dt(dtype))
    cs = ref.rope(table.shape[1] * page)
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu), dist=dist, rope=_cuda(cs), kscale=0.7)
    assert sfa.get_device_status() == 0
    check_rows(o, lse, q, cache, table, lens, cu, page, dist, cs, 0.7, 1.0, dtype == "bf16")


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("dist", [None, list(range(90))])
def test_attend_nan_value_among_rows(sfa, rows, dist):
    """A stored NaN in a value block reaches those rows that attend its key, in that block's dims, and
    no others, whatever shares a tile with it."""
    import torch

    rng = np.random.default_rng(15)
    n, page = 200, 16
    cache, table = make_cache(rng, [n], page, 2, garbage=False)
    q = torch.from_numpy(rng.standard_normal((rows, 8, 64))).float().cuda()
    args = (_cuda(table), _i32([n]))
    cu = _i32([0, rows])
    clean, lse = sfa.kv4_attend(q, _cuda(cache), *args, cu_q=cu, dist=dist)
    key = n - 2 if rows == 3 else n - 35
    for old in (key, n - rows - 60):
        cache[table[0, old // page], 1, 64 * page + 8 * (old % page) + 4 + 2] = 127  # KV head 1, dims 32 .. 47
    o, lse2 = sfa.kv4_attend(q, _cuda(cache), *args, cu_q=cu, dist=dist)
    pos = np.arange(n - rows, n)
    W = n if dist is None else len(dist) - 1
    hit = np.zeros(rows, bool)
    for old in (key, n - rows - 60):
        hit |= (old <= pos) & (old >= pos - W)
    assert hit.any() and (rows == 3 or dist is None or not hit.all())
    want = torch.zeros((rows, 8, 64), dtype=torch.bool)
    want[torch.from_numpy(hit), 4:, 32:48] = True
    assert torch.equal(o.isnan().cpu(), want)
    assert torch.equal(o[~want.cuda()], clean[~want.cuda()]) and torch.equal(lse, lse2)
    assert sfa.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,Hq,dist", [(1, 8, None), (1, 8, [0, 3, 60]), (3, 8, list(range(70))), (6, 8, list(range(200))),
                                         (80, 8, list(range(200))), (80, 8, None), (33, 8, [0, 1, 5])])
def test_attend_far_below_zero(sfa, dtype, new, Hq, dist):
    """All logits equal and far below zero (-800), rows of a tile reaching their first key in different steps: the
    mean of the values, as with any other logit."""
    import torch

    rng = np.random.default_rng(16)
    n, page, Hkv = 900, 64, 2
    cache, table = make_cache(rng, [n], page, Hkv)
    code, s8 = ref.quantise(np.full((n, Hkv, 64), -2.0, np.float32))
    for p in range(n):
        cache[table[0, p // page], :, 32 * (p % page):][:, :32] = code[p, :, 0::2] | (code[p, :, 1::2] << 4)
        cache[table[0, p // page], :, 64 * page + 8 * (p % page):][:, :4] = s8[p]
    k, v = stored(cache, table, 0, n, page)
    assert (k == k[0, 0, 0]).all()
    q = torch.full((new, Hq, 64), 50.0, dtype=_dt(dtype))
    for spare in (0, 100):  # columns of the block table
        t = np.pad(table, ((0, 0), (0, spare)), constant_values=-1)
        o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(t), _i32([n]), cu_q=_i32([0, new]), dist=dist, rope_theta=0)
        assert sfa.get_device_status() == 0
        check_rows(o, lse, q, cache, table, [n], [0, new], page, dist, None, 1.0, 1.0, dtype == "bf16")
        assert (lse < -700).all()


@pytest.mark.parametrize("new", [1, 5, 90])
def test_attend_captured(sfa, new):
    """A captured call (one that splits its rows, with its workspace from the graph's own memory), replayed
    with other queries and lengths, gives the eager call's bits; two graphs replayed at once on two streams
    do not disturb each other."""
    import torch

    rng = np.random.default_rng(17)
    lens, page, R = [2000, 900, 130], 32, 3
    cache, table = make_cache(rng, lens, page, 2)
    c, t, rope = _cuda(cache), _cuda(table), sfa.rope_table(table.shape[1] * page)
    cu = _i32(np.arange(R + 1) * new) if new > 1 else None
    made = []
    for i in range(2):
        q = torch.zeros((R * new, 8, 64), dtype=torch.bfloat16, device="cuda")
        n = _i32(lens)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                got = sfa.kv4_attend(q, c, t, n, cu_q=cu, rope=rope)
        made.append((q, n, side, graph, got))
    for step in range(4):
        want = []
        for i, (q, n, side, graph, got) in enumerate(made):
            q.copy_(torch.from_numpy(rng.standard_normal(tuple(q.shape))))
            n.copy_(_i32([x - 7 * step - i for x in lens]))
            want.append(sfa.kv4_attend(q, c, t, n, cu_q=cu, rope=rope))
        torch.cuda.synchronize()
        for _ in range(5):
            for q, n, side, graph, got in made:
                with torch.cuda.stream(side):
                    graph.replay()
        torch.cuda.synchronize()
        for w, (q, n, side, graph, got) in zip(want, made):
            assert torch.equal(w[0], got[0]) and torch.equal(w[1], got[1])
    assert sfa.get_device_status() == 0
    # a table that a call would have to make first is refused inside a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="before the capture"):
            sfa.kv4_attend(q, c, t, n, cu_q=cu, rope_theta=12345.0)
        q.add_(0)


def test_attend_on_another_stream(sfa):
    """Inputs made on one stream and used on another that waits for it; the default stream's table is shared."""
    import torch

    rng = np.random.default_rng(18)
    lens, page = [700, 40], 16
    cache, table = make_cache(rng, lens, page, 2)
    q = torch.from_numpy(rng.standard_normal((2, 8, 64))).float().cuda()
    args = (_cuda(cache), _cuda(table), _i32(lens))
    want = sfa.kv4_attend(q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q2 = q * 2
        got = sfa.kv4_attend(q2 / 2, *args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_python_refusals(sfa):
    """Wrong types, shapes, strides and devices are refused before anything is launched."""
    import torch

    cache, table = sfa.kv4_cache(4, 2, 16), torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    lens = _i32([1, 1, 1])
    q = torch.zeros((3, 8, 64), device="cuda")
    ok = lambda **kw: sfa.kv4_attend(kw.pop("q", q), kw.pop("cache", cache), kw.pop("table", table), kw.pop("lens", lens), **kw)  # noqa: E731
    ok()
    with pytest.raises(TypeError):
        ok(q=q.half())
    for kw in (dict(q=q[:, :, :32]), dict(q=q[0]), dict(q=q.transpose(0, 1)), dict(q=torch.zeros((3, 8, 128), device="cuda")[:, :, ::2]),
               dict(q=torch.zeros((3, 8 * 64 + 1), device="cuda")[:, :512].unflatten(1, (8, 64))), dict(q=q.cpu()), dict(cache=cache[:, :, :100]),
               dict(cache=cache.int()), dict(table=table.long()), dict(table=table.t()), dict(table=table.cpu()), dict(lens=lens[:2]),
               dict(lens=lens.float()), dict(cu_q=lens), dict(cu_q=_i32([0, 1, 2, 3]).long()), dict(kscale=0.0), dict(vscale=float("nan")),
               dict(o=torch.zeros((3, 8, 64), dtype=torch.bfloat16, device="cuda")), dict(lse=torch.zeros((3, 7), device="cuda")),
               dict(rope=torch.zeros((5, 32), device="cuda")), dict(rope=torch.zeros((5, 32, 2), dtype=torch.float64, device="cuda")), dict(q=q[:2])):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(dist=[1, 2]), dict(dist=[0, -1]), dict(dist=list(range(0, 1000, 2))), dict(q=torch.zeros((3, 7, 64), device="cuda"))):
        with pytest.raises(sfa.SfaError):
            ok(**kw)
    k = torch.zeros((3, 2, 64), device="cuda")
    for a in ((k, k.bfloat16(), cache, lens, lens), (k, k[:2], cache, lens, lens), (k, k, cache, lens[:2], lens), (k, k, cache, lens, lens.float()),
              (k[:, :1], k[:, :1], cache, lens, lens)):
        with pytest.raises(ValueError):
            sfa.kv4_append(*a)
    with pytest.raises(ValueError):
        sfa.kv4_read(cache, lens, k=k, v=k[:2])
    free = _i32([0, 1, 2, 3])
    for a in ((lens[:2], lens, table, free, lens[:1]), (lens, lens, table, free, lens), (lens, lens, table.long(), free, lens[:1])):
        with pytest.raises(ValueError):
            sfa.kv4_plan(*a, page=16, rows=4)
    with pytest.raises(ValueError):
        sfa.kv4_plan(lens, lens, table, free, lens[:1], page=16, rows=-1)
    with pytest.raises(sfa.SfaError):
        sfa.kv4_plan(lens, lens, table, free, lens[:1], page=17, rows=4)
    # nothing to do is no error
    assert sfa.kv4_attend(q[:0], cache, table[:0], lens[:0])[0].shape == (0, 8, 64)
    sfa.kv4_append(k[:0], k[:0], cache, lens[:0], lens[:0])
    assert sfa.kv4_read(cache, lens[:0])[0].shape == (0, 2, 64)
    assert sfa.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,dist", [(8, 2, FIB), (4, 4, [0, 1, 2, 5, 40]), (4, 2, [0]), (2, 2, list(range(32))), (8, 2, [0, 300])])
def test_attend_many_rows_of_few_keys(sfa, dtype, Hq, Hkv, dist):
    """Enough rows that several share a warp's columns: rows of one request and of neighbours, requests
    without rows, rows without all their keys, a stored NaN value among them, an odd number of rows and
    rows behind the last."""
    import torch

    rng = np.random.default_rng(19)
    page = 16
    lens = [1700 // Hkv, 5, 0, 900, 40, 2400 // Hkv]
    new = [1650 // Hkv, 5, 0, 33, 1, 1500 // Hkv]
    cache, table = make_cache(rng, lens, page, Hkv, garbage=True)
    nan_at = lens[0] - 100  # request 0, KV head 0, dims 16 .. 31
    cache[table[0, nan_at // page], 0, 64 * page + 8 * (nan_at % page) + 5] = 127
    cu = np.concatenate([[0], np.cumsum(new)])
    N = int(cu[-1]) + 60
    q = torch.from_numpy(rng.standard_normal((N, Hq, 64))).to(_dt(dtype))
    cs = ref.rope(table.shape[1] * page)
    o = torch.full((N, Hq, 64), 3.0, dtype=_dt(dtype), device="cuda")
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu), dist=dist, rope=_cuda(cs), o=o)
    assert sfa.get_device_status() == 0
    assert N * Hkv > 3040 and (o[cu[-1]:] == 3).all()
    G = Hq // Hkv
    pos = np.arange(lens[0] - new[0], lens[0])
    hit = np.isin(pos - nan_at, dist)
    assert hit.any()
    want = torch.zeros((N, Hq, 64), dtype=torch.bool)
    want[torch.from_numpy(np.flatnonzero(hit)), :G, 16:32] = True
    assert torch.equal(o.isnan().cpu(), want)
    clean = cache.copy()
    clean[table[0, nan_at // page], 0, 64 * page + 8 * (nan_at % page) + 5] = 0  # what the other dims see of it
    o = torch.where(want.cuda(), torch.zeros_like(o), o)
    on, qn = o.double().cpu().numpy(), q.double().numpy()
    for r, n in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        if a == b:
            continue
        k, v = stored(clean, table, r, n, page)
        wo, wl, av, sz = ref.attend(qn[a:b], k, v, np.arange(n - (b - a), n), dist, 1.0, 1.0, cs)
        bo, bl = ref.bounds(wo, wl, av, sz, dtype == "bf16")
        wo[want[a:b].numpy()] = 0
        assert (np.abs(on[a:b] - wo) <= bo).all() and (np.abs(lse[a:b].double().cpu().numpy() - wl) <= bl).all(), r


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2)])
def test_attend_many_tokens_of_few_keys(sfa, Hq, Hkv):
    """One row a request, more requests than a wave: the same rows as a call for a few of them, bit for bit or within
    the bound (other rows in a tile do not change a row's sums, only their order)."""
    import torch

    rng = np.random.default_rng(20)
    R, page = 1601 if Hkv == 2 else 1700, 16
    lens = [int(x) for x in rng.integers(0, 60, R)]
    cache, table = make_cache(rng, lens, page, Hkv)
    q = torch.from_numpy(rng.standard_normal((R, Hq, 64))).float()
    cs = ref.rope(table.shape[1] * page)
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), dist=[0, 1, 2, 3, 8, 33], rope=_cuda(cs))
    assert sfa.get_device_status() == 0
    check_rows(o, lse, q, cache, table, lens, list(range(R + 1)), page, [0, 1, 2, 3, 8, 33], cs, 1.0, 1.0, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_native_calls_and_ctypes_calls(sfa, dtype, monkeypatch):
    """A step's four calls through the native binding and without it: the same bits, the same tensors handed
    through, on the caller's stream, slices of wider rows, outputs given or made."""
    import torch
    from static_offset_sparse_gb300 import kv4

    native = kv4._native()
    assert native is not None
    rng = np.random.default_rng(23)
    page, R, P = 16, 3, 40
    rope = sfa.rope_table(160)
    wide = torch.from_numpy(rng.standard_normal((2, 61, 14, 64))).to(_dt(dtype)).cuda()
    out = []
    for use in (native, None):
        calls = []
        if use is not None:
            class Counted:
                def __getattr__(self, name):
                    def call(*a):
                        r = getattr(native, name)(*a)
                        calls.append((name, r is not None))
                        return r
                    return call
            monkeypatch.setattr(kv4, "_native", lambda: counted)
            counted = Counted()
        else:
            monkeypatch.setattr(kv4, "_native", lambda: None)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = []
        with torch.cuda.stream(side):
            cache = sfa.kv4_cache(P, 2, page)
            table, free = _i32(np.full((R, 10), -1)), _i32(np.arange(P))
            lens, nf = _i32([0] * R), _i32([P])
            for step, new in enumerate(([60, 0, 1], [2, 30, 17])):
                qkv = wide[step]
                given = dict(seq_lens_out=lens, n_free_out=nf) if step else {}
                cu, slots, pos, l2, n2 = sfa.kv4_plan(_i32(new), lens, table, free, nf, page=page, rows=61, **given)
                if step:
                    assert l2 is lens and n2 is nf
                lens, nf = l2, n2
                sfa.kv4_append(qkv[:, 8:10], qkv[:, 11:13], cache, slots, pos, rope=rope, kscale=0.5)
                k, v = sfa.kv4_read(cache, slots, dtype=_dt(dtype), kscale=0.5)
                o, lse = torch.zeros((61, 8, 64), dtype=_dt(dtype), device="cuda"), torch.zeros((61, 8), device="cuda")
                a = (qkv[:, :8], cache, table, lens)
                r = sfa.kv4_attend(*a, cu_q=cu, rope=rope, kscale=0.5, o=o, lse=lse)
                assert r[0] is o and r[1] is lse
                o2, l2 = sfa.kv4_attend(*a, cu_q=cu, rope=rope, kscale=0.5, dist=[0, 1, 2, 5, 40])
                last = (cu[1:].long() - 1).clamp(min=0)
                o3, l3 = sfa.kv4_attend(qkv[last, :8], cache, table, lens, rope_theta=0)
                if step and use is not None:  # a table by its theta: made by the first call, found by the second
                    a3, before = (qkv[last, :8], cache, table, lens), len(calls)
                    theta = 777.0 if dtype == "f32" else 555.0
                    sfa.kv4_attend(*a3, rope_theta=theta)
                    o4, l4 = sfa.kv4_attend(*a3, rope_theta=theta)
                    o5, l5 = sfa.kv4_attend(*a3, rope=sfa.rope_table(160, theta))
                    assert calls[before:] == [("attend", True)] * 2 and torch.equal(o4, o5) and torch.equal(l4, l5)
                    del calls[before:]
                n = sum(new)
                got += [t.clone() for t in (cu, slots, pos, lens, nf, table, free[:int(nf)], cache, k, v, o[:n], lse[:n], o2[:n], l2[:n], o3, l3)]
        side.synchronize()
        out.append(got)
        if use is not None:
            assert len(calls) == 12 and all(took for _, took in calls), calls
    for a, b in zip(*out):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
    # what is not in order goes the long way, with its reasons
    monkeypatch.setattr(kv4, "_native", lambda: native)
    q = wide[0][:3, :8]
    assert native.attend(q, cache, table, lens, None, None, None, 1, 1.0, None, None, None) is None
    assert native.attend(q.cpu(), cache, table, lens, None, None, None, 1.0, 1.0, None, None, None) is None
    assert native.attend(q, cache, table, lens[:2], None, None, None, 1.0, 1.0, None, None, None) is None
    for bad in (dict(kscale=0.0), dict(vscale=float("nan")), dict(rope=rope[:, :16]), dict(lse=lse.double())):
        with pytest.raises(ValueError):
            sfa.kv4_attend(q, cache, table, lens, **{"rope": rope, **bad})
    with pytest.raises((ValueError, RuntimeError)):
        sfa.kv4_attend(q[:, :6], cache, table, lens, rope=rope)  # 3 heads a KV head

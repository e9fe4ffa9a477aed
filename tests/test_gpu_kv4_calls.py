"""The paged 4-bit cache's calls as programs make them: tables made elsewhere, calls back to back, rows out of
range among rows in range, batches that keep every team busy for several chunks."""
import threading

import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import FIB, _cuda, _dt, _i32, check_rows, make_cache, sfa, stored  # noqa: F401 (sfa: the fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the RoPE table that a call finds


def _small(sfa, seed, width=None):
    import torch

    rng = np.random.default_rng(seed)
    lens, page = [300, 77], 16
    cache, table = make_cache(rng, lens, page, 2)
    if width:
        table = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
    q = torch.from_numpy(rng.standard_normal((2, 8, 64))).float()
    return (q.cuda(), _cuda(cache), _cuda(table), _i32(lens)), (q, cache, table, lens, [0, 1, 2], page)


def _right(sfa, got, plain, theta):
    q, cache, table, lens, cu, page = plain
    check_rows(*got, q, cache, table, lens, cu, page, None, ref.rope(table.shape[1] * page, theta), 1.0, 1.0, False)


def test_table_made_on_a_busy_stream(sfa):
    """rope_table on a stream with work ahead of it, then a call without rope= on one that waits for nothing."""
    import torch

    args, plain = _small(sfa, 31)
    T, theta = plain[2].shape[1] * plain[5], 4321.0
    sfa.rope_table(T, 1e3)
    sfa.kv4_attend(*args, rope_theta=1e3)  # kernels are loaded, which waits for the device
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        spoiled = torch.full((1024, 32, 2), float("nan"), device="cuda")  # what the table's memory held before
        del spoiled
        torch.cuda._sleep(200_000_000)
        sfa.rope_table(T, theta)
    with torch.cuda.stream(b):
        got = sfa.kv4_attend(*args, rope_theta=theta)
    torch.cuda.synchronize()
    _right(sfa, got, plain, theta)


def test_table_of_a_capture(sfa):
    """forward in a capture makes a table that only replays fill: an eager call of its length makes its own,
    and the graph's replays are right whatever was captured beside it."""
    import torch

    args, plain = _small(sfa, 32)
    T, theta = plain[2].shape[1] * plain[5], 8765.0
    rng = np.random.default_rng(5)
    q, k, v = (torch.from_numpy(rng.standard_normal((1, h, T, 64))).to(torch.bfloat16).cuda() for h in (8, 2, 2))
    sfa.forward_int(q, k, v, dist=FIB)  # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = sfa.forward_int(q, k, v, dist=FIB, rope_theta=theta)
        o2, _ = sfa.forward_int(o, k, v, dist=FIB, rope_theta=theta)
    got = sfa.kv4_attend(*args, rope_theta=theta)
    torch.cuda.synchronize()
    _right(sfa, got, plain, theta)
    graph.replay()
    torch.cuda.synchronize()
    wo, wl = sfa.forward_int(q, k, v, dist=FIB, rope_theta=theta)
    assert torch.equal(o, wo) and torch.equal(lse, wl)
    assert torch.equal(o2, sfa.forward_int(wo, k, v, dist=FIB, rope_theta=theta)[0])
    assert sfa.get_device_status() == 0


def test_first_calls_of_two_threads(sfa):
    """Two threads with a stream each, both first to want a table."""
    import torch

    args, plain = _small(sfa, 33)
    torch.cuda.synchronize()
    for theta in (1234.5, 2345.5, 3456.5, 4567.5):
        got, gate = [None, None], threading.Barrier(2)

        def call(i):
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                torch.cuda._sleep(2_000_000)
                gate.wait()
                got[i] = sfa.kv4_attend(*args, rope_theta=theta)
                stream.synchronize()

        threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        for g in got:
            _right(sfa, g, plain, theta)


def test_tables_of_growing_block_tables(sfa):
    """Block tables of many widths: the same rotations, a table shared by all of them, the cache's memory within
    a few times the longest."""
    import torch
    from static_offset_sparse_gb300 import api

    theta = 6543.0
    args, plain = _small(sfa, 34)
    want = sfa.kv4_attend(*args, rope=_cuda(ref.rope(3000, theta)))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for width in range(args[2].shape[1], 400):
        t = torch.nn.functional.pad(args[2], (0, width - args[2].shape[1]), value=-1)
        got = sfa.kv4_attend(args[0], args[1], t, args[3], rope_theta=theta)
    del t
    _right(sfa, got, plain, theta)
    assert torch.cuda.memory_allocated() - before < 4 * 6400 * 256
    tab = sfa.rope_table(6390, theta)
    assert tab.is_contiguous() and torch.equal(sfa.rope_table(100, theta), tab[:100])
    assert np.abs(tab.double().cpu().numpy() - ref.rope(6390, theta)).max() <= 2.0 ** -23
    assert len({x.untyped_storage().data_ptr() for (n, th, i), x in api._ROPE_CACHE.items() if th == theta}) <= 4
    assert torch.equal(want[1].isfinite(), got[1].isfinite())


# ------------------------------------------------------------------ calls back to back


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,width,Hq", [(1, 700, 8), (3, 700, 16), (40, 300, 8)])
def test_calls_with_other_inputs_in_turn(sfa, dtype, new, width, Hq):
    """Calls that split their rows, two inputs in turn over one workspace, nothing between them: each gives its
    own result again.  (A kernel starts while the one before it writes what it will read.)"""
    import torch

    rng = np.random.default_rng(41)
    page, R = 64, 3
    inputs = []
    for lens in ([9000, 5000, 700], [8000, 9100, 41]):
        cache, table = make_cache(rng, lens, page, 2)
        table = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
        q = torch.from_numpy(rng.standard_normal((R * new, Hq, 64))).to(_dt(dtype)).cuda()
        inputs.append((q, _cuda(cache), _cuda(table), _i32(lens)))
    cu = _i32(np.arange(R + 1) * new) if new > 1 else None
    n = max(sfa.kv4_workspace_size(*x[:3]) for x in inputs)
    assert n > 0
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
    want = [sfa.kv4_attend(*x, cu_q=cu, rope_theta=0) for x in inputs]
    out = [[(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for w in want] for _ in range(10)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for turn in out:
            for x, (o, lse) in zip(inputs, turn):
                sfa.kv4_attend(*x, cu_q=cu, rope_theta=0, ws=ws, o=o, lse=lse)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for turn in out:
            for w, got in zip(want, turn):
                assert torch.equal(w[0], got[0]) and torch.equal(w[1], got[1])
                got[0].zero_()
    assert sfa.get_device_status() == 0


@pytest.mark.parametrize("R,dist", [(5, None), (5, FIB), (60, FIB), (900, [0, 1, 2, 5])])
def test_rows_written_by_the_call_before(sfa, R, dist):
    """append and attend in turn over the same slots, two contents in turn: attention reads what the call just
    before it wrote."""
    import torch

    rng = np.random.default_rng(42)
    page, lens = 16, [20] * R
    cache, table = make_cache(rng, lens, page, 2)
    c, t, n = _cuda(cache), _cuda(table), _i32(lens)
    q = torch.from_numpy(rng.standard_normal((R, 8, 64))).to(torch.bfloat16).cuda()
    slots = _i32([int(table[r, p // page]) * page + p % page for r in range(R) for p in range(20)])
    pos = _i32([p for r in range(R) for p in range(20)])
    kv = [torch.from_numpy(rng.standard_normal((2, R * 20, 2, 64))).to(torch.bfloat16).cuda() for _ in range(2)]
    want = []
    for x in kv:
        sfa.kv4_append(x[0], x[1], c, slots, pos, rope_theta=0)
        torch.cuda.synchronize()
        want.append(sfa.kv4_attend(q, c, t, n, dist=dist, rope_theta=0))
        torch.cuda.synchronize()
    out = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            for x in kv:
                sfa.kv4_append(x[0], x[1], c, slots, pos, rope_theta=0)
                out.append(sfa.kv4_attend(q, c, t, n, dist=dist, rope_theta=0))
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for i, got in enumerate(out):
            assert torch.equal(want[i % 2][0], got[0]) and torch.equal(want[i % 2][1], got[1]), i
    assert not torch.equal(want[0][0], want[1][0]) and sfa.get_device_status() == 0


# ------------------------------------------------------------------ numbers at the ends of their range


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,width,dist", [(1, 30, [0, 1, 7, 200]), (1, 80, None), (1, 200, None), (3, 200, None), (6, 200, None),
                                            (40, 60, None), (40, 60, list(range(70)))])
@pytest.mark.parametrize("kscale", [1e-7, 1e-20, 2.0 ** -126, 2.0 ** -140])
def test_attend_small_kscale(sfa, dtype, new, width, dist, kscale):
    """Zero and tiny queries times a small kscale: a masked key stays masked, whichever kernel the
    call goes to (gather, cluster, stream with one to four column tiles, prompts)."""
    import torch

    rng = np.random.default_rng(51)
    lens, page, Hq = [500, 130, 41], 32, 8
    cache, table = make_cache(rng, lens, page, 2)
    table = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
    cu = np.arange(len(lens) + 1) * new
    q = torch.from_numpy(rng.standard_normal((cu[-1], Hq, 64)))
    q[::2] *= 0
    q[:, 1] *= 2.0 ** -110
    q = q.to(_dt(dtype))
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu) if new > 1 else None, dist=dist, rope_theta=0,
                            kscale=kscale)
    assert sfa.get_device_status() == 0
    check_rows(o, lse, q, cache, table, lens, cu, page, dist, None, float(np.float32(kscale)), 1.0, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,width,dist", [(1, 30, [0, 1, 7, 200]), (1, 80, None), (1, 200, None), (3, 200, None), (6, 200, None),
                                            (40, 60, None), (40, 60, list(range(70)))])
@pytest.mark.parametrize("kscale", [1.0, 1e-7])
def test_attend_large_queries(sfa, dtype, new, width, dist, kscale):
    """Logits of any size, far beyond those that fp32 can tell apart by less than 1: finite results, and where one key
    stands out by more than the logits' error, its value alone, whichever kernel the call goes to."""
    import torch

    rng = np.random.default_rng(52)
    lens, page, Hq = [500, 130, 41], 32, 8
    cache, table = make_cache(rng, lens, page, 2)
    padded = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
    cu = np.arange(len(lens) + 1) * new
    q = torch.from_numpy(rng.standard_normal((cu[-1], Hq, 64)))
    q *= torch.tensor([2.0 ** e for e in (16, 21, 23, 24, 25, 27, 60, 100)])[None, :, None]
    q = q.to(_dt(dtype))
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(padded), _i32(lens), cu_q=_i32(cu) if new > 1 else None, dist=dist, rope_theta=0,
                            kscale=kscale)
    assert sfa.get_device_status() == 0
    ks, alone, bf16 = float(np.float32(kscale)), 0, dtype == "bf16"
    # Probabilities are whole f16 steps of 2^-24 at least (fp32 outputs: their second part is), while the largest of a
    # column is 2^8 or more (bf16 prompts; 2^11 else), and so is the sum: half a step of each key's is 2^-33 (2^-36 for
    # fp32 outputs) of its value.  It counts where the key that stands out has a zero and the others all but no weight.
    floor = 2.0 ** (-33 if bf16 else -36)
    on, ln, qn = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    for r, n in enumerate(lens):
        k, v = stored(cache, table, r, n, page)
        a, b = cu[r], cu[r + 1]
        pos = np.arange(n - (b - a), n)
        wo, wl, av, sz = ref.attend(qn[a:b], k, v, pos, dist, ks, 1.0, None)
        bo, bl = ref.bounds(wo, wl, av, sz, bf16)
        for i, p in enumerate(pos):
            js = np.arange(p + 1) if dist is None else np.array([p - s for s in dist if s <= p])
            limit = bo[i] + floor * np.repeat(np.abs(v[js]).sum(0), 4, 0)
            assert (np.abs(on[a + i] - wo[i]) <= limit).all(), (r, i, float((np.abs(on[a + i] - wo[i]) / limit).max()))
            assert (np.abs(ln[a + i] - wl[i]) <= bl[i]).all(), (r, i)
            for h in range(Hq):
                t = k[js, h // 4] * ks @ qn[a + i, h] / 8
                two = np.sort(t)[-2:]
                if len(t) > 1 and two[1] - two[0] > 4 * 2.0 ** -18.5 * sz[i, h] + 40:  # the others' weights: below 2^-57
                    alone += 1
                    assert np.array_equal(on[a + i, h], v[js[t.argmax()], h // 4])
    assert alone > 2 * new


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,width,dist", [(1, 4, [0, 1]), (1, 300, None), (3, 300, None), (40, 30, None)])
def test_lse_of_few_small_logits(sfa, dtype, new, width, dist):
    """Thousands of log-sum-exps of a few logits near zero, where the largest terms cancel: within the bound, and
    without a bias (an eighth of it)."""
    import torch

    rng = np.random.default_rng(53)
    R, page = 400, 16
    lens = [int(x) for x in rng.integers(new, new + 4, R)]
    cache, table = _shared_pages(rng, lens, page, 2, width)
    cu = np.arange(R + 1) * new
    q = torch.from_numpy(0.3 * rng.standard_normal((R * new, 8, 64))).to(_dt(dtype))
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu) if new > 1 else None, dist=dist, rope_theta=0,
                            kscale=0.01)
    assert sfa.get_device_status() == 0
    ln, qn, off = lse.double().cpu().numpy(), q.double().numpy(), []
    for r, n in enumerate(lens):
        k, v = stored(cache, table, r, n, page)
        a, b = cu[r], cu[r + 1]
        wo, wl, av, sz = ref.attend(qn[a:b], k, v, np.arange(n - new, n), dist, float(np.float32(0.01)), 1.0, None)
        bl = ref.bounds(wo, wl, av, sz, dtype == "bf16")[1]
        off.append(((ln[a:b] - wl) / bl).ravel())
    off = np.concatenate(off)
    assert np.abs(off).max() <= 1, float(np.abs(off).max())
    assert abs(off.mean()) <= 1 / 8, float(off.mean())


# ------------------------------------------------------------------ rows out of range among rows in range


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,new,width,dist", [(8, 2, 3, 90, [0, 1, 7, 200]), (8, 2, 9, 40, None), (8, 2, 2, 300, None), (8, 2, 4, 300, None),
                                                   (8, 2, 7, 300, None), (32, 1, 2, 300, list(range(600))), (8, 2, 70, 40, None),
                                                   (8, 2, 70, 90, list(range(70))), (2, 2, 600, 300, [0, 3])])
@pytest.mark.parametrize("kind", ["rope", "table", "short"])
def test_attend_skips_only_the_bad_rows(sfa, dtype, Hq, Hkv, new, width, dist, kind):
    """Rows behind the RoPE table's or the block table's end, or before the request's first: zero rows and the
    status; the others of the request, and of other requests, as ever (gather, cluster, stream with one to four
    column tiles, prompts)."""
    import torch

    rng = np.random.default_rng(61)
    page, cap = 32, 32 * width
    lens = [cap, 900, 40]
    cache, table = make_cache(rng, lens, page, Hkv)
    table = np.ascontiguousarray(table[:, :width])
    cu = np.array([0, new, 2 * new, 2 * new + min(new, 40)])
    told, lost = list(lens), {0: 0, 1: 0, 2: 0}  # what the call is told; rows that are lost at a request's end (or begin)
    cs = ref.rope(cap)
    if kind == "rope":
        cs, lost[0] = cs[:cap - 1], 1
    elif kind == "table":
        told[0], lost[0] = cap + new - 1, new - 1
    else:
        told[1], lost[1] = new - 1, -1
    q = torch.from_numpy(rng.standard_normal((cu[-1], Hq, 64))).to(_dt(dtype))
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(told), cu_q=_i32(cu), dist=dist, rope=_cuda(cs))
    assert sfa.get_device_status() == 6
    o, lse, qn = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    for r in range(3):
        k, v = stored(cache, table, r, lens[r], page)
        rows = np.arange(cu[r], cu[r + 1])
        pos = told[r] - len(rows) + np.arange(len(rows))
        fine = (pos >= 0) & (pos < len(cs))
        assert (~fine).sum() == abs(lost[r]) and fine.any()
        assert not o[rows[~fine]].any() and np.isneginf(lse[rows[~fine]]).all()
        wo, wl, av, sz = ref.attend(qn[rows[fine]], k, v, pos[fine], dist, 1.0, 1.0, cs)
        bo, bl = ref.bounds(wo, wl, av, sz, dtype == "bf16")
        assert (np.abs(o[rows[fine]] - wo) <= bo).all() and (np.abs(lse[rows[fine]] - wl) <= bl).all(), r


# ------------------------------------------------------------------ batches that keep every team busy for several chunks


def _shared_pages(rng, lens, page, H, width, P=61):
    """A small pool whose pages many requests share, rows quantised normal numbers; block tables of `width` pages."""
    x = (rng.standard_normal((2, P, page, H, 64)) * np.exp(0.5 * rng.standard_normal((2, 1, 1, H, 64)))).astype(np.float32)
    parts = []
    for codes, scales in (ref.quantise(x[0]), ref.quantise(x[1])):
        parts.append(((codes[..., 0::2] | codes[..., 1::2] << 4), scales))
    flat = lambda a: a.transpose(0, 2, 1, 3).reshape(P, H, -1)  # noqa: E731
    cache = np.concatenate([flat(parts[0][0]), flat(parts[1][0]), flat(np.concatenate([parts[0][1], parts[1][1]], -1))], -1)
    table = rng.integers(0, P, (len(lens), width)).astype(np.int32)
    for r, n in enumerate(lens):
        table[r, -(-n // page):] = -1
    return np.ascontiguousarray(cache.astype(np.uint8)), table


BATCHES = [  # R, most rows, block table rows, Hq, Hkv, page, new rows of a request (None: one), what it reaches
    (300, 6000, 6000, 8, 2, 64, None),  # eight columns: several chunks a team, their sums in both buffers, join of many columns
    (700, 3000, 6016, 4, 4, 32, None),  # more requests than threads, chunks of 1024 and more
    (150, 2000, 2048, 8, 2, 16, None),  # one chunk a request
    (200, 4000, 5000, 16, 1, 64, None),  # two column tiles
    (100, 3000, 4000, 8, 2, 32, (2, 4)),  # the same from rows
    (90, 3000, 4000, 8, 2, 64, (4, 8)),  # four column tiles, queries in shared memory for two KV heads
    (90, 3000, 4000, 32, 1, 128, None),  # the same from heads
    (300, 2000, 2048, 16, 2, 64, (2, 4)),  # the same in one chunk
    (500, 300, 512, 8, 2, 16, (20, 40)),  # prompts: more items than threads, units that end inside a CTA's share
    (40, 3000, 4096, 8, 2, 64, (9, 130)),  # prompts: units over several CTAs
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(BATCHES)))
@pytest.mark.parametrize("window", [None, 700])
def test_attend_large_batches(sfa, dtype, case, window):
    """Enough requests that the teams walk over several chunks, requests and heads each."""
    import torch

    R, most, rows, Hq, Hkv, page, new = BATCHES[case]
    rng = np.random.default_rng(70 + case)
    least = new[1] if new else 1
    lens = [int(x) for x in np.exp(rng.uniform(np.log(least), np.log(most + 1), R))]
    lens[3], lens[R // 2], lens[-1] = most, 0 if new is None else least, most
    news = [int(x) for x in rng.integers(new[0], new[1] + 1, R)] if new else [1] * R
    cache, table = _shared_pages(rng, lens, page, Hkv, -(-rows // page))
    cu = np.concatenate([[0], np.cumsum(news)])
    q = torch.from_numpy(1.5 * rng.standard_normal((cu[-1], Hq, 64))).to(_dt(dtype))
    cs = ref.rope(rows)
    dist = None if window is None else list(range(window))
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu) if new else None, dist=dist, rope=_cuda(cs))
    assert sfa.get_device_status() == 0
    o, lse, qn = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    picked = set(rng.choice(R, min(R, max(8, 1500 // (Hq * max(news)))), replace=False)) | {3, R // 2, R - 1}
    for r in sorted(picked):
        a, b, n = cu[r], cu[r + 1], lens[r]
        if n == 0:
            assert not o[a:b].any() and np.isneginf(lse[a:b]).all()
            continue
        k, v = stored(cache, table, r, n, page)
        wo, wl, av, sz = ref.attend(qn[a:b], k, v, np.arange(n - (b - a), n), dist, 1.0, 1.0, cs)
        bo, bl = ref.bounds(wo, wl, av, sz, dtype == "bf16")
        assert (np.abs(o[a:b] - wo) <= bo).all() and (np.abs(lse[a:b] - wl) <= bl).all(), (r, float((np.abs(o[a:b] - wo) / bo).max()))
    assert np.isfinite(o).all() and not np.isnan(lse).any()


@pytest.mark.parametrize("Hq,Hkv,dtype", [(8, 2, "f32"), (8, 2, "bf16"), (16, 1, "bf16"), (32, 1, "f32")])
def test_rows_of_a_large_batch_are_their_own(sfa, Hq, Hkv, dtype):
    """One row a request, hundreds of them: a row's bits stay whatever the other requests' lengths make of the
    shares of work, over calls and runs."""
    import torch

    rng = np.random.default_rng(81)
    R, page, rows = 300, 64, 6016
    lens = [int(x) for x in rng.integers(1, rows, R)]
    cache, table = _shared_pages(rng, [rows] * R, page, Hkv, rows // page)
    q = torch.from_numpy(rng.standard_normal((R, Hq, 64))).to(_dt(dtype)).cuda()
    args, rope = (_cuda(cache), _cuda(table)), _cuda(ref.rope(rows))
    o, lse = sfa.kv4_attend(q, *args, _i32(lens), rope=rope)
    for turn in range(4):
        kept = rng.random(R) < (1.0, 0.5, 0.1, 0.02)[turn]
        other = [n if keep else int(rng.integers(0, rows)) for n, keep in zip(lens, kept)]
        o2, l2 = sfa.kv4_attend(q, *args, _i32(other), rope=rope)
        same = torch.from_numpy(np.array(other) == np.array(lens)).cuda()
        assert same.any() and torch.equal(o[same], o2[same]) and torch.equal(lse[same], l2[same])
    assert sfa.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,rows,dist", [(16, 4, 2000, FIB), (8, 8, 3900, list(range(0, 80, 2))), (8, 4, 3900, list(range(50)) + list(range(60, 216, 2))),
                                              (16, 4, 2000, list(range(0, 260, 2)))])
def test_attend_many_rows_side_by_side(sfa, dtype, Hq, Hkv, rows, dist):
    """Rows enough that several share a warp's columns over some tiles of keys each (and, with 130 keys, that they do
    not): requests of one row and of hundreds, a stored NaN value among them, rows behind the last."""
    import torch

    rng = np.random.default_rng(91)
    page, G = 16, Hq // Hkv
    news = [1, 700, 2, 1, 333, 5]
    news.append(rows - sum(news))
    lens = [int(n + x) for n, x in zip(news, rng.integers(0, 400, len(news)))]
    cache, table = _shared_pages(rng, lens, page, Hkv, -(-max(lens) // page), P=300)
    table[1] = np.where(table[1] >= 0, rng.permutation(300)[:1].repeat(table.shape[1]) % 7 + 290, -1)  # pages of its own
    for r in range(len(lens)):
        if r != 1:
            table[r] = np.where(table[r] >= 290, table[r] - 290, table[r])
    own = int(table[1, 0])
    cache[own, 0, 64 * page + 8 * 3 + 5] = 127  # row 3 of the page that request 1 repeats: KV head 0, dims 16 .. 31
    cu = np.concatenate([[0], np.cumsum(news)])
    q = torch.from_numpy(rng.standard_normal((rows + 9, Hq, 64))).to(_dt(dtype))
    cs = ref.rope(table.shape[1] * page)
    o = torch.full(tuple(q.shape), 3.0, dtype=_dt(dtype), device="cuda")
    o, lse = sfa.kv4_attend(q.cuda(), _cuda(cache), _cuda(table), _i32(lens), cu_q=_i32(cu), dist=dist, rope=_cuda(cs), o=o)
    assert sfa.get_device_status() == 0 and (o[rows:] == 3).all()
    o, lse, qn = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    clean = cache.copy()
    clean[own, 0, 64 * page + 8 * 3 + 5] = 0
    for r, n in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        if b - a > 700:  # a part of the longest
            a = b - 400
        k, v = stored(clean, table, r, n, page)
        pos = np.arange(n - (b - a), n)
        wo, wl, av, sz = ref.attend(qn[a:b], k, v, pos, dist, 1.0, 1.0, cs)
        bo, bl = ref.bounds(wo, wl, av, sz, dtype == "bf16")
        if r == 1:
            hit = np.array([any((p - s) % page == 3 for s in dist if s <= p) for p in pos])
            nan = np.zeros(wo.shape, bool)
            nan[hit, :G, 16:32] = True
            assert np.array_equal(np.isnan(o[a:b]), nan)
            wo[nan] = 0
            o[a:b][nan] = 0
        assert (np.abs(o[a:b] - wo) <= bo).all() and (np.abs(lse[a:b] - wl) <= bl).all(), r

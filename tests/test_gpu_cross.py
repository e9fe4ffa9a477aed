"""Attention to states of another length, its gradients, and decode steps behind a shared prefix, against the
64-bit definitions of cross_ref.py."""
import ctypes
import math

import pytest
import torch

import cross_ref as ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def sfa(sfa_lib):
    import static_offset_sparse_gb300 as s

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s.get_device_status()
    return s


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _inputs(seed, B, Tq, Tk, Hq, Hkv, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
    return normal(B, Hq, Tq, 64) * scale, normal(B, Hkv, Tk, 64), normal(B, Hkv, Tk, 64), normal(B, Hq, Tq, 64)


def _spoil(x, lens, what=NAN):
    """x [B, H, T, ...] with `what` behind the lengths."""
    if lens is not None:
        x = x.clone()
        for b, n in enumerate(lens):
            x[b, :, n:] = what
    return x


def _forward(sfa, q, k, v, nq, nk, **kw):
    got = sfa.cross_forward(q.cuda(), k.cuda(), v.cuda(), q_len=_i32(nq), kv_len=_i32(nk), **kw)
    assert sfa.get_device_status() == 0
    return got


def _check_forward(sfa, q, k, v, nq, nk):
    o, lse = _forward(sfa, q, k, v, nq, nk)
    wo, wl, bo, bl = ref.forward(q, k, v, nq, nk)
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)
    return o, lse


def _check_backward(sfa, q, k, v, do, nq, nk):
    """Gradients from o and lse as the forward's exact values round to them, all spoiled behind the lengths."""
    o, lse, _, _ = ref.forward(_spoil(q, nq, 0.0), _spoil(k, nk, 0.0), _spoil(v, nk, 0.0), nq, nk)
    o, lse = o.to(q.dtype), lse.float()
    clean = ref.backward(_spoil(q, nq, 0.0), _spoil(k, nk, 0.0), _spoil(v, nk, 0.0), o, lse, _spoil(do, nq, 0.0), nq, nk)
    o, lse, do = _spoil(o, nq), _spoil(lse, nq), _spoil(do, nq)
    got = sfa.cross_backward(*(x.cuda() for x in (q, k, v, o, lse, do)), q_len=_i32(nq), kv_len=_i32(nk))
    assert sfa.get_device_status() == 0
    for name, g, w, b in zip(("dq", "dk", "dv"), got, *clean):
        ref.check(name, g, w, b)
    return got


# (B, Tq, Tk, Hq, Hkv, lengths of queries, lengths of keys)
SIZES = [
    (1, 1, 1, 1, 1, None, None),
    (1, 1, 300, 8, 2, None, None),
    (3, 1, 777, 8, 2, None, [777, 0, 130]),
    (2, 3, 5, 4, 2, None, None),
    (2, 2, 64, 12, 4, [2, 1], [64, 63]),
    (1, 7, 1000, 32, 1, None, None),
    (1, 1, 4100, 3, 3, None, None),
    (2, 17, 65, 8, 8, [17, 0], [65, 1]),
    (1, 64, 64, 4, 1, None, None),
    (1, 63, 129, 6, 2, None, None),
    (1, 130, 127, 2, 2, None, None),
    (2, 33, 500, 24, 2, [33, 20], [257, 500]),
    (1, 200, 1000, 5, 1, None, None),
    (1, 129, 3000, 8, 2, [129], [2999]),
    (2, 300, 128, 8, 2, [299, 1], [128, 77]),
    (4, 257, 256, 2, 1, [257, 128, 0, 3], [256, 129, 5, 0]),
    (1, 1025, 70, 4, 4, None, None),
    (1, 40, 9000, 8, 8, None, None),
]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv,nq,nk", SIZES)
def test_forward(sfa, B, Tq, Tk, Hq, Hkv, nq, nk, dtype):
    q, k, v, _ = _inputs(B * 1000 + Tq + Tk, B, Tq, Tk, Hq, Hkv, dtype)
    _check_forward(sfa, _spoil(q, nq), _spoil(k, nk), _spoil(v, nk), nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv,nq,nk", SIZES)
def test_backward(sfa, B, Tq, Tk, Hq, Hkv, nq, nk, dtype):
    q, k, v, do = _inputs(B * 1000 + Tq + Tk + 1, B, Tq, Tk, Hq, Hkv, dtype)
    _check_backward(sfa, _spoil(q, nq), _spoil(k, nk), _spoil(v, nk), do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [2, 70])
def test_infinite_padding(sfa, Tq, dtype):
    q, k, v, do = _inputs(5, 2, Tq, 200, 4, 2, dtype)
    nq, nk = [Tq, Tq - 1], [133, 200]
    q, k, v = _spoil(q, nq, INF), _spoil(k, nk, -INF), _spoil(v, nk, INF)
    _check_forward(sfa, q, k, v, nq, nk)
    _check_backward(sfa, q, k, v, do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 90])
def test_strided_views(sfa, Tq, dtype):
    """Queries of a [B, T, H, 64] projection, keys and values of a joint one with heads before rows."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(2, Tq, 3 * 8, 64, generator=gen).to(dtype).cuda()
    kv = torch.randn(2, 150, 2, 2, 64, generator=gen).to(dtype).cuda()
    q, k, v = x[:, :, 8:16].transpose(1, 2), kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    assert not q.is_contiguous() or Tq == 1
    o, lse = sfa.cross_forward(q, k, v)
    o2, lse2 = sfa.cross_forward(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    do = torch.randn(2, 8, Tq, 64, generator=gen).to(dtype).cuda()
    for a, b in zip(sfa.cross_backward(q, k, v, o, lse, do), sfa.cross_backward(q.contiguous(), k.contiguous(), v.contiguous(), o, lse, do)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 700), (100, 300)])
def test_far_logits(sfa, Tq, Tk, dtype):
    """Logits of 2^30 and more, all of a row below -2^30, and queries of zeros: no NaN, one key takes all."""
    q, k, v, _ = _inputs(7, 1, Tq, Tk, 4, 2, dtype)
    k = k.abs()
    q = q.sign() * 2.0 ** 30
    q[:, 1] = -q[:, 1].abs()
    q[:, 3] = 0
    o, lse = _forward(sfa, q, k, v, None, None)
    s = q.double() @ k.double().repeat_interleave(2, 1).transpose(-1, -2) / 8
    top = s.amax(-1)
    # fp32 products of 2^30: off by 66 u of the terms' sizes
    size = (q.double().abs() @ k.double().repeat_interleave(2, 1).abs().transpose(-1, -2) / 8).amax(-1)
    assert bool(((lse.cpu().double() - torch.logsumexp(s, -1)).abs() <= 70 * ref.U * size + 1e-3)[:, :3].all())
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all()) and bool(top.isfinite().all())
    near = s >= top[..., None] - 140 * ref.U * size[..., None]  # keys that may take all
    vv = v.double().repeat_interleave(2, 1)
    alone = near.sum(-1) == 1
    r = ref.half_step(dtype)
    pick = torch.gather(vv, 2, s.argmax(-1)[..., None].expand(-1, -1, -1, 64))
    off = ((o.cpu().double() - pick).abs() - 2 * r * pick.abs() - 1e-6)[:, :3][alone[:, :3]]
    assert off.numel() == 0 or float(off.max()) <= 0


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 100])
def test_nan_stays_in_its_rows(sfa, Tq, dtype):
    q, k, v, do = _inputs(8, 2, Tq, 200, 8, 2, dtype)
    q[0, 3, Tq // 2] = NAN
    k[1, 1, 150] = NAN
    o, lse = _forward(sfa, q, k, v, None, None)
    bad = torch.zeros(2, 8, Tq, dtype=torch.bool)
    bad[0, 3, Tq // 2] = True
    bad[1, 4:] = True
    assert torch.equal(lse.isnan().cpu(), bad) and torch.equal(o.isnan().any(-1).cpu(), bad)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_lengths_out_of_range(sfa, dtype):
    q, k, v, do = (x.cuda() for x in _inputs(9, 3, 20, 40, 4, 2, dtype))
    o, lse = sfa.cross_forward(q, k, v, q_len=_i32([20, 21, 20]), kv_len=_i32([-1, 40, 41]))
    assert sfa.get_device_status() == 6
    assert not o.any() and bool((lse == -INF).all())
    grads = sfa.cross_backward(q, k, v, o, lse, do, q_len=_i32([20, 21, 20]), kv_len=_i32([-1, 40, 41]))
    assert sfa.get_device_status() == 6
    assert not any(g.any() for g in grads)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 5000), (200, 2000), (3000, 40)])
def test_same_bits_again_and_in_a_graph(sfa, Tq, Tk, dtype):
    q, k, v, do = (x.cuda() for x in _inputs(10, 1, Tq, Tk, 8, 2, dtype))
    lens = dict(q_len=_i32([Tq]), kv_len=_i32([Tk - 3]))

    def step():
        o, lse = sfa.cross_forward(q, k, v, **lens)
        return (o, lse, *sfa.cross_backward(q, k, v, o, lse, do, **lens))

    first = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = [x.clone() for x in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for x in out:
        x.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, out):
        assert torch.equal(a, b) and torch.equal(a, c)
    # other contents and lengths in the same graph
    q.copy_(torch.randn_like(q))
    lens["kv_len"].fill_(max(1, Tk // 3))
    want = [x.clone() for x in step()]
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(want, out):
        assert torch.equal(a, c)


def test_python_refusals(sfa):
    q, k, v, do = (x.cuda() for x in _inputs(11, 2, 5, 9, 4, 2, torch.bfloat16))
    o, lse = sfa.cross_forward(q, k, v)
    bad = [((q, k.float(), v), {}), ((q, k, v[:, :, :8]), {}), ((q, k[:1], v[:1]), {}), ((q[0], k, v), {}),
           ((q[..., :32], k, v), {}), ((q, k, v.expand(2, 2, 9, 64)[:, :1].expand(2, 2, 9, 64)), {}),
           ((q, k, v), dict(q_len=_i32([1]))), ((q, k, v), dict(kv_len=_i32([1, 2]).long())), ((q, k, v), dict(o=o.float())),
           ((q, k, v), dict(lse=lse[:, :, :4])), ((q, k, v), dict(o=o.transpose(1, 2).contiguous().transpose(1, 2)))]
    for args, kw in bad:
        with pytest.raises((ValueError, TypeError)):
            sfa.cross_forward(*args, **kw)
    with pytest.raises(TypeError):
        sfa.cross_forward(q.half(), k.half(), v.half())
    with pytest.raises(ValueError):
        sfa.cross_backward(q, k, v, o, lse, do.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        sfa.cross_backward(q, k, v, o, lse.double(), do)
    with pytest.raises(sfa.SfaError):
        sfa.cross_forward(q[:, :3], k, v)


def test_outputs_and_workspace_of_the_caller(sfa):
    q, k, v, do = (x.cuda() for x in _inputs(12, 1, 5, 3001, 8, 2, torch.bfloat16))
    want = sfa.cross_forward(q, k, v)
    o, lse = torch.empty_like(q), torch.empty(1, 8, 5, device="cuda")
    ws = torch.full((sfa.cross_workspace_size(q, k, v) + 64,), 255, dtype=torch.uint8, device="cuda")
    got = sfa.cross_forward(q, k, v, o=o, lse=lse, ws=ws)
    assert got[0] is o and got[1] is lse and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert bool((ws[-64:] == 255).all())
    grads = sfa.cross_backward(q, k, v, o, lse, do)
    ws = torch.full((sfa.cross_workspace_size(q, k, v, backward=True) + 64,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(x, NAN) for x in (q, k, v)]
    sfa.cross_backward(q, k, v, o, lse, do, dq=outs[0], dk=outs[1], dv=outs[2], ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs)) and bool((ws[-64:] == 255).all())


# ------------------------------------------------------------------ decode steps behind a shared prefix


def _prefix_inputs(seed, B, P, T, Hq, Hkv, dtype):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
    return normal(B, Hq + 2 * Hkv, 64), normal(Hkv, P, 64), normal(Hkv, P, 64), normal(B, Hkv, T, 64), normal(B, Hkv, T, 64)


def _step(sfa, qkv, pk, pv, kc, vc, pos, Hq, **kw):
    Hkv = pk.shape[0]
    return sfa.prefix_decode(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pk, pv, kc, vc, _i32(pos), **kw)


PREFIXES = [
    (1, 1, 1, 1, 1, [0]),
    (1, 0, 40, 8, 2, [39]),
    (2, 3, 5, 8, 2, [4, 0]),
    (3, 100, 30, 4, 4, [29, 0, 7]),
    (5, 1000, 600, 6, 2, [0, 599, 300, 256, 255]),
    (17, 129, 64, 32, 1, [(7 * i) % 64 for i in range(17)]),
    (33, 2000, 300, 8, 1, [(37 * i) % 300 for i in range(33)]),
    (130, 257, 33, 8, 2, [(5 * i) % 33 for i in range(130)]),
    (40, 5000, 20, 24, 2, [i % 20 for i in range(40)]),
    (16, 50, 2100, 8, 8, [(523 * i) % 2100 for i in range(16)]),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,P,T,Hq,Hkv,pos", PREFIXES)
def test_prefix(sfa, B, P, T, Hq, Hkv, pos, dtype):
    qkv, pk, pv, kc, vc = _prefix_inputs(B + P + T, B, P, T, Hq, Hkv, dtype)
    for b, t in enumerate(pos):  # what stands behind, and at, the step's row is not read
        kc[b, :, t:] = NAN
        vc[b, :, t:] = NAN
    rope = sfa.rope_table(P + T).cpu()
    dev = [x.cuda() for x in (qkv, pk, pv, kc, vc)]
    o, lse = _step(sfa, *dev, pos, Hq)
    assert sfa.get_device_status() == 0
    r = ref.half_step(dtype)
    for b, t in enumerate(pos):
        kc[b, :, t], vc[b, :, t] = dev[3][b, :, t].cpu(), qkv[b, Hq + Hkv:]
        x = qkv[b, Hq:Hq + Hkv]
        want = ref.rotated(x, rope[P + t])
        pair = x.double().abs() + x.double().roll(32, -1).abs()
        ref.check("new key", dev[3][b, :, t], want, r * want.abs() + 3 * (1 + r) * ref.U * pair + 1e-37)
    assert torch.equal(dev[3].cpu().nan_to_num(99.0), kc.nan_to_num(99.0)) and torch.equal(dev[4].cpu().nan_to_num(99.0), vc.nan_to_num(99.0))
    wo, wl, bo, bl = ref.prefix(qkv[:, :Hq], pk, pv, kc, vc, pos, rope)
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_prefix_rows_out_of_range(sfa, dtype):
    qkv, pk, pv, kc, vc = (x.cuda() for x in _prefix_inputs(3, 4, 70, 20, 8, 2, dtype))
    before = kc.clone(), vc.clone()
    whole = _step(sfa, qkv, pk, pv, kc.clone(), vc.clone(), [3, 4, 19, 5], 8)
    o, lse = _step(sfa, qkv, pk, pv, kc, vc, [3, -1, 19, 20], 8)
    assert sfa.get_device_status() == 6
    for b in (1, 3):
        assert not o[b].any() and bool((lse[b] == -INF).all())
        assert torch.equal(kc[b], before[0][b]) and torch.equal(vc[b], before[1][b])
    for b in (0, 2):
        assert torch.equal(o[b], whole[0][b]) and torch.equal(lse[b], whole[1][b])


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_prefix_without_new_rows_and_rotation(sfa, dtype):
    """Caches that hold the step's rows, rows of the caller's own strides, no rotation."""
    B, P, T, Hq, Hkv = 6, 300, 50, 8, 2
    qkv, pk, pv, kc, vc = _prefix_inputs(4, B, P, T, Hq, Hkv, dtype)
    pos = [49, 0, 3, 17, 22, 31]
    wide = torch.zeros(Hkv, P + 24, 64, dtype=dtype)
    wide[:, :P] = pk
    for rope in (None, sfa.rope_table(P + T)):
        o, lse = sfa.prefix_decode(qkv.cuda()[:, :Hq], None, None, wide.cuda()[:, :P], pv.cuda(), kc.cuda(), vc.cuda(), _i32(pos),
                                   rope=rope, rope_theta=0 if rope is None else 1e4)
        wo, wl, bo, bl = ref.prefix(qkv[:, :Hq], pk, pv, kc, vc, pos, None if rope is None else rope.cpu())
        ref.check("o", o, wo, bo)
        ref.check("lse", lse, wl, bl)


def test_prefix_steps_as_a_user_makes_them(sfa):
    """A prefix laid out by rope_keys, then steps captured once and replayed while pos counts up: the same as
    decode_int over caches that hold everything, key by key unrotated."""
    B, P, T, Hq, Hkv = 3, 90, 6, 8, 2
    gen = torch.Generator().manual_seed(6)
    normal = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    raw_k, raw_v = normal(1, Hkv, P, 64), normal(1, Hkv, P, 64)
    pk, pv = sfa.rope_keys(raw_k)[0], raw_v[0]
    kc, vc = torch.full((B, Hkv, T, 64), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((B, Hkv, T, 64), NAN, dtype=torch.bfloat16, device="cuda")
    rope, pos, qkv = sfa.rope_table(P + T), _i32([0] * B), normal(B, Hq + 2 * Hkv, 64)

    def step():
        return sfa.prefix_decode(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pk, pv, kc, vc, pos, rope=rope)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    dense_k, dense_v = (torch.cat([x.expand(B, -1, -1, -1), torch.zeros(B, Hkv, T, 64, dtype=x.dtype, device="cuda")], 2).contiguous() for x in (raw_k, raw_v))
    for t in range(T):
        qkv.copy_(normal(B, Hq + 2 * Hkv, 64))
        pos.fill_(t)
        graph.replay()
        dense_k[:, :, P + t], dense_v[:, :, P + t] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        want, wlse = sfa.decode_int(qkv[:, :Hq].contiguous(), dense_k, dense_v, pos + P, dist=list(range(P + T)))
        # keys here are rounded once more after the rotation, probabilities and outputs to bf16: logits of up to
        # 2^-8 sum |q k| / 8 (24 is beyond the largest here) and values of 4 at most
        assert float((lse - wlse).abs().max()) < 2.0 ** -8 * 24
        assert float((o.float() - want.float()).abs().max()) < 4 * (2 * 2.0 ** -8 * 24 + 3 * 2.0 ** -8)
    assert sfa.get_device_status() == 0


def test_prefix_python_refusals(sfa):
    B, P, T, Hq, Hkv = 2, 10, 4, 8, 2
    qkv, pk, pv, kc, vc = (x.cuda() for x in _prefix_inputs(7, B, P, T, Hq, Hkv, torch.bfloat16))
    q, kn, vn, pos = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], _i32([0, 1])
    good = dict(q=q, k_new=kn, v_new=vn, prefix_k=pk, prefix_v=pv, k_cache=kc, v_cache=vc, pos=pos)
    sfa.prefix_decode(**good)
    bad = [dict(q=q[:1]), dict(q=q.float()), dict(k_new=None), dict(v_new=vn[:, :1]), dict(prefix_k=pk[:1]), dict(prefix_v=pv[:, :9]),
           dict(prefix_k=pk.transpose(0, 1).contiguous().transpose(0, 1)), dict(k_cache=kc.transpose(1, 2)), dict(v_cache=vc[:, :, :3]),
           dict(pos=pos.long()), dict(pos=pos[:1]), dict(rope=torch.zeros(5, 32, device="cuda")), dict(o=torch.zeros(B, Hq, 64, device="cuda"))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            sfa.prefix_decode(**{**good, **kw})
    with pytest.raises(sfa.SfaError):
        sfa.prefix_decode(**good, rope=sfa.rope_table(P + T - 1))


# ------------------------------------------------------------------ where it can go wrong


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 900), (5, 900), (130, 900)])
def test_logits_that_rise_along_the_keys(sfa, Tq, Tk, dtype):
    """Each key's logits are far above the ones before it, in steps and by single keys: sums are moved many times."""
    q, k, v, do = _inputs(20, 1, Tq, Tk, 4, 2, dtype)
    q = q.abs()
    rise = torch.arange(Tk, dtype=torch.float32)[:, None] // 50 * 0.7 + (torch.arange(Tk)[:, None] == 600) * 40.0
    k = (k.abs() * 0.3 + rise).to(dtype)
    _check_forward(sfa, q, k, v, None, None)
    _check_backward(sfa, q, k, v, do, None, None)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 5, 70])
@pytest.mark.parametrize("dead", [10, 96, 300])
def test_keys_of_minus_infinity(sfa, Tq, dead, dtype):
    """The first keys' logits are -inf: as if they were not there; all of them: NaN, as a softmax has it."""
    q, k, v, _ = _inputs(21, 1, Tq, 333, 4, 2, dtype)
    q = q.abs() + 0.1
    k[:, :, :dead] = -INF
    k[:, :, dead:] -= 40  # logits of -100 and less: nothing of them may be lost against the dead ones
    o, lse = _forward(sfa, q, k, v, None, None)
    wo, wl, bo, bl = ref.forward(q, k[:, :, dead:], v[:, :, dead:])
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)
    o, lse = _forward(sfa, q, torch.full_like(k, -INF), v, None, None)
    assert bool(o.isnan().all()) and not bool(lse.isfinite().any())


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 5, 140])
def test_huge_numbers(sfa, Tq, dtype):
    """2^100 in a dim of the queries where keys are zero, and in one of the values where gradients are."""
    q, k, v, do = _inputs(22, 1, Tq, 333, 4, 2, dtype)
    q[..., 0], k[..., 0] = 2.0 ** 100, 0.0
    v[..., 3], do[..., 3] = v[..., 3] * 2.0 ** 100, 0.0
    _check_forward(sfa, q, k, v, None, None)
    _check_backward(sfa, q, k, v, do, None, None)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv", [(3, 50, 4, 2), (40, 150, 4, 1), (1, 200, 3, 1)])
def test_many_ragged_sequences(sfa, Tq, Tk, Hq, Hkv, dtype):
    """More sequences than SMs, lengths from none to all."""
    B = 413
    q, k, v, do = _inputs(22, B, Tq, Tk, Hq, Hkv, dtype)
    gen = torch.Generator().manual_seed(23)
    nq, nk = (torch.randint(0, n + 1, (B,), generator=gen).tolist() for n in (Tq, Tk))
    _check_forward(sfa, _spoil(q, nq), _spoil(k, nk), _spoil(v, nk), nq, nk)
    _check_backward(sfa, _spoil(q, nq), _spoil(k, nk), _spoil(v, nk), do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv", [(100, 300, 300, 8, 2), (413, 40, 150, 4, 1), (130, 400, 500, 8, 2)])
def test_many_ragged_sequences_again_and_again(sfa, B, Tq, Tk, Hq, Hkv, dtype):
    """Many short units an SM, one behind the other: every call gives the same bits."""
    gen = torch.Generator().manual_seed(7)
    q, k, v, do = (x.cuda() for x in _inputs(5, B, Tq, Tk, Hq, Hkv, dtype))
    nq, nk = (_i32(torch.randint(0, n + 1, (B,), generator=gen).tolist()) for n in (Tq, Tk))
    first = sfa.cross_forward(q, k, v, q_len=nq, kv_len=nk)
    grads = sfa.cross_backward(q, k, v, *first, do, q_len=nq, kv_len=nk)
    for _ in range(60):
        again = sfa.cross_forward(q, k, v, q_len=nq, kv_len=nk)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        again = sfa.cross_backward(q, k, v, *first, do, q_len=nq, kv_len=nk)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
    assert sfa.get_device_status() == 0


def test_backward_of_a_large_batch(sfa):
    """Enough steps an SM for dq, and dk and dv, to be launches of their own."""
    B, Tq, Tk = 17, 1000, 2040
    q, k, v, do = _inputs(25, B, Tq, Tk, 4, 2, torch.bfloat16)
    gen = torch.Generator().manual_seed(26)
    nq, nk = (torch.randint(n // 2, n + 1, (B,), generator=gen).tolist() for n in (Tq, Tk))
    nq[3], nk[5] = 0, 0
    _check_backward(sfa, _spoil(q, nq), _spoil(k, nk), _spoil(v, nk), do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_one_long_sequence_among_empty_ones(sfa, dtype):
    B, Tq, Tk = 9, 200, 5000
    q, k, v, do = _inputs(24, B, Tq, Tk, 2, 1, dtype)
    nq, nk = [0, 0, 5, 0, 200, 0, 0, 200, 0], [5000, 0, 0, 3, 4999, 0, 1, 0, 9]
    _check_forward(sfa, q, k, v, nq, nk)
    _check_backward(sfa, q, k, v, do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 40])
def test_offsets_past_32_bits(sfa, Tq, dtype):
    """Keys and values whose sequences, heads and rows lie more than 2^31 numbers apart."""
    B, Tk, Hkv = 2, 130, 2
    q, k, v, do = _inputs(25, B, Tq, Tk, 4, Hkv, dtype)
    want = sfa.cross_forward(q.cuda(), k.cuda(), v.cuda())
    grads = sfa.cross_backward(q.cuda(), k.cuda(), v.cuda(), *want, do.cuda())
    n = (1 << 31) + 64 * 1024
    buf = torch.empty(n + 64 * 1024 * 64, dtype=dtype, device="cuda")
    for strides in ((n, 64 * Tk, 64), (64 * Tk, n, 64), (64 * Hkv * 8, 64 * 8, (1 << 31) // (Tk - 1) // 64 * 64 + 64 * 32)):
        assert sum((m - 1) * s for m, s in zip((B, Hkv, Tk), strides)) + 64 <= buf.numel()
        views = []
        for x in (k, v):
            view = torch.as_strided(buf, (B, Hkv, Tk, 64), (*strides, 1))
            view.copy_(x)
            got = (view, v.cuda()) if x is k else (k.cuda(), view)
            o, lse = sfa.cross_forward(q.cuda(), *got)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            assert all(torch.equal(a, b) for a, b in zip(sfa.cross_backward(q.cuda(), *got, o, lse, do.cuda()), grads))
            views.append(view)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 700), (3, 65), (100, 300), (257, 1)])
def test_nothing_is_written_beside_the_outputs(sfa, Tq, Tk, dtype):
    q, k, v, do = (x.cuda() for x in _inputs(26, 2, Tq, Tk, 6, 2, dtype))
    nk = _i32([Tk, max(1, Tk // 2)])

    def guarded(shape, dt):
        n = math.prod(shape)
        whole = torch.full((n + 512,), 3.0, dtype=dt, device="cuda")
        return whole, whole[256:256 + n].view(shape)

    held = [guarded(q.shape, dtype), guarded(q.shape[:3], torch.float32), guarded(q.shape, dtype), guarded(k.shape, dtype), guarded(k.shape, dtype)]
    o, lse, dq, dk, dv = (x for _, x in held)
    sfa.cross_forward(q, k, v, kv_len=nk, o=o, lse=lse)
    sfa.cross_backward(q, k, v, o, lse, do, kv_len=nk, dq=dq, dk=dk, dv=dv)
    plain = sfa.cross_forward(q, k, v, kv_len=nk)
    for a, b in zip((o, lse, dq, dk, dv), (*plain, *sfa.cross_backward(q, k, v, *plain, do, kv_len=nk))):
        assert torch.equal(a, b)  # (the calls with outputs of the caller go the ctypes way, the others the native one)
    for whole, _ in held:
        assert bool((whole[:256] == 3).all()) and bool((whole[-256:] == 3).all())


def test_broadcast_keys_are_refused(sfa):
    """One source for a batch is expanded by the caller's copy (its gradient is a sum the caller takes)."""
    q, k = torch.zeros(3, 2, 4, 64, device="cuda"), torch.zeros(1, 2, 9, 64, device="cuda")
    with pytest.raises(ValueError):
        sfa.cross_forward(q, k.expand(3, 2, 9, 64), k.expand(3, 2, 9, 64))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_calls_at_once_on_two_streams(sfa, dtype):
    """Two streams' calls overlap: each has a workspace of its own."""
    q, k, v, do = (x.cuda() for x in _inputs(27, 1, 300, 4000, 8, 2, dtype))
    q2, k2, v2, do2 = (x.cuda() for x in _inputs(28, 2, 1, 7000, 8, 2, dtype))
    o, lse = sfa.cross_forward(q, k, v)
    o2, lse2 = sfa.cross_forward(q2, k2, v2)
    want, want2 = sfa.cross_backward(q, k, v, o, lse, do), sfa.cross_backward(q2, k2, v2, o2, lse2, do2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got, got2 = [], []
    for _ in range(5):
        with torch.cuda.stream(a):
            got.append((*sfa.cross_forward(q, k, v), *sfa.cross_backward(q, k, v, o, lse, do)))
        with torch.cuda.stream(b):
            got2.append((*sfa.cross_forward(q2, k2, v2), *sfa.cross_backward(q2, k2, v2, o2, lse2, do2)))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(s, t) for s, t in zip(x, (o, lse, *want)))
    for x in got2:
        assert all(torch.equal(s, t) for s, t in zip(x, (o2, lse2, *want2)))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_prefix_both_ways_and_again(sfa, dtype):
    """The native call, the ctypes call (outputs of the caller), a second one: the same bits, caches as after one."""
    B, P, T, Hq, Hkv = 37, 1500, 90, 8, 2
    qkv, pk, pv, kc, vc = (x.cuda() for x in _prefix_inputs(30, B, P, T, Hq, Hkv, dtype))
    pos = [(11 * i) % T for i in range(B)]
    sfa.rope_table(P + T)
    o, lse = _step(sfa, qkv, pk, pv, kc, vc, pos, Hq)
    after = kc.clone(), vc.clone()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    _step(sfa, qkv, pk, pv, kc, vc, pos, Hq, o=o2, lse=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(kc, after[0]) and torch.equal(vc, after[1])


def test_a_training_step_and_steps_after_it(sfa):
    """An encoder with a signed set, a decoder's cross attention over it trained by one gradient step against
    differences, then single tokens over the same states: each as a program would call it."""
    gen = torch.Generator().manual_seed(31)
    normal = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    B, Tk, Tq = 2, 128, 48
    x, kv, v0 = normal(B, 4, Tk, 64), normal(B, 2, Tk, 64), normal(B, 2, Tk, 64)
    states, _ = sfa.forward_int(x, kv, v0, dist=[-3, -2, -1, 0, 1, 2, 3])
    k = states[:, :2].float().mul(2).bfloat16()
    v = states[:, 2:].contiguous()
    q, do = normal(B, 8, Tq, 64), normal(B, 8, Tq, 64)
    lens = _i32([Tk, 77])
    o, lse = sfa.cross_forward(q, k, v, kv_len=lens)
    dq, dk, dv = sfa.cross_backward(q, k, v, o, lse, do, kv_len=lens)
    # the change of sum(o dO) along a direction against the gradients' product with it, in 64 bits; the quotient's
    # own error is h^2 times a third derivative (h = 2^-8: below 1e-3 of it), the gradients' 2^-7 of their terms
    u = [torch.randn(t.shape, generator=gen).double() for t in (q, k, v)]
    h = 2.0 ** -8

    def value(sign):
        moved = [t.cpu().double() + sign * h * w for t, w in zip((q, k, v), u)]
        return float((ref.forward(*moved, None, [Tk, 77])[0] * do.cpu().double()).sum())

    slope = (value(1) - value(-1)) / (2 * h)
    terms = [(g.cpu().double() * w) for g, w in zip((dq, dk, dv), u)]
    scale = math.sqrt(sum(float((t * t).sum()) for t in terms))
    assert abs(slope - sum(float(t.sum()) for t in terms)) <= 2.0 ** -7 * scale * 4 + 1e-3 * abs(slope)
    for t in range(3):
        one, one_lse = sfa.cross_forward(q[:, :, t:t + 1], k, v, kv_len=lens)
        # another order of sums, probabilities and outputs rounded to bf16 in both
        wo, wl, bo, bl = ref.forward(q[:, :, t:t + 1].cpu(), k.cpu(), v.cpu(), None, [Tk, 77])
        ref.check("o", one, wo, bo)
        assert float((one.float() - o[:, :, t:t + 1].float()).abs().max()) <= 2 * float(bo.max())
        assert float((one_lse - lse[:, :, t:t + 1]).abs().max()) <= 2 * float(bl.max())


# bf16 on the tensor cores: CTA 0 leaves out a tile of keys or values (forward), a step (backward)
@pytest.mark.parametrize("call,skip", [("forward", 0), ("forward", 5), ("backward", 0), ("backward", 3), ("prefix", 2)])
def test_cross_wait_times_out_and_context_recovers(sfa, sfa_lib, call, skip):
    gen = torch.Generator().manual_seed(516)
    q, k, v, do = (torch.randn(1, h, t, 64, generator=gen).bfloat16() for h, t in ((4, 600), (2, 800), (2, 800), (4, 600)))
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = sfa.cross_forward(*dev)
    rows = torch.randn(40, 8, 64, generator=gen).bfloat16().cuda()
    cache = torch.randn(2, 40, 2, 30, 64, generator=gen).bfloat16().cuda()
    pos = torch.arange(40, dtype=torch.int32, device="cuda") % 30

    def run():
        if call == "forward":
            return sfa.cross_forward(*dev)
        if call == "backward":
            return sfa.cross_backward(*dev, o, lse, do.cuda())
        return sfa.prefix_decode(rows[:, :4], rows[:, 4:6], rows[:, 6:], dev[1][0], dev[2][0], cache[0], cache[1], pos)

    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    assert sfa.get_device_status() == 0
    try:
        assert sfa_lib.sfa_debug_inject(ctypes.c_int64(2000000), ctypes.c_int32(skip)) == 0  # about 1 ms
        run()
        torch.cuda.synchronize()
    finally:
        assert sfa_lib.sfa_debug_inject(ctypes.c_int64(0), ctypes.c_int32(-1)) == 0
    assert sfa.get_device_status() == 5  # SFA_ERR_TIMEOUT
    assert sfa.get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
    assert sfa.get_device_status() == 0
    if call == "forward":
        wo, wl, bo, bl = ref.forward(q, k, v)
        ref.check("o", want[0], wo, bo)
        ref.check("lse", want[1], wl, bl)


# ------------------------------------------------------------------ infinities and NaN in keys that count


def _odd_key(seed, Tq, Tk, dtype, what):
    """Inputs of two ragged sequences, queries above 0, and one key of KV head 1 of the first that is `what`."""
    q, k, v, do = _inputs(seed, 2, Tq, Tk, 4, 2, dtype)
    nq, nk = [Tq - (Tq + 2) // 3, Tq], [Tk, Tk - 3]
    k[0, 1, Tk // 2] = what
    return _spoil(q.abs() + 0.1, nq), _spoil(k, nk), _spoil(v, nk), do, nq, nk


ODD_SIZES = [(5, 40), (70, 40), (70, 900), (300, 200)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", ODD_SIZES)
@pytest.mark.parametrize("what", [NAN, INF, -INF])
def test_dq_behind_the_queries_is_zero_whatever_a_key_holds(sfa, what, Tq, Tk, dtype):
    q, k, v, do, nq, nk = _odd_key(40, Tq, Tk, dtype, what)
    o, lse, _, _ = ref.forward(*(_spoil(x, n, 0.0) for x, n in ((q, nq), (k, nk), (v, nk))), nq, nk)
    dq, dk, dv = sfa.cross_backward(*(x.cuda() for x in (q, k, v, o.to(dtype), lse.float(), do)), q_len=_i32(nq), kv_len=_i32(nk))
    assert sfa.get_device_status() == 0
    assert bool((dq[0, :, nq[0]:] == 0).all())
    assert bool((dk[1, :, nk[1]:] == 0).all()) and bool((dv[1, :, nk[1]:] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", ODD_SIZES)
@pytest.mark.parametrize("what", [NAN, -INF])
def test_gradients_of_a_key_of_minus_infinity(sfa, what, Tq, Tk, dtype):
    """Its probabilities are 0, and so are its dk and dv, whatever rows a tile holds besides those that count (dq:
    0 times -inf, NaN).  A key of NaN makes all of its head's gradients NaN, and none of another's."""
    q, k, v, do, nq, nk = _odd_key(41, Tq, Tk, dtype, what)
    dq, dk, dv = _check_backward(sfa, q, k, v, do, nq, nk)
    if what == -INF:
        assert bool((dk[0, 1, Tk // 2] == 0).all()) and bool((dv[0, 1, Tk // 2] == 0).all())
        assert bool(dk[0].isfinite().all()) and bool(dv[0].isfinite().all())
    assert bool(dq[0, :2].isfinite().all()) and bool(dq[1].isfinite().all())
    assert bool(dq[0, 2:, :nq[0]].isnan().all())


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", ODD_SIZES)
def test_gradients_of_rows_whose_lse_is_infinite(sfa, Tq, Tk, dtype):
    """A logit of +inf: its row's softmax is not defined, and neither is what its probabilities enter.  (Other keys'
    probabilities are 0, so their dv is too.)"""
    q, k, v, do, nq, nk = _odd_key(42, Tq, Tk, dtype, INF)
    dq, dk, dv = _check_backward(sfa, q, k, v, do, nq, nk)
    assert bool(dq[0, 2:, :nq[0]].isnan().all()) and bool(dk[0, 1].isnan().all()) and bool(dv[0, 1, Tk // 2].isnan().all())
    assert bool((dv[0, 1, :Tk // 2] == 0).all()) and bool((dv[0, 1, Tk // 2 + 1:] == 0).all())
    assert bool(dq[0, :2].isfinite().all()) and bool(dk[0, 0].isfinite().all()) and bool(dq[1].isfinite().all())


# fp32: own rows up to 2^16 and, with more of them, up to four rows a KV head and call share a launch with the prefix
@pytest.mark.parametrize("B,P,T,Hq,Hkv", [(8, 300, 2000, 16, 4), (8, 300, 2100, 16, 4), (4, 300, 5000, 8, 8), (5, 300, 5000, 8, 8)])
def test_prefix_in_one_launch_and_apart(sfa, B, P, T, Hq, Hkv):
    qkv, pk, pv, kc, vc = _prefix_inputs(43, B, P, T, Hq, Hkv, torch.float32)
    pos = [(T - 1) * (i + 1) // B for i in range(B)]
    dev = [x.cuda() for x in (qkv, pk, pv, kc, vc)]
    o, lse = _step(sfa, *dev, pos, Hq)
    assert sfa.get_device_status() == 0
    wo, wl, bo, bl = ref.prefix(qkv[:, :Hq], pk, pv, dev[3].cpu(), dev[4].cpu(), pos, sfa.rope_table(P + T).cpu())
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)


def _guarded_ws(n):
    """n bytes with 256 guarded ones before and behind."""
    buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + n]


def _guards_hold(buf):
    return bool((buf[:256] == 255).all()) and bool((buf[-256:] == 255).all())


# few rows in parts, few rows in a cluster, tiles in parts; the tensor cores' one and two launches
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv,ragged", [(1, 1, 20000, 8, 2, False), (8, 1, 1500, 8, 2, True), (2, 37, 777, 4, 4, True),
                                                   (1, 333, 1000, 8, 2, False), (1, 130, 9000, 8, 2, True), (17, 1000, 2040, 4, 2, True)])
def test_workspaces_of_exact_size(sfa, B, Tq, Tk, Hq, Hkv, ragged, dtype):
    q, k, v, do = (x.cuda() for x in _inputs(61, B, Tq, Tk, Hq, Hkv, dtype))
    lens = dict(q_len=_i32([Tq - i % Tq for i in range(B)]), kv_len=_i32([Tk - 7 * i for i in range(B)])) if ragged else {}
    want = sfa.cross_forward(q, k, v, **lens)
    buf, ws = _guarded_ws(sfa.cross_workspace_size(q, k, v))
    got = sfa.cross_forward(q, k, v, ws=ws, **lens)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and _guards_hold(buf)
    grads = sfa.cross_backward(q, k, v, *want, do, **lens)
    buf, ws = _guarded_ws(sfa.cross_workspace_size(q, k, v, backward=True))
    got = sfa.cross_backward(q, k, v, *want, do, ws=ws, **lens)
    assert all(torch.equal(a, b) for a, b in zip(grads, got)) and _guards_hold(buf)
    assert bool((ws != 255).any())


# no prefix, prefix and own rows in one launch, apart (tiles; streams), the tensor cores
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,P,T,Hq,Hkv", [(5, 0, 700, 8, 2), (3, 1000, 300, 8, 2), (40, 1000, 90, 8, 2), (32, 100, 1025, 8, 8), (130, 9000, 40, 8, 2)])
def test_prefix_workspaces_of_exact_size(sfa, B, P, T, Hq, Hkv, dtype):
    qkv, pk, pv, kc, vc = (x.cuda() for x in _prefix_inputs(62, B, P, T, Hq, Hkv, dtype))
    pos = [(37 * i) % T for i in range(B)]
    want = _step(sfa, qkv, pk, pv, kc, vc, pos, Hq)
    buf, ws = _guarded_ws(sfa.prefix_workspace_size(qkv[:, :Hq], pk, kc))
    got = _step(sfa, qkv, pk, pv, kc, vc, pos, Hq, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and _guards_hold(buf) and bool((ws != 255).any())
    with pytest.raises(ValueError):
        sfa.prefix_workspace_size(qkv[:, :Hq], pk[:, :, :32], kc)
    with pytest.raises(ValueError):
        sfa.prefix_workspace_size(qkv[:, :Hq].cpu(), pk, kc)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B", [3, 40])
def test_captured_prefix_steps_against_the_definition(sfa, B, dtype):
    """A step captured once and replayed while pos counts up, each replay against the 64-bit definition over the
    caches as it left them; zeros, the plain mean of the values and o without the own rows are far outside the bound."""
    P, T, Hq, Hkv = 90, 6, 8, 2
    gen = torch.Generator().manual_seed(60)
    normal = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
    pk, pv = normal(Hkv, P, 64), normal(Hkv, P, 64)
    kc, vc = (torch.full((B, Hkv, T, 64), NAN, dtype=dtype, device="cuda") for _ in range(2))
    rope, pos, qkv = sfa.rope_table(P + T), _i32([0] * B), normal(B, Hq + 2 * Hkv, 64).cuda()
    dk, dv = pk.cuda(), pv.cuda()

    def step():
        return sfa.prefix_decode(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], dk, dv, kc, vc, pos, rope=rope)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    tab = rope.cpu()
    for t in range(T):
        new = normal(B, Hq + 2 * Hkv, 64)
        qkv.copy_(new)
        pos.fill_(t)
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        keys, values = kc.cpu(), vc.cpu()
        want = ref.rotated(new[:, Hq:Hq + Hkv], tab[P + t])
        pair = new[:, Hq:Hq + Hkv].double().abs() + new[:, Hq:Hq + Hkv].double().roll(32, -1).abs()
        r = ref.half_step(dtype)
        ref.check("new key", keys[:, :, t], want, r * want.abs() + 3 * (1 + r) * ref.U * pair + 1e-37)
        assert torch.equal(values[:, :, t], new[:, Hq + Hkv:]) and bool(keys[:, :, t + 1:].isnan().all())
        wo, wl, bo, bl = ref.prefix(new[:, :Hq], pk, pv, keys, values, [t] * B, tab)
        ref.check("o", o, wo, bo)
        ref.check("lse", lse, wl, bl)
        every = torch.cat([pv.expand(B, -1, -1, -1), values[:, :, :t + 1]], 2).double().mean(2).repeat_interleave(Hq // Hkv, 1)
        alone, alone_lse, _, _ = ref.forward(ref.rotated(new[:, :Hq], tab[P + t]).transpose(0, 1)[None], pk[None], pv[None])
        for wrong in (torch.zeros_like(wo), every, alone[0].transpose(0, 1)):
            with pytest.raises(AssertionError):
                ref.check("wrong o", wrong, wo, bo)
        with pytest.raises(AssertionError):
            ref.check("wrong lse", alone_lse[0].transpose(0, 1), wl, bl)
    assert sfa.get_device_status() == 0


# ------------------------------------------------------------------ plans that the sizes above do not reach


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv", [(50, 33, 300, 16, 4), (76, 33, 200, 8, 4), (51, 33, 200, 24, 6), (77, 20, 100, 8, 2)])
def test_several_whole_units_an_sm(sfa, B, Tq, Tk, Hq, Hkv, dtype):
    """Batches of equal lengths and more units than SMs: each CTA has whole ones, so that nothing is joined."""
    q, k, v, do = _inputs(50, B, Tq, Tk, Hq, Hkv, dtype)
    _check_forward(sfa, q, k, v, None, None)
    _check_backward(sfa, q, k, v, do, None, None)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_more_sequences_than_threads(sfa, dtype):
    """A CTA's threads share out the sequences: several each, most of them short or empty."""
    B, Tq, Tk, Hq, Hkv = 1601, 9, 40, 4, 1
    q, k, v, do = _inputs(51, B, Tq, Tk, Hq, Hkv, dtype)
    gen = torch.Generator().manual_seed(52)
    nq, nk = (torch.randint(-n, n + 1, (B,), generator=gen).clamp(min=0).tolist() for n in (Tq, Tk))
    q, k, v = _spoil(q, nq), _spoil(k, nk), _spoil(v, nk)
    _check_forward(sfa, q, k, v, nq, nk)
    _check_backward(sfa, q, k, v, do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv", [(3, 1, 1500, 8, 2), (3, 200, 1500, 8, 2), (1, 150, 9000, 6, 2)])
def test_strided_views_with_lengths(sfa, B, Tq, Tk, Hq, Hkv, dtype):
    """[B, T, H, 64] projections as they are, rows behind the lengths NaN, calls of many parts: as dense ones."""
    q, k, v, do = _inputs(53, B, Tq, Tk, Hq, Hkv, dtype)
    nq, nk = [Tq, Tq - Tq // 3, Tq // 2][:B], [Tk - 1, Tk // 3, Tk][:B]
    q, k, v = _spoil(q, nq), _spoil(k, nk), _spoil(v, nk)
    lens = dict(q_len=_i32(nq), kv_len=_i32(nk))
    kv = torch.stack([k, v]).permute(1, 3, 0, 2, 4).contiguous().cuda()  # [B, T, (k, v), H, 64]
    views = q.transpose(1, 2).contiguous().cuda().transpose(1, 2), kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    assert not views[1].is_contiguous()
    o, lse = _check_forward(sfa, q, k, v, nq, nk)
    assert all(torch.equal(a, b) for a, b in zip(sfa.cross_forward(*views, **lens), (o, lse)))
    dense = sfa.cross_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), **lens)
    assert all(torch.equal(a, b) for a, b in zip(sfa.cross_backward(*views, o, lse, do.cuda(), **lens), dense))
    _check_backward(sfa, *(x.cpu() for x in views), do, nq, nk)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk", [(2, 1, 333), (1, 1, 20000), (2, 5, 333), (2, 70, 333), (1, 140, 9000)])
def test_a_logit_of_infinity_makes_its_rows_nan(sfa, B, Tq, Tk, dtype):
    q, k, v, _ = _inputs(44, B, Tq, Tk, 4, 2, dtype)
    k[0, 1, Tk // 3] = INF
    o, lse = _forward(sfa, q.abs() + 0.1, k, v, None, None)
    assert bool(o[0, 2:].isnan().all()) and bool(lse[0, 2:].isnan().all())
    assert bool(o[0, :2].isfinite().all()) and bool(lse[0, :2].isfinite().all()) and bool(o[1:].isfinite().all())

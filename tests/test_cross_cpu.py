"""Attention to states of another length and the decode step behind a prefix, without a GPU: refusals of the C ABI
and of the Python names, workspace sizes, and the plain definitions that the GPU tests use."""
import ctypes as C

import pytest
import torch

import cross_ref as ref

P, ODD = 4096, 4098  # never dereferenced: every call below is refused first


def _desc(**kw):
    from static_offset_sparse_gb300._lib import CrossDesc

    B, Tq, Tk, Hq, Hkv = (kw.get(n, d) for n, d in (("B", 2), ("Tq", 30), ("Tk", 50), ("Hq", 8), ("Hkv", 2)))
    d = dict(B=B, Tq=Tq, Tk=Tk, Hq=Hq, Hkv=Hkv, D=64, dtype=1, q_stride=(64 * Hq * Tq, 64 * Tq, 64),
             k_stride=(64 * Hkv * Tk, 64 * Tk, 64), v_stride=(64 * Hkv * Tk, 64 * Tk, 64))
    d.update(kw)
    for n in ("q_stride", "k_stride", "v_stride"):
        d[n] = (C.c_int64 * 3)(*d[n])
    return CrossDesc(**d)


def _prefix(**kw):
    from static_offset_sparse_gb300._lib import PrefixDesc

    d = dict(B=3, P=100, T=40, Hq=8, Hkv=2, D=64, dtype=1, q_stride=512, k_stride=128, v_stride=128, prefix_k_stride=6400,
             prefix_v_stride=6400)
    d.update(kw)
    return PrefixDesc(**d)


BAD = [(dict(B=0), 1), (dict(Tq=0), 1), (dict(Tk=0), 1), (dict(Tk=-5), 1), (dict(Hkv=0), 1), (dict(dtype=2), 1), (dict(D=128), 2),
       (dict(Hq=7), 2), (dict(Hq=66, Hkv=2), 2), (dict(Tq=(1 << 24) + 1), 2), (dict(B=1 << 20, Tq=1 << 10), 2),
       (dict(B=1 << 20, Tk=1 << 10, Tq=1), 2), (dict(q_stride=(64, 63, 64)), 1), (dict(k_stride=(6400, 3200, 32)), 1),
       (dict(v_stride=(6400, 3200, 68)), 1), (dict(k_stride=(0, 3200, 64)), 1), (dict(v_stride=(6400, -3200, 64)), 1),
       (dict(q_stride=(1 << 38, 1920, 64)), 1), (dict(q_len=ODD), 1), (dict(kv_len=ODD), 1)]


@pytest.mark.parametrize("kw,rc", BAD)
def test_cross_refusals(sfa_lib, kw, rc):
    d, n = _desc(**kw), C.c_size_t(0)
    for back in (0, 1):
        assert sfa_lib.sfa_cross_workspace_size(d, back, C.byref(n)) == rc
    assert sfa_lib.sfa_cross_forward(d, P, P, P, P, P, P, 1 << 40, None) == rc
    assert sfa_lib.sfa_cross_backward(d, *[P] * 10, 1 << 40, None) == rc


def test_cross_pointer_and_workspace_refusals(sfa_lib):
    d, n = _desc(B=1, Tq=1, Tk=5000, Hkv=8), C.c_size_t(0)
    assert sfa_lib.sfa_cross_workspace_size(d, 0, C.byref(n)) == 0 and n.value > 0
    assert sfa_lib.sfa_cross_workspace_size(d, 0, None) == 1
    assert sfa_lib.sfa_cross_workspace_size(None, 0, C.byref(n)) == 1
    for i in range(6):
        for bad in (None, ODD):
            args = [P] * 6
            args[i] = bad
            if bad is None and i == 4:
                continue  # lse may be left out
            args[i] = 4097 if i == 4 else args[i]
            assert sfa_lib.sfa_cross_forward(d, *args, 1 << 40, None) == 1, i
    assert sfa_lib.sfa_cross_forward(d, *[P] * 6, n.value - 1, None) == 3
    for i in range(10):
        for bad in (None, 4097 if i == 4 else ODD):
            args = [P] * 10
            args[i] = bad
            assert sfa_lib.sfa_cross_backward(d, *args, 1 << 40, None) == 1, i
    assert sfa_lib.sfa_cross_workspace_size(d, 1, C.byref(n)) == 0
    assert sfa_lib.sfa_cross_backward(d, *[P] * 10, n.value - 1, None) == 3


def test_strides_of_single_entries_are_not_looked_at(sfa_lib):
    n = C.c_size_t(0)
    d = _desc(B=1, Tq=1, Tk=1, Hq=1, Hkv=1, q_stride=(3, 5, 7), k_stride=(0, -1, 0), v_stride=(1, 1, 1))
    assert sfa_lib.sfa_cross_workspace_size(d, 0, C.byref(n)) == 0


@pytest.mark.parametrize("kw,rc", [(dict(B=0), 1), (dict(P=-1), 1), (dict(T=0), 1), (dict(Hkv=0), 1), (dict(dtype=5), 1), (dict(D=32), 2),
                                   (dict(Hq=7), 2), (dict(Hq=130), 2), (dict(P=(1 << 24) + 1), 2), (dict(B=1 << 22), 2),
                                   (dict(B=1 << 20, T=1 << 12, Hq=2), 2), (dict(q_stride=511), 1), (dict(q_stride=516), 1), (dict(q_stride=448), 1),
                                   (dict(k_stride=64), 1), (dict(v_stride=132), 1), (dict(prefix_k_stride=6336), 1),
                                   (dict(prefix_v_stride=6401), 1), (dict(rope=P, rope_T=139), 1), (dict(rope=ODD, rope_T=140), 1)])
def test_prefix_refusals(sfa_lib, kw, rc):
    n = C.c_size_t(0)
    assert sfa_lib.sfa_prefix_workspace_size(_prefix(**kw), C.byref(n)) == rc
    assert sfa_lib.sfa_prefix_decode(_prefix(**kw), *[P] * 11, 1 << 40, None) == rc


def test_prefix_pointer_and_workspace_refusals(sfa_lib):
    d, n = _prefix(), C.c_size_t(0)
    assert sfa_lib.sfa_prefix_workspace_size(d, C.byref(n)) == 0 and n.value > 0
    assert sfa_lib.sfa_prefix_decode(d, *[P] * 11, n.value - 1, None) == 3
    for i in range(11):
        odd = 4097 if i in (7, 9) else ODD
        for bad in (None, odd):
            args = [P] * 11
            args[i] = bad
            if bad is None and i == 9:
                continue  # lse may be left out
            assert sfa_lib.sfa_prefix_decode(d, *args, 1 << 40, None) == 1, i


def _aligned(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("P,T,parts", [(1000, 64, 9 + 1), (1300, 1000, 10 + 9), (300, 1200, 4 + 10)])
def test_parts_behind_a_prefix_are_not_cut_to_what_a_cluster_takes(sfa_lib, P, T, parts):
    """A prefix's and the own rows' parts, sqrt(rows / 12) each and one for 64 rows at most, are joined through the
    workspace: 32 rows of queries in fp32, then (64 sums, maximum and sum) of each part and row."""
    n = C.c_size_t(0)
    d = _prefix(B=4, P=P, T=T, dtype=0, prefix_k_stride=64 * P, prefix_v_stride=64 * P)
    assert sfa_lib.sfa_prefix_workspace_size(d, C.byref(n)) == 0
    assert n.value == _aligned(32 * 256) + _aligned(parts * 32 * 256) + _aligned(parts * 32 * 8)


def test_python_refusals():
    import static_offset_sparse_gb300 as sfa

    q, k = torch.zeros(1, 2, 3, 64), torch.zeros(1, 2, 5, 64)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.cross_forward(q, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.cross_backward(q, k, k, q, q[..., 0], q)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.prefix_decode(q[:, :, 0], q[:, :, 0], q[:, :, 0], k[0], k[0], k, k, torch.zeros(1, dtype=torch.int32))


# ------------------------------------------------------------------ the definitions themselves


def test_definition_against_a_dense_softmax():
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, h, t, 64, generator=gen, dtype=torch.float64) for h, t in ((4, 5), (2, 7), (2, 7)))
    o, lse, _, _ = ref.forward(q, k, v, [5, 3], [7, 4])
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    s = q @ kk.transpose(-1, -2) / 8
    s[1, :, :, 4:] = -torch.inf
    want = torch.softmax(s, -1) @ vv
    want[1, :, 3:] = 0
    assert torch.allclose(o, want, rtol=0, atol=1e-13)
    assert torch.allclose(lse[0], torch.logsumexp(s[0], -1)) and bool((lse[1, :, 3:] == -torch.inf).all())


def test_gradients_against_differences():
    gen = torch.Generator().manual_seed(2)
    q, k, v, do = (torch.randn(2, h, t, 64, generator=gen, dtype=torch.float64) for h, t in ((4, 3), (2, 6), (2, 6), (4, 3)))
    lens = [3, 2], [6, 4]

    def loss():
        return float((ref.forward(q, k, v, *lens)[0] * do).sum())

    o, lse, _, _ = ref.forward(q, k, v, *lens)
    got, _ = ref.backward(q, k, v, o, lse.nan_to_num(neginf=0.0), do, *lens)
    for x, g in zip((q, k, v), got):
        for i in torch.randint(0, x.numel(), (40,), generator=gen).tolist():
            flat, old, h = x.view(-1), float(x.view(-1)[i]), 1e-5
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            # third-order remainder h^2 and the differences' own rounding, 1e-16 |loss| / h
            assert abs((up - down) / (2 * h) - float(g.view(-1)[i])) < 1e-7


def test_prefix_workspace_size_refuses_cpu_tensors():
    import static_offset_sparse_gb300 as sfa

    cache = torch.zeros(1, 2, 5, 64)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.prefix_workspace_size(torch.zeros(1, 4, 64), torch.zeros(2, 7, 64), cache)

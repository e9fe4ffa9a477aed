"""Plain 64-bit definitions of attention to states of another length and of a decode step behind a shared
prefix, with how far a kernel's numbers may be from them.

Bounds.  u = 2^-24 is half a step of fp32, r that of the tensors' type (bf16 2^-8, fp32 2^-24).  A logit is a sum of
64 products, scaled: off by 66 u S at most, S the sum of its terms' sizes.  A probability then is off by twice that
(its own and its sum's), the exponential's 2^-21, and what n terms added in fp32 lose, n u.  Those that enter a
product in bf16 are rounded once more (r).  Outputs are rounded once (r of the exact value)."""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def lengths(lens, B, T):
    return [T] * B if lens is None else [int(x) for x in lens]


def forward(q, k, v, q_len=None, kv_len=None):
    """o, lse and the bounds of both (CPU tensors in any type)."""
    r = half_step(q.dtype)
    B, Hq, Tq, _ = q.shape
    Hkv, Tk = k.shape[1:3]
    nq, nk = lengths(q_len, B, Tq), lengths(kv_len, B, Tk)
    q, k, v = q.double(), k.double(), v.double()
    o, lse = torch.zeros(B, Hq, Tq, 64, dtype=torch.float64), torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros(B, Hq, Tq, dtype=torch.float64)
    for b in range(B):
        if nk[b] == 0 or nq[b] == 0:
            continue
        for h in range(Hq):
            kk, vv, qq = k[b, h // (Hq // Hkv), :nk[b]], v[b, h // (Hq // Hkv), :nk[b]], q[b, h, :nq[b]]
            s = qq @ kk.T / 8
            size = (qq.abs() @ kk.abs().T / 8).amax(-1, keepdim=True)
            lse[b, h, :nq[b]] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            o[b, h, :nq[b]] = p @ vv
            e = 2 * 66 * U * size + 2.0 ** -20 + nk[b] * U
            bo[b, h, :nq[b]] = (e + (r if r > U else 0) + nk[b] * U) * (p @ vv.abs()) + r * (p @ vv).abs() + 1e-37
            bl[b, h, :nq[b]] = (e + 4 * U * lse[b, h, :nq[b], None].abs())[:, 0]
    return o, lse, bo, bl


def backward(q, k, v, o, lse, do, q_len=None, kv_len=None):
    """(dq, dk, dv) and their bounds, as functions of the o and lse that are given."""
    r = half_step(q.dtype)
    B, Hq, Tq, _ = q.shape
    Hkv, Tk = k.shape[1:3]
    nq, nk = lengths(q_len, B, Tq), lengths(kv_len, B, Tk)
    q, k, v, o, lse, do = (x.double() for x in (q, k, v, o, lse, do))
    g = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    e = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    rr = r if r > U else 0
    for b in range(B):
        if nk[b] == 0 or nq[b] == 0:
            continue
        for h in range(Hq):
            G = h // (Hq // Hkv)
            kk, vv, qq, dd = k[b, G, :nk[b]], v[b, G, :nk[b]], q[b, h, :nq[b]], do[b, h, :nq[b]]
            p = torch.exp(qq @ kk.T / 8 - lse[b, h, :nq[b], None])
            size = qq.abs() @ kk.abs().T / 8 + lse[b, h, :nq[b], None].abs()
            ep = 66 * U * size + 2.0 ** -21  # of each p, relative
            delta = (o[b, h, :nq[b]] * dd).sum(-1, keepdim=True)
            ds = p * (dd @ vv.T - delta)
            terms = dd.abs() @ vv.abs().T + (o[b, h, :nq[b]] * dd).abs().sum(-1, keepdim=True)
            eds = ep * ds.abs() + 66 * U * p * terms  # of each ds, absolute
            n_q, n_k = nk[b], nq[b] * (Hq // Hkv)
            g[0][b, h, :nq[b]] = ds @ kk / 8
            e[0][b, h, :nq[b]] = (eds + (rr + n_q * U) * ds.abs()) @ kk.abs() / 8
            g[1][b, G, :nk[b]] += ds.T @ qq / 8
            e[1][b, G, :nk[b]] += (eds + (rr + n_k * U) * ds.abs()).T @ qq.abs() / 8
            g[2][b, G, :nk[b]] += p.T @ dd
            e[2][b, G, :nk[b]] += ((ep + rr + n_k * U) * p).T @ dd.abs()
    return g, [x + 2 * r * y.abs() + 1e-37 for x, y in zip(e, g)]  # (a sum of parts in fp32, and the output's rounding)


def rotated(x, rows):
    """x [..., 64] rotated by rows [..., 32, 2] (cos, sin) of a RoPE table."""
    a, b, cos, sin = x[..., :32].double(), x[..., 32:].double(), rows[..., 0].double(), rows[..., 1].double()
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def prefix(q, prefix_k, prefix_v, k_cache, v_cache, pos, rope):
    """o, lse and their bounds for caches that hold the step's rows; rows out of range are empty."""
    r = half_step(q.dtype)
    B, Hq, _ = q.shape
    Hkv, P, _ = prefix_k.shape
    T = k_cache.shape[2]
    o, lse = torch.zeros(B, Hq, 64, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    # the query after its rotation: three roundings in fp32, and 2^-16 where it is held in two bf16 parts
    eq = 3 * U + (2.0 ** -16 if r > U else 0)
    for b in range(B):
        t = int(pos[b])
        if not 0 <= t < T:
            continue
        qq = rotated(q[b], rope[P + t]) if rope is not None else q[b].double()
        for h in range(Hq):
            G = h // (Hq // Hkv)
            kk = torch.cat([prefix_k[G], k_cache[b, G, :t + 1]]).double()
            vv = torch.cat([prefix_v[G], v_cache[b, G, :t + 1]]).double()
            s = kk @ qq[h] / 8
            # (a rotated number is off by its pair's size)
            pair = qq[h].abs() + qq[h].roll(32).abs()
            size = (kk.abs() @ qq[h].abs() / 8).max()
            moved = eq * (kk.abs() @ pair / 8).max()
            n = P + t + 1
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            o[b, h] = p @ vv
            e = 2 * (66 * U * size + moved) + 2.0 ** -20 + n * U
            bo[b, h] = (e + (r if r > U else 0) + n * U) * (p @ vv.abs()) + r * o[b, h].abs() + 1e-37
            bl[b, h] = e + 4 * U * lse[b, h].abs()
    return o, lse, bo, bl


def check(name, got, want, bound):
    """Each number within its bound; infinities and NaN in the same places."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{name}: NaN in other places"
    fine = want.isfinite()
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{name}: infinities in other places"
    off = ((got - want).abs() / bound)[fine]
    off[(got == want)[fine]] = 0.0
    if off.numel():
        worst = float(off.max())
        print(f"{name}: {worst:.3f} of the bound")
        assert worst <= 1.0, f"{name}: {worst:.3g} times the bound, {float((got - want)[fine].abs().max()):.3g} off"

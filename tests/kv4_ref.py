"""Plain definitions of the paged 4-bit cache's operators, in numpy and 64 bits."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values():
    """The number of each e4m3 byte (NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f / 512 if e == 0 else 2.0 ** (e - 7) * (1 + f / 8)
        out[b] = np.nan if b & 127 == 127 else (-x if b & 128 else x)
    return out


E4M3 = e4m3_values()


def nearest(x, values):
    """Index of the nearest of the ascending values (their last bits alternate), ties to the even index."""
    mid = (values[1:] + values[:-1]) / 2  # exact: few bits
    lo = np.searchsorted(mid, x, side="left")  # x on a midpoint counts to the lower value
    hi = np.searchsorted(mid, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def quantise(x):
    """fp32 [..., 64] -> codes [..., 64], scale bytes [..., 4], with the stated fp32 quotients."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], 4, 16)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = np.abs(b).max(-1)
        s8 = nearest(np.minimum((m / np.float32(6)).astype(np.float64), 448.0), E4M3[:127])
        s8 = np.where(np.isnan(m), 127, s8)
        s = E4M3[s8].astype(np.float32)[..., None]
        y = np.where(s == 0, np.float32(0), b / s)
        code = nearest(np.minimum(np.abs(y.astype(np.float64)), 6.0), E2M1[:8]) + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), s8.astype(np.uint8)


def values(codes, s8):
    """codes [..., 64] and scale bytes [..., 4] as numbers."""
    return (E2M1[codes].reshape(*codes.shape[:-1], 4, 16) * E4M3[s8][..., None]).reshape(codes.shape)


def rope(T, theta=1e4):
    """fp32 [T, 32, 2] (cos, sin)."""
    a = np.arange(T)[:, None] * theta ** (-np.arange(32) / 32.0)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate32(x, cs):
    """fp32 rotation of x [N, H, 64], each product and sum rounded once."""
    x = np.asarray(x, np.float32)
    c, s, a, b = cs[:, None, :, 0], cs[:, None, :, 1], x[..., :32], x[..., 32:]
    return np.concatenate([a * c - b * s, a * s + b * c], -1)


def rotate(x, cs):
    c, s = cs[:, None, :, 0].astype(np.float64), cs[:, None, :, 1].astype(np.float64)
    a, b = x[..., :32], x[..., 32:]
    return np.concatenate([a * c - b * s, a * s + b * c], -1)


def pack(cache, page, slot, k, v):
    """Write one row's codes and scale bytes (k, v: (codes [H, 64], bytes [H, 4])) into a cache array."""
    p, r = divmod(slot, page)
    for i, (c, s) in enumerate((k, v)):
        cache[p, :, 32 * page * i + 32 * r:][:, :32] = c[:, 0::2] | (c[:, 1::2] << 4)
        cache[p, :, 64 * page + 8 * r + 4 * i:][:, :4] = s


def unpack(cache, page, slots):
    """Stored keys and values [N, H, 64] in 64 bits, scales of 1."""
    out = []
    p, r = np.asarray(slots) // page, np.asarray(slots) % page
    rows = np.asarray(cache)[p]  # [N, H, 72 page]
    for i in (0, 1):
        at = 32 * page * i + 32 * r[:, None] + np.arange(32)
        by = np.take_along_axis(rows, np.broadcast_to(at[:, None], rows.shape[:2] + (32,)), -1)
        st = 64 * page + 8 * r[:, None] + 4 * i + np.arange(4)
        s8 = np.take_along_axis(rows, np.broadcast_to(st[:, None], rows.shape[:2] + (4,)), -1)
        codes = np.stack([by & 15, by >> 4], -1).reshape(*by.shape[:2], 64)
        out.append(values(codes, s8))
    return out


class Pool:
    """The bookkeeping of kv4_plan, request by request."""

    def __init__(self, table, free, lens, page):
        self.table, self.free, self.lens, self.page = table, list(free), list(lens), page

    def step(self, new, rows):
        S, slots, pos, cu = self.page, [], [], [0]
        for r, x in enumerate(new):
            if x < 0:
                self.free += [int(p) for p in self.table[r, :-(-self.lens[r] // S)]]
        for r, x in enumerate(new):
            if x < 0:
                self.lens[r] = 0
            else:
                for j in range(-(-self.lens[r] // S), -(-(self.lens[r] + x) // S)):
                    self.table[r, j] = self.free.pop()
                for p in range(self.lens[r], self.lens[r] + x):
                    slots.append(int(self.table[r, p // S]) * S + p % S)
                    pos.append(p)
                self.lens[r] += x
            cu.append(len(slots))
        fill = [-1] * (rows - len(slots))
        return cu, slots + fill, pos + fill


def attend(q, keys, vals, pos, dist, scale, vscale, cs):
    """One request's rows: q [n, Hq, 64] at positions pos over keys, vals [len, H, 64] (rotated, stored
    numbers).  Returns o, lse and, per row and head, sum p |v| [n, Hq, 64] and the size of the logits'
    terms, max over keys of sum |q_d k_d| / 8: what rounding errors are relative to."""
    n, Hq, _ = q.shape
    H = keys.shape[1]
    G = Hq // H
    x = rotate(q, cs[pos]) if cs is not None else q
    o, lse = np.zeros((n, Hq, 64)), np.full((n, Hq), -np.inf)
    av, sz = np.zeros((n, Hq, 64)), np.zeros((n, Hq))
    for i, p in enumerate(pos):
        js = np.arange(p + 1) if dist is None else np.array(sorted({p - d for d in dist if d <= p}))
        for h in range(Hq):
            k, v = keys[js, h // G] * scale, vals[js, h // G] * vscale
            t = k @ x[i, h] / 8
            m = t.max()
            e = np.exp(t - m)
            z = e.sum()
            o[i, h], lse[i, h] = e @ v / z, m + np.log(z)
            av[i, h] = e @ np.abs(v) / z
            # rotation mixes pairs: the terms' size by the pair's length
            r = np.hypot(x[i, h, :32], x[i, h, 32:])
            sz[i, h] = (np.abs(k) @ np.concatenate([r, r]) / 8).max()
    return o, lse, av, sz


def bounds(o, lse, av, sz, bf16):
    """What a right kernel may be off by.

    Logits: the query's fp32 rotation (3 roundings of 2^-24 of the pair's length), its two f16 parts
    (2^-22), at most 8 chained fp32 accumulations of exact 16-term products, allowed 2^-22 each of the
    terms' size: 2^-22 (0.75 + 1 + 8) < 2^-18.7 of sum |q k| / 8; then the subtraction of the maximum
    and 2^x, 2^-22 of the logit's size and 2^-22: together d = 2^-18.5 sz + 2^-22.  A probability and
    the sum are each off by at most d relatively (first order: 2 d for the quotient; 2^-20 covers the sums'
    own roundings and the second order).  Values: bf16 outputs round probabilities to f16 (2^-11) and
    the result to bf16 (2^-8); fp32 outputs keep 22 bits of probabilities (2^-21) and round to 2^-24.
    """
    d = 2.0 ** -18.5 * sz + 2.0 ** -22
    rel = 2 * d + 2.0 ** -20 + (2.0 ** -11 if bf16 else 2.0 ** -21)
    bo = rel[..., None] * av + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(o) + 1e-30
    bl = d + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
    return bo, bl

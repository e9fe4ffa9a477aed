"""The operators around a paged key/value cache held in 4 bits: their cases and their plain forms.

A cache is uint8 [pages, Hkv, 72 * page]: one (page, head) block holds `page` rows of keys
(32 bytes: 64 dims of e2m1, dim 2i in the low and 2i + 1 in the high half of byte i), then `page`
rows of values (the same), then `page` rows of 8 scales (e4m3: keys' dims 0-15, 16-31, 32-47,
48-63, then the values').  A stored value is code * scale * (kscale or vscale).  Keys are stored
rotated at their own position.  Row p of a request lies in page block_table[request, p // page] at
row p % page; slot = page id * page size + row.

plan     block tables, slot and position maps of one serving step, from request lengths
append   rotates, quantises and writes new key/value rows, and reads back what was stored
read     rows of the cache as numbers
attend   attention of new query rows over the cached prefix, all of it or a shared offset list

`own` chooses between the plain forms below and the package's calls.
"""
import math
import random

import torch

own = False

PHI = 0.6180339887498949  # steps of fractional parts that spread sizes over their range
SQ2 = 0.4142135623730951


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a decode step's bookkeeping: 256 requests, a token each, a few leaving
        dict(name="plan tokens", op="plan", R=256, page=64, len_lo=1, len_hi=8192, new_lo=1, new_hi=1, gone=37),
        # admission of many prompts at once into small pages, requests leaving and idling between
        dict(name="plan prompts", op="plan", R=611, page=16, len_lo=1, len_hi=900, new_lo=1, new_hi=700, gone=5),
        # the new tokens of one layer in a decode step of 32 requests
        dict(name="append tokens", op="append", N=32, T=16384, Hkv=2, page=64, dtype="bf16", ks=1.0, vs=1.0),
        # the rows of a batch of prompts, one layer (32 sequences of 1024, a ragged end)
        dict(name="append prompts", op="append", N=32741, T=2048, Hkv=2, page=16, dtype="bf16", ks=0.5, vs=0.25),
        # a short shared prefix read back, in 32 bits
        dict(name="read prefix", op="read", N=333, Hkv=4, page=32, dtype="f32", ks=1.0, vs=1.0),
        # whole prompts read back for a dense pass over them
        dict(name="read prompts", op="read", N=65536, Hkv=2, page=64, dtype="bf16", ks=1.0, vs=0.5),
        # a decode step on window 0..8 and Fibonacci rungs, caches of up to 16384 rows
        dict(name="offsets tokens", op="attend", R=32, Hq=8, Hkv=2, ctx_lo=1024, ctx_hi=16384, new_lo=1, new_hi=1,
             page=64, dtype="bf16", dist="fib", ks=1.0, vs=1.0),
        # pieces of prompts on the same offsets (32 requests, about 8000 new rows)
        dict(name="offsets prompts", op="attend", R=32, Hq=8, Hkv=2, ctx_lo=1024, ctx_hi=4096, new_lo=100, new_hi=500,
             page=16, dtype="bf16", dist="fib", ks=1.0, vs=1.0),
        # one short request over its whole prefix, in 32 bits: latency alone
        dict(name="prefix token", op="attend", R=1, Hq=8, Hkv=2, ctx_lo=1000, ctx_hi=1000, new_lo=1, new_hi=1,
             page=16, dtype="f32", dist="all", ks=1.0, vs=1.0),
        # one long request over its whole prefix: the work of one row over the whole card
        dict(name="prefix long", op="attend", R=1, Hq=16, Hkv=2, ctx_lo=400001, ctx_hi=400001, new_lo=1, new_hi=1,
             page=64, dtype="bf16", dist="all", ks=0.75, vs=1.0),
        # a serving batch of ragged lengths, a token each, over the whole prefix
        dict(name="prefix batch", op="attend", R=128, Hq=8, Hkv=2, ctx_lo=1024, ctx_hi=32768, new_lo=1, new_hi=1,
             page=64, dtype="bf16", dist="all", ks=1.0, vs=1.0),
        # pieces of prompts over a cached prefix
        dict(name="prefix prompts", op="attend", R=8, Hq=8, Hkv=2, ctx_lo=2048, ctx_hi=16384, new_lo=300, new_hi=700,
             page=64, dtype="bf16", dist="all", ks=1.0, vs=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "read", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    scales = dict(ks=rng.choice([1.0, 0.5, 0.7]), vs=rng.choice([1.0, 0.25, 1.3]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "plan":
        tokens = rng.random() < 0.5
        return dict(op=op, R=_log(rng, 1, 1200), page=page, len_lo=1, len_hi=_log(rng, 30, 6000),
                    new_lo=1, new_hi=1 if tokens else _log(rng, 2, 400), gone=rng.choice([0, 3, 11]))
    if op == "append":
        return dict(op=op, N=_log(rng, 1, 40000), T=_log(rng, 64, 16384), Hkv=rng.choice([1, 2, 4, 5]), page=page,
                    dtype=dtype, **scales)
    if op == "read":
        return dict(op=op, N=_log(rng, 1, 60000), Hkv=rng.choice([1, 2, 4, 5]), page=page, dtype=dtype, **scales)
    Hq, Hkv = rng.choice([(8, 2), (8, 2), (4, 4), (16, 2), (8, 1), (6, 3), (32, 1), (16, 4)])
    if rng.random() < 0.4:  # pieces of prompts
        R, hi = _log(rng, 1, 16), _log(rng, 16, 4000)
        new_hi = min(hi, _log(rng, 2, 300))
        new_lo = max(1, new_hi // 3)
        if rng.random() < 0.3:  # or a few tokens each
            new_lo, new_hi = 1, min(hi, 6)
    else:
        R, hi = _log(rng, 1, 160), _log(rng, 1, 20000)
        new_lo = new_hi = 1
    return dict(op=op, R=R, Hq=Hq, Hkv=Hkv, ctx_lo=max(new_hi, hi // 8), ctx_hi=hi, new_lo=new_lo, new_hi=new_hi, page=page,
                dtype=dtype, dist=rng.choice(["all", "all", "fib", "pow2", "window", "christoffel"]), **scales)


def _spread(n, lo, hi, step):
    """n whole numbers from lo to hi, even in their logarithm."""
    a, b = math.log(lo), math.log(hi + 0.999)
    return [min(hi, max(lo, int(math.exp(a + (b - a) * (((i + 1) * step) % 1.0))))) for i in range(n)]


def _requests(c):
    """Lengths and new rows of each request (fixed by the case; the seed gives the contents)."""
    if c["op"] == "plan":
        lens = [0 if i % 9 == 4 else x for i, x in enumerate(_spread(c["R"], c["len_lo"], c["len_hi"], PHI))]
        new = [0 if i % 13 == 6 else x for i, x in enumerate(_spread(c["R"], c["new_lo"], c["new_hi"], SQ2))]
        if c["gone"]:
            new = [-1 if i % c["gone"] == c["gone"] - 1 else x for i, x in enumerate(new)]
        return lens, new
    new = _spread(c["R"], c["new_lo"], c["new_hi"], SQ2)
    return [max(a, b) for a, b in zip(_spread(c["R"], c["ctx_lo"], c["ctx_hi"], PHI), new)], new


def _dist(c):
    """The offset list of an attend case; None: the whole prefix."""
    if c["dist"] == "all":
        return None
    if c["dist"] == "fib":  # window 0..8 and 1, 2, 3, 5, ..., 987
        f = [1, 2]
        while len(f) < 15:
            f.append(f[-1] + f[-2])
        return sorted(set(range(9)) | set(f))
    if c["dist"] == "pow2":  # window 0..8 and 1, 2, 4, ..., 1024
        return sorted(set(range(9)) | {1 << i for i in range(11)})
    if c["dist"] == "window":
        return list(range(500))
    return sorted({0} | {j for j in range(1024) if (j + 1) * 128 // 1024 - j * 128 // 1024})  # Christoffel 128/1024


def _es(c):
    return 2 if c["dtype"] == "bf16" else 4


def work(c):
    S = c["page"]
    if c["op"] == "plan":
        lens, new = _requests(c)
        rows = sum(max(0, x) for x in new)
        pages = sum(-(-(0 if x < 0 else n) // S) for n, x in zip(lens, new))
        after = sum(-(-(n + x) // S) for n, x in zip(lens, new) if x >= 0)
        gone = sum(-(-n // S) for n, x in zip(lens, new) if x < 0)
        return {"bytes": 4 * (4 * c["R"] + 2 * (after - pages) + 2 * gone + 2 * rows), "flops": rows}
    if c["op"] == "append":
        rows = c["N"] * c["Hkv"]
        return {"bytes": rows * (128 * _es(c) * 2 + 2 * 72) + c["N"] * 8 + min(c["N"], c["T"]) * 256, "flops": rows * 64 * 12}
    if c["op"] == "read":
        rows = c["N"] * c["Hkv"]
        return {"bytes": rows * (128 * _es(c) + 72) + c["N"] * 4, "flops": rows * 128}
    lens, new = _requests(c)
    d, pairs, rows = _dist(c), 0, 0
    for n, x in zip(lens, new):
        if d is None:
            pairs += x * (n - x) + x * (x + 1) // 2
            rows += n
        else:
            # every row that some query reaches: all new ones, and older ones through some offset
            pairs += sum(sum(1 for s in d if s <= p) for p in range(n - x, n))
            seen = set()
            for p in range(n - x, n):
                seen.update(p - s for s in d if s <= p)
            rows += len(seen)
    q = sum(new)
    return {"bytes": rows * c["Hkv"] * 72 + q * c["Hq"] * (128 * _es(c) + 4) + q * 256, "flops": pairs * c["Hq"] * 256}


# ------------------------------------------------------------------ inputs


def _rope(T, device):
    """fp32 [T, 32, 2] (cos, sin) of t * 1e4^(-2j/64), the angles in 64 bits."""
    t = torch.arange(T, dtype=torch.float64, device=device)
    f = torch.pow(torch.tensor(1e4, dtype=torch.float64, device=device), torch.arange(32, dtype=torch.float64, device=device) / -32)
    a = t[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).float()


def _quantise(x):
    """fp32 [..., 64] -> codes uint8 [..., 32], scales uint8 [..., 4]: scale = e4m3(amax / 6) of each
    16 dims (448 at most), code = e2m1(x / scale), both to nearest with ties to even; a zero scale
    has zero codes, a block with a NaN has a NaN scale."""
    b = x.unflatten(-1, (4, 16))
    six = torch.full((1,), 6.0, device=x.device)  # a tensor: torch multiplies by the reciprocal of a number
    s8 = (b.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    y = torch.where(s == 0, torch.zeros_like(b), b / s)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(y).to(torch.uint8)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8)


def _values(codes, scales):
    """The numbers that codes and scales stand for, fp32 [..., 64] (exact)."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float32, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()
    return (lut[c].unflatten(-1, (4, 16)) * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _parts(cache, S):
    """Views of a cache: key codes, value codes [P, Hkv, S, 32] and scales [P, Hkv, S, 8]."""
    k, v, s = cache[..., :32 * S], cache[..., 32 * S:64 * S], cache[..., 64 * S:]
    return k.unflatten(-1, (S, 32)), v.unflatten(-1, (S, 32)), s.unflatten(-1, (S, 8))


def _fill(cache, S, g):
    """Every row of the pool, as normal keys and values leave it, some dims larger than others."""
    P, H = cache.shape[:2]
    k, v, s = _parts(cache, S)
    wide = torch.exp(0.5 * torch.randn((2, H, 1, 64), generator=g, device="cuda"))
    at = max(1, (1 << 24) // (H * S * 64))
    for p in range(0, P, at):
        n = min(at, P - p)
        for i, part in enumerate((k, v)):
            x = torch.randn((n, H, S, 64), generator=g, device="cuda") * wide[i]
            c, sc = _quantise(x)
            part[p:p + n] = c
            s[p:p + n, ..., 4 * i:4 * i + 4] = sc


def _table(lens, S, P, width, g):
    """A block table whose requests hold pages in random order, -1 behind them, and the free pages."""
    order = torch.randperm(P, generator=g, device="cuda").int()
    held = torch.tensor([-(-n // S) for n in lens], device="cuda")
    j = torch.arange(width, device="cuda")
    first = torch.cumsum(held, 0) - held
    has = j[None] < held[:, None]
    table = torch.where(has, order[(first[:, None] + j[None]).clamp(max=P - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), order, int(sum(-(-n // S) for n in lens))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    S, op = c["page"], c["op"]
    s = {"case": c, "op": op, "page": S}
    if op == "plan":
        lens, new = _requests(c)
        most = max(n + max(0, x) for n, x in zip(lens, new))
        width = -(-most // S) + 1
        used = sum(-(-n // S) for n in lens)
        extra = sum(-(-(n + max(0, x)) // S) for n, x in zip(lens, new)) - used
        P = used + extra + 7
        table, order, used = _table(lens, S, P, width, g)
        free = torch.full((P,), -1, dtype=torch.int32, device="cuda")
        free[:P - used] = order[used:]
        s.update(lens=_i32(lens), new=_i32(new), table=table, free=free, n_free=_i32([P - used]), rows=sum(max(0, x) for x in new) + 5)
        return s
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s.update(ks=c["ks"], vs=c["vs"], dtype=dt)
    if op in ("append", "read"):
        N, H = c["N"], c["Hkv"]
        P = -(-(N + 3 * S) // S)
        s["cache"] = torch.zeros((P, H, 72 * S), dtype=torch.uint8, device="cuda")
        # runs of consecutive rows in pages of random order, as requests of many lengths leave them
        pages = torch.randperm(P, generator=g, device="cuda")
        at = torch.arange(N, device="cuda") + int(torch.randint(0, S, (1,), generator=g, device="cuda"))
        s["slots"] = (pages[at // S] * S + at % S).int()
        if op == "read":
            _fill(s["cache"], S, g)
            return s
        s["pos"] = ((torch.arange(N, device="cuda") * 7 + 1 + seed % 5) % c["T"]).int() if N < 64 else (torch.arange(N, device="cuda") % c["T"]).int()
        s["rope"] = _rope(c["T"], "cuda")
        wide = torch.exp(0.5 * torch.randn((2, H, 64), generator=g, device="cuda"))
        s["k"], s["v"] = ((torch.randn((N, H, 64), generator=g, device="cuda") * wide[i]).to(dt) for i in (0, 1))
        return s
    lens, new = _requests(c)
    width = max(-(-n // S) for n in lens)
    P = sum(-(-n // S) for n in lens) + 3
    s["cache"] = torch.empty((P, c["Hkv"], 72 * S), dtype=torch.uint8, device="cuda")
    _fill(s["cache"], S, g)
    s["table"] = _table(lens, S, P, width, g)[0]
    s["lens"] = _i32(lens)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu"] = None if max(new) == 1 else _i32(cu)
    s["most"] = max(new)
    s["rope"] = _rope(width * S, "cuda")
    s["dist"] = _dist(c)
    s["q"] = (1.5 * torch.randn((cu[-1], c["Hq"], 64), generator=g, device="cuda")).to(dt)
    return s


# ------------------------------------------------------------------ plain forms


def _rotate(x, cs):
    """x fp32 [N, H, 64] rotated by cs [N, 32, 2]: pairs (j, j + 32), each product rounded once."""
    c, n = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * n, a * n + b * c], dim=-1)


def _plan(s):
    S, lens, table, free, n_free, rows = s["page"], s["lens"], s["table"], s["free"], s["n_free"], s["rows"]
    dev, F, M = lens.device, free.numel(), table.shape[1]
    gone = s["new"] < 0
    new = s["new"].clamp(min=0)
    held = (lens + S - 1) // S
    kept = torch.where(gone, 0, lens)
    after = kept + new
    have = torch.where(gone, 0, held)
    need = (after + S - 1) // S - have
    back = held - have
    nf = n_free.long()
    j = torch.arange(M, device=dev)
    # the stack of free pages: the old ones, then those of the requests that leave
    rank = (torch.cumsum(back, 0) - back)[:, None] + j
    stack = torch.cat([free, free[:1]])
    stack[torch.where(gone[:, None] & (j < held[:, None]), (nf + rank).clamp(max=F), F)] = table
    top = nf + back.sum()
    rank = (torch.cumsum(need, 0) - need)[:, None] + j - have[:, None]
    takes = (j >= have[:, None]) & (j < (have + need)[:, None])
    table.copy_(torch.where(takes, stack[(top - 1 - rank).clamp(0, F)], table))
    left = top - need.sum()
    i = torch.arange(F, device=dev)
    free.copy_(torch.where((i >= nf) & (i < left), stack[:F], free))
    cu = torch.zeros(lens.numel() + 1, dtype=torch.int32, device=dev)
    cu[1:] = torch.cumsum(new, 0)
    r = torch.arange(rows, device=dev)
    req = torch.searchsorted(cu[1:], r.int(), right=True).clamp(max=lens.numel() - 1)
    pos = kept[req] + r - cu[req]
    fine = r < cu[-1]
    slots = table[req, (pos // S).clamp(0, M - 1)] * S + pos % S
    return {"cu": cu, "slots": torch.where(fine, slots, -1).int(), "pos": torch.where(fine, pos, -1).int(),
            "lens": after.int(), "n_free": left.int(), "table": table, "free": free}


def _read(s, slots):
    S = s["page"]
    k, v, sc = _parts(s["cache"], S)
    p, r = slots.long() // S, slots.long() % S
    scales = sc[p, :, r]
    return ((_values(k[p, :, r], scales[..., :4]) * s["ks"]).to(s["dtype"]), (_values(v[p, :, r], scales[..., 4:]) * s["vs"]).to(s["dtype"]))


def _append(s):
    S = s["page"]
    k, v, sc = _parts(s["cache"], S)
    p, r = s["slots"].long() // S, s["slots"].long() % S
    ks, vs = (torch.full((1,), s[n], dtype=torch.float32, device=sc.device) for n in ("ks", "vs"))
    kc, ksc = _quantise(_rotate(s["k"].float(), s["rope"][s["pos"].long()]) / ks)
    vc, vsc = _quantise(s["v"].float() / vs)
    k[p, :, r], v[p, :, r], sc[p, :, r] = kc, vc, torch.cat([ksc, vsc], dim=-1)
    return _read(s, s["slots"])


def _rows(s):
    """Request, place among its new rows and position of each query row."""
    n = s["q"].shape[0]
    r = torch.arange(n, device=s["q"].device)
    if s["cu"] is None:
        return r, torch.zeros_like(r), s["lens"].long() - 1
    cu = s["cu"].long()
    req = torch.searchsorted(cu[1:], r, right=True)
    return req, r - cu[req], s["lens"].long()[req] - (cu[req + 1] - r)


def _attend(s):
    S, q, dist = s["page"], s["q"], s["dist"]
    N, Hq, D = q.shape
    cache, table = s["cache"], s["table"].long().clamp(min=0)
    H = cache.shape[1]
    G = Hq // H
    req, i, pos = _rows(s)
    q = (_rotate(q.float(), s["rope"][pos]) * 0.125).unflatten(1, (H, G))
    kc, vc, sc = _parts(cache, S)
    if dist is not None:
        at = pos[:, None] - torch.tensor(dist, device=q.device)
        fine = at >= 0
        at = at.clamp(min=0)
        p, r = table[req[:, None], at // S], at % S
        scales = sc[p, :, r]  # [N, n, H, 8]
        x = torch.einsum("nhgd,nkhd->nhgk", q, _values(kc[p, :, r], scales[..., :4]))
        x = (x * s["ks"]).masked_fill(~fine[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        o = torch.einsum("nhgk,nkhd->nhgd", e, _values(vc[p, :, r], scales[..., 4:])) / z * s["vs"]
        lse = m + torch.log(z)
    else:
        R, L, T = table.shape[0], table.shape[1] * S, s["most"]
        qp = torch.zeros((R, H, T, G, D), dtype=torch.float32, device=q.device)
        qp[req, :, i] = q
        scales = sc[table].transpose(1, 2).flatten(2, 3)  # [R, H, L, 8]
        keys = _values(kc[table].transpose(1, 2).flatten(2, 3), scales[..., :4])
        x = torch.matmul(qp.flatten(2, 3), keys.transpose(-1, -2)) * s["ks"]
        del keys
        most = torch.full((R, T), -1, dtype=torch.long, device=q.device)
        most[req, i] = pos
        fine = (torch.arange(L, device=q.device) <= most[..., None]).repeat_interleave(G, dim=1)
        x = x.masked_fill_(~fine[:, None], -math.inf)
        m = x.amax(-1, keepdim=True).clamp(min=-1e30)
        e = x.sub_(m).exp_()
        z = e.sum(-1, keepdim=True)
        o = torch.matmul(e, _values(vc[table].transpose(1, 2).flatten(2, 3), scales[..., 4:])) / z * s["vs"]
        lse = (m + torch.log(z)).unflatten(2, (T, G))[req, :, i]
        o = o.unflatten(2, (T, G))[req, :, i]
    return {"o": o.flatten(1, 2).to(s["dtype"]), "lse": lse.flatten(1)}


# ------------------------------------------------------------------ one pass


def _own(s):
    import static_offset_sparse_gb300 as sfa

    if s["op"] == "plan":
        cu, slots, pos, lens, n_free = sfa.kv4_plan(s["new"], s["lens"], s["table"], s["free"], s["n_free"], page=s["page"], rows=s["rows"])
        return {"cu": cu, "slots": slots, "pos": pos, "lens": lens, "n_free": n_free, "table": s["table"], "free": s["free"]}
    if s["op"] == "append":
        sfa.kv4_append(s["k"], s["v"], s["cache"], s["slots"], s["pos"], rope=s["rope"], kscale=s["ks"], vscale=s["vs"])
    if s["op"] in ("append", "read"):
        return sfa.kv4_read(s["cache"], s["slots"], dtype=s["dtype"], kscale=s["ks"], vscale=s["vs"])
    o, lse = sfa.kv4_attend(s["q"], s["cache"], s["table"], s["lens"], cu_q=s["cu"], dist=s["dist"], rope=s["rope"], kscale=s["ks"], vscale=s["vs"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plan, "append": _append, "attend": _attend}[state["op"]](state) if state["op"] != "read" else _read(state, state["slots"])


# ------------------------------------------------------------------ 64 bits


def _two(e):
    """2^e in 64 bits for whole e, from its bits (pow is not exact on the GPU, and ties need it)."""
    return ((e + 1023) << 52).view(torch.float64)


def _near(x, mantissa, least, most):
    """x in 64 bits to the nearest value with `mantissa` bits behind the leading one, exponents from `least`, at most `most`."""
    e = ((x.abs().contiguous().view(torch.int64) >> 52) - 1023).clamp(min=least)
    step = _two(e - mantissa)
    return (torch.round(x / step) * step).clamp(-most, most)


def _block(cache, S, page, head):
    """One (page, head) block in 64 bits: keys and values [S, 64]."""
    b = cache[page, head].reshape(-1)
    out = []
    for i in (0, 1):
        y = b[32 * S * i:32 * S * (i + 1)].reshape(S, 32)
        n = torch.empty((S, 64), dtype=torch.long, device=b.device)
        n[:, 0::2], n[:, 1::2] = (y % 16).long(), (y // 16).long()
        e, f = (n % 8) // 2, (n % 2).double()
        mag = torch.where(e == 0, 0.5 * f, _two(e - 1) * (1 + 0.5 * f))
        sc = b[64 * S:].reshape(S, 8)[:, 4 * i:4 * i + 4].long()
        se, sf = (sc % 128) // 8, (sc % 8).double()
        sv = torch.where(se == 0, sf / 512, _two(se - 7) * (1 + sf / 8))
        out.append(torch.where(n >= 8, -mag, mag) * sv.repeat_interleave(16, dim=1))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    S, op = s["page"], s["op"]
    if op == "plan":
        return None
    if op == "append":
        out = []
        for x, z, turn in ((s["k"], s["ks"], True), (s["v"], s["vs"], False)):
            x = x.double()
            if turn:
                w = torch.view_as_complex(s["rope"].double())[s["pos"].long()]
                y = torch.complex(x[..., :32], x[..., 32:]) * w[:, None]
                x = torch.cat([y.real, y.imag], dim=-1)
            x = (x / z).reshape(*x.shape[:2], 4, 16)
            sc = _near(x.abs().amax(-1, keepdim=True) / 6, 3, -6, 448.0)
            y = torch.where(sc > 0, x / torch.where(sc > 0, sc, 1.0), 0.0)
            out.append((_near(y, 1, 0, 6.0) * sc * z).flatten(-2))
        return tuple(out)
    cache, H = s["cache"], s["cache"].shape[1]
    if op == "read":
        page, row = s["slots"].long() // S, s["slots"].long() % S
        out = [torch.empty((page.numel(), H, 64), dtype=torch.float64, device="cuda") for _ in (0, 1)]
        for h in range(H):
            b = cache[page, h]
            for i in (0, 1):
                y = b[:, 32 * S * i:32 * S * (i + 1)].reshape(-1, S, 32).gather(1, row[:, None, None].expand(-1, 1, 32))
                sc = b[:, 64 * S:].reshape(-1, S, 8).gather(1, row[:, None, None].expand(-1, 1, 8))[..., 4 * i:4 * i + 4]
                # a pool of one row a page, and the block's own reading of it
                one = torch.cat([y.flatten(1), y.flatten(1), sc.flatten(1), sc.flatten(1)], dim=1)
                flat = torch.cat([one[:, :32].flatten(), one[:, 32:64].flatten(), one[:, 64:].flatten()])
                out[i][:, h] = _block(flat[None, None], page.numel(), 0, 0)[0] * (s["ks"], s["vs"])[i]
        return tuple(out)
    q, dist = s["q"].double(), s["dist"]
    N, Hq, _ = q.shape
    G = Hq // H
    o, lse = torch.empty((N, Hq, 64), dtype=torch.float64, device="cuda"), torch.empty((N, Hq), dtype=torch.float64, device="cuda")
    lens, table = s["lens"].tolist(), s["table"].tolist()
    cu = list(range(len(lens) + 1)) if s["cu"] is None else s["cu"].tolist()
    for r, n in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        at = torch.arange(n - (b - a), n, device="cuda")
        w = torch.view_as_complex(s["rope"].double())[at]
        x = torch.complex(q[a:b, :, :32], q[a:b, :, 32:]) * w[:, None]
        x = torch.cat([x.real, x.imag], dim=-1)
        gap = at[:, None] - torch.arange(n, device="cuda")
        fine = gap >= 0
        if dist is not None:
            among = torch.zeros(max(dist) + 2, dtype=torch.bool, device="cuda")
            among[torch.tensor(dist, device="cuda")] = True
            fine &= among[gap.clamp(0, max(dist) + 1)]
        pages = torch.tensor(table[r][:-(-n // S)], device="cuda")
        for h in range(H):
            b8 = cache[pages, h]  # the request's blocks, joined into one
            k, v = _block(torch.cat([b8[:, :32 * S].flatten(), b8[:, 32 * S:64 * S].flatten(), b8[:, 64 * S:].flatten()])[None, None], len(pages) * S, 0, 0)
            t = torch.einsum("thd,kd->htk", x[:, h * G:(h + 1) * G], k[:n] * s["ks"]) / 8
            t = t.masked_fill(~fine, -math.inf)
            z = torch.logsumexp(t, dim=-1)
            lse[a:b, h * G:(h + 1) * G] = z.T
            o[a:b, h * G:(h + 1) * G] = torch.einsum("htk,kd->thd", torch.exp(t - z[..., None]), v[:n] * s["vs"])
    return {"o": o, "lse": lse}

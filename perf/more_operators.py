"""Attention to states of another length, and decode steps of a batch that shares a prefix: their cases and plain forms.

Head dim 64, logits scaled by 1/8, query head h reads KV head h // (Hq // Hkv).

cross     attention of q [B, Hq, Tq, 64] to an encoder's keys and values [B, Hkv, Tk, 64], sequence b's first
          kv_len[b] rows; rows from q_len[b] on, and rows without a key, are zeros with lse = -inf
grads     its gradients dq, dk, dv from o, lse and dO (zeros behind the lengths)
prefix    one decode step: k_new and v_new of each sequence go to row pos[b] of its own cache (the key rotated
          at P + pos[b]), then q, rotated there too, attends the P rows that all sequences share and rows
          0..pos[b] of its own; keys are held rotated

`own` chooses between the plain forms below and the package's calls.
"""
import math

import torch

own = False

SQ2 = 0.4142135623730951  # steps of fractional parts that spread sizes over their range
PHI = 0.6180339887498949
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a decoder's step over encoder states of a translation or speech batch, one new token each
        dict(name="cross tokens", op="cross", B=32, Tq=1, Tk=1500, Hq=8, Hkv=2, ragged=True, dtype="bf16"),
        # a short prompt of a decoder over ragged sources, in 32 bits
        dict(name="cross short f32", op="cross", B=4, Tq=37, Tk=777, Hq=4, Hkv=4, ragged=True, dtype="f32"),
        # one prompt over one very long source: the work of few rows over the whole card
        dict(name="cross long", op="cross", B=1, Tq=130, Tk=65536, Hq=8, Hkv=2, ragged=False, dtype="bf16"),
        # the forward pass of a training batch, ragged on both sides
        dict(name="cross batch", op="cross", B=32, Tq=1024, Tk=2048, Hq=8, Hkv=2, ragged=True, dtype="bf16"),
        # many queries to a short caption's states, as many KV heads as query heads
        dict(name="grads caption", op="grads", B=4, Tq=4096, Tk=77, Hq=8, Hkv=8, ragged=False, dtype="bf16"),
        # a small training batch in 32 bits
        dict(name="grads f32", op="grads", B=2, Tq=333, Tk=1000, Hq=8, Hkv=2, ragged=True, dtype="f32"),
        # the backward pass of a training batch, ragged on both sides
        dict(name="grads batch", op="grads", B=32, Tq=1024, Tk=2048, Hq=8, Hkv=2, ragged=True, dtype="bf16"),
        # few sequences behind a short instruction, in 32 bits: latency alone
        dict(name="prefix few f32", op="prefix", B=4, P=1000, T=64, Hq=8, Hkv=2, dtype="f32"),
        # a serving batch behind a long document
        dict(name="prefix batch", op="prefix", B=128, P=16384, T=2048, Hq=8, Hkv=2, dtype="bf16"),
        # hundreds of samples of one prompt, 8 query heads a KV head
        dict(name="prefix samples", op="prefix", B=500, P=32001, T=700, Hq=16, Hkv=2, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "grads", "grads", "prefix", "prefix"])
    Hq, Hkv = rng.choice([(8, 2), (8, 2), (4, 4), (16, 2), (8, 1), (6, 2), (12, 4), (32, 1)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "prefix":
        c = dict(op=op, B=_log(rng, 1, 500), P=_log(rng, 1, 32000), T=_log(rng, 1, 4096), Hq=Hq, Hkv=Hkv, dtype=dtype)
        while c["B"] * c["T"] * c["Hkv"] > 1 << 20 or c["B"] * c["Hq"] * (c["P"] + c["T"]) > (1 << 28) / (8 if dtype == "f32" else 1):
            big = max(("B", "P", "T"), key=lambda n: c[n])
            c[big] = (c[big] + 1) // 2
        return c
    c = dict(op=op, B=_log(rng, 1, 48), Tq=1 if op == "cross" and rng.random() < 0.25 else _log(rng, 2, 4096),
             Tk=_log(rng, 1 if op == "cross" else 16, 20000),  # (over one key every gradient but dv is zero)
             Hq=Hq, Hkv=Hkv, ragged=rng.random() < 0.6, dtype=dtype)
    while c["B"] * c["Hq"] * c["Tq"] * c["Tk"] > (1 << 29) / (16 if dtype == "f32" else 1):
        big = max(("B", "Tq", "Tk"), key=lambda n: c[n] * (32 if n == "B" else 1))
        c[big] = (c[big] + 1) // 2
    return c


def _spread(n, lo, hi, step):
    """n whole numbers from lo to hi, even in their logarithm."""
    a, b = math.log(lo), math.log(hi + 0.999)
    return [min(hi, max(lo, int(math.exp(a + (b - a) * (((i + 1) * step) % 1.0))))) for i in range(n)]


def _lengths(c):
    """Valid rows of queries and keys of each sequence (fixed by the case; the seed gives the contents)."""
    if not c["ragged"]:
        return [c["Tq"]] * c["B"], [c["Tk"]] * c["B"]
    nq = [c["Tq"]] * c["B"] if c["Tq"] == 1 else _spread(c["B"], max(1, c["Tq"] // 3), c["Tq"], SQ2)
    nk = [0 if i % 23 == 17 else x for i, x in enumerate(_spread(c["B"], max(1, c["Tk"] // 4), c["Tk"], PHI))]
    return nq, nk


def _rows(c):
    """The row of its own cache at which each sequence of a prefix case stands."""
    return [x - 1 for x in _spread(c["B"], max(1, c["T"] // 8), c["T"], PHI)]


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "prefix":
        own_rows = sum(t + 1 for t in _rows(c))
        return {"bytes": c["Hkv"] * 128 * es * (c["P"] + own_rows) + c["B"] * (c["Hq"] * (128 * es + 4) + c["Hkv"] * 128 * es),
                "flops": 256.0 * c["Hq"] * (c["B"] * c["P"] + own_rows)}
    nq, nk = _lengths(c)
    pairs = c["Hq"] * sum(a * b for a, b in zip(nq, nk))
    rows = c["Hq"] * sum(a for a, b in zip(nq, nk) if b)
    keys = c["Hkv"] * sum(b for a, b in zip(nq, nk) if a)
    whole_q, whole_k = c["B"] * c["Hq"] * c["Tq"], c["B"] * c["Hkv"] * c["Tk"]
    if c["op"] == "cross":  # q, k, v read; o, lse written, whole
        return {"bytes": 64 * es * (rows + 2 * keys + whole_q) + 4 * whole_q, "flops": 256.0 * pairs}
    return {"bytes": 64 * es * (3 * rows + 2 * keys + whole_q + 2 * whole_k) + 4 * rows, "flops": 640.0 * pairs}


# ------------------------------------------------------------------ inputs


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    if c["op"] == "prefix":
        P, T = c["P"], c["T"]
        qkv = normal(B, Hq + 2 * Hkv, 64)  # a projection's rows: query, key and value heads
        angle = torch.arange(P + T, dtype=torch.float64, device="cuda")[:, None] * 1e4 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
        return dict(op=c["op"], q=qkv[:, :Hq], k_new=qkv[:, Hq:Hq + Hkv], v_new=qkv[:, Hq + Hkv:], prefix_k=normal(Hkv, P, 64),
                    prefix_v=normal(Hkv, P, 64), k_cache=normal(B, Hkv, T, 64), v_cache=normal(B, Hkv, T, 64), pos=ints(_rows(c)),
                    rope=torch.stack([angle.cos(), angle.sin()], -1).float())
    nq, nk = _lengths(c)
    s = dict(op=c["op"], q=normal(B, Hq, c["Tq"], 64), k=normal(B, Hkv, c["Tk"], 64), v=normal(B, Hkv, c["Tk"], 64), q_len=None, kv_len=None)
    if c["ragged"]:
        s["q_len"], s["kv_len"] = ints(nq), ints(nk)
    if c["op"] == "grads":
        s["do"] = normal(B, Hq, c["Tq"], 64)
        s["o"], s["lse"] = _cross(s)
    return s


# ------------------------------------------------------------------ plain forms


def _mask(s):
    """Which (query, key) pairs of a cross case count: [B, 1, 1, Tq, Tk], and which queries have a key."""
    B, _, Tq, _ = s["q"].shape
    Tk = s["k"].shape[2]
    i, j = torch.arange(Tq, device="cuda"), torch.arange(Tk, device="cuda")
    if s["kv_len"] is None:
        return torch.ones(1, 1, 1, 1, 1, dtype=torch.bool, device="cuda"), torch.ones(1, 1, 1, 1, 1, dtype=torch.bool, device="cuda")
    rows = (i < s["q_len"][:, None])[:, None, None, :, None]
    keys = (j < s["kv_len"][:, None])[:, None, None, None, :]
    return rows & keys, rows & (s["kv_len"] > 0)[:, None, None, None, None]


def _grouped(s):
    """q as [B, Hkv, G, Tq, 64], k and v as [B, Hkv, 1, Tk, 64], in 32 bits."""
    B, Hq, Tq, _ = s["q"].shape
    Hkv = s["k"].shape[1]
    return s["q"].float().reshape(B, Hkv, Hq // Hkv, Tq, 64), s["k"].float()[:, :, None], s["v"].float()[:, :, None]


def _cross(s):
    q, k, v = _grouped(s)
    mask, some = _mask(s)
    x = (q @ k.transpose(-1, -2) * 0.125).masked_fill(~mask, -math.inf)
    top = x.amax(-1, keepdim=True).masked_fill(~some, 0.0)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v / total).masked_fill(~some, 0.0)
    lse = (top + total.log())[..., 0]
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(s["q"].shape[:3])


def _grads(s):
    q, k, v = _grouped(s)
    do = s["do"].float().reshape(q.shape)
    mask, some = _mask(s)
    lse = s["lse"].reshape(q.shape[:-1])[..., None].masked_fill(~some, 0.0)
    p = (q @ k.transpose(-1, -2) * 0.125 - lse).exp().masked_fill(~mask, 0.0)
    delta = (s["o"].float().reshape(q.shape) * do).sum(-1, keepdim=True)
    ds = p * (do @ v.transpose(-1, -2) - delta) * 0.125
    dq, dk, dv = ds @ k, (ds.transpose(-1, -2) @ q).sum(2), (p.transpose(-1, -2) @ do).sum(2)
    return dq.reshape(s["q"].shape).to(s["q"].dtype), dk.to(s["k"].dtype), dv.to(s["v"].dtype)


def _rotated(x, cos, sin):
    a, b = x.float()[..., :32], x.float()[..., 32:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _prefix(s):
    B, Hq, _ = s["q"].shape
    Hkv, P, _ = s["prefix_k"].shape
    pos = s["pos"].long()
    cos, sin = s["rope"][P + pos][:, None].unbind(-1)
    b = torch.arange(B, device="cuda")
    s["k_cache"][b, :, pos] = _rotated(s["k_new"], cos, sin).to(s["k_cache"].dtype)
    s["v_cache"][b, :, pos] = s["v_new"]
    q = _rotated(s["q"], cos, sin).reshape(B, Hkv, Hq // Hkv, 64) * 0.125
    shared = torch.einsum("bhgd,hpd->bhgp", q, s["prefix_k"].float())
    rest = q @ s["k_cache"].float().transpose(-1, -2)
    rest = rest.masked_fill((torch.arange(rest.shape[-1], device="cuda") > pos[:, None])[:, None, None], -math.inf)
    x = torch.cat([shared, rest], -1)
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (torch.einsum("bhgp,hpd->bhgd", p[..., :P], s["prefix_v"].float()) + p[..., P:] @ s["v_cache"].float()) / total
    return o.reshape(s["q"].shape).to(s["q"].dtype), (top + total.log()).reshape(B, Hq), s["k_cache"], s["v_cache"]


def run(s):
    if own:
        import static_offset_sparse_gb300 as sfa

        if s["op"] == "cross":
            return sfa.cross_forward(s["q"], s["k"], s["v"], q_len=s["q_len"], kv_len=s["kv_len"])
        if s["op"] == "grads":
            return sfa.cross_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], q_len=s["q_len"], kv_len=s["kv_len"])
        o, lse = sfa.prefix_decode(s["q"], s["k_new"], s["v_new"], s["prefix_k"], s["prefix_v"], s["k_cache"], s["v_cache"], s["pos"],
                                   rope=s["rope"])
        return o, lse, s["k_cache"], s["v_cache"]
    return {"cross": _cross, "grads": _grads, "prefix": _prefix}[s["op"]](s)


# ------------------------------------------------------------------ in 64 bits


def _exact_row_block(q, k, v, nk):
    """Probabilities over the first nk keys, their log sum and products, for q [G, rows, 64], k and v [Tk, 64]."""
    x = q @ k[:nk].T / 8
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    return p, lse, p @ v[:nk]


def exact(c, seed):
    s = prepare(c, seed)
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "prefix":
        P, T = c["P"], c["T"]
        freq = 1e4 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), (P + s["pos"].double())[:, None, None] * freq)

        def rotated(x):
            y = torch.complex(x[..., :32].double(), x[..., 32:].double()) * turn
            return torch.cat([y.real, y.imag], -1)

        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        q, new = rotated(s["q"]), rotated(s["k_new"]).to(s["k_cache"].dtype).double()
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        pk, pv = s["prefix_k"].double(), s["prefix_v"].double()
        for b, t in enumerate(_rows(c)):
            kc[b, :, t], vc[b, :, t] = new[b], s["v_new"][b].double()
            for h in range(c["Hkv"]):
                heads = slice(h * G, (h + 1) * G)
                _, lse[b, heads], o[b, heads] = _exact_row_block(q[b, heads], torch.cat([pk[h], kc[b, h, : t + 1]]),
                                                                torch.cat([pv[h], vc[b, h, : t + 1]]), P + t + 1)
        return o, lse, kc, vc
    nq, nk = _lengths(c)
    B, Hq, Tq, _ = s["q"].shape
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    if c["op"] == "cross":
        o, lse = torch.zeros_like(q), torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64, device="cuda")
    else:
        dq, dk, dv, do = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), s["do"].double()
    for b in range(B):
        for h in range(c["Hkv"]):
            at = (b, slice(h * G, (h + 1) * G), slice(0, nq[b]))
            if not nk[b]:
                continue
            p, ls, out = _exact_row_block(q[at], k[b, h], v[b, h], nk[b])
            if c["op"] == "cross":
                o[at], lse[at] = out, ls
                continue
            dp = do[at] @ v[b, h, : nk[b]].T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / 8
            dq[at] = ds @ k[b, h, : nk[b]]
            dk[b, h, : nk[b]] = torch.einsum("gij,gid->jd", ds, q[at])
            dv[b, h, : nk[b]] = torch.einsum("gij,gid->jd", p, do[at])
    return (o, lse) if c["op"] == "cross" else (dq, dk, dv)

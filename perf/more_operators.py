"""The operators between a decoder's projections and behind its logits, as cases
that can be timed and compared: the norm of queries and keys with the rotation
and the write into the paged cache, attention over packed prompts, attention of
drafted tokens over the cache, and log probabilities with their alternatives.

Where `own` is false `run` computes them in elementary torch operations in 32
bits (angles and long sums in 64); where it is true it makes the library's calls.

Layouts: queries, keys and values [tokens][heads][dim] in bf16, rows possibly
part of a wider projection; cache pages [pages][heads][page][dim] in bf16, or
e4m3 with an E8M0 byte per 32 values [pages][heads][page][dim/32]; packed
sequences as offsets [sequences + 1]; drafted tokens see the context and the
drafted tokens whose bits are set in their 64-bit word.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
NEG = float("-inf")


# ---------------------------------------------------------------------------
# Cases.
def _qk(T, Hq, Hkv, D, Dv, R, rot, cache, page, k_out, far, norm=True, pad=0):
    return {"op": "qk", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "Dv": Dv, "R": R, "rot": rot, "cache": cache,
            "page": page, "k_out": k_out, "far": far, "norm": norm, "pad": pad}


def _att(nq, nk, Hq, Hkv, D, Dv, causal=True, tail=0, pad=0):
    """nq, nk: the sequences' lengths as a text, "17,300"."""
    return {"op": "att", "nq": nq, "nk": nk, "Hq": Hq, "Hkv": Hkv, "D": D, "Dv": Dv, "causal": causal,
            "tail": tail, "pad": pad}


def _tree(B, L, spread, n, ragged, Hq, Hkv, D, Dv, cache, page):
    """B sequences of up to L cached tokens (evenly spread from L / spread on), up to n drafted ones each."""
    return {"op": "tree", "B": B, "L": L, "spread": spread, "n": n, "ragged": ragged, "Hq": Hq, "Hkv": Hkv,
            "D": D, "Dv": Dv, "cache": cache, "page": page}


def _lp(T, V, M, k, dtype, ban=0, pad=0):
    return {"op": "lp", "T": T, "V": V, "M": M, "k": k, "dtype": dtype, "ban": ban, "pad": pad}


def listed():
    cases = [
        # decode: the new token's heads, its key and value go into the cache
        ("qk, one token", _qk(1, 64, 8, 128, 128, 128, "halves", "bf16", 64, False, 100000)),
        # a drafted batch with padding rows, part of each head turned, into an 8-bit cache
        ("qk, odd batch to 8 bits", _qk(517, 20, 5, 64, 64, 32, "pairs", "mxfp8", 16, False, 1000000, pad=8)),
        # prefill: a long chunk, keys for the attention and the cache
        ("qk, prefill", _qk(8192, 64, 8, 128, 128, 128, "halves", "bf16", 64, True, 8192)),
        # the smallest prompt
        ("attention, short prompt", _att("37", "37", 64, 8, 128, 128)),
        # ordinary prompts of different lengths, packed, with unused rows behind them
        ("attention, packed prompts", _att("1,700,33,1290,64,2047,129", "1,700,33,1290,64,2047,129", 32, 8, 128, 128,
                                           tail=9, pad=64)),
        # a later chunk of a prompt over all of its keys, queries and keys wider than values
        ("attention, later chunk", _att("512,300", "4608,300", 20, 20, 192, 128)),
        # the longest prompt
        ("attention, long prompt", _att("8192", "8192", 32, 8, 128, 128)),
        # decode: one sequence
        ("tree, one token", _tree(1, 4000, 1, 1, False, 64, 8, 128, 128, "bf16", 64)),
        # drafted trees of a few sequences over an 8-bit cache
        ("tree, drafts over 8 bits", _tree(6, 5000, 4, 16, True, 64, 8, 128, 128, "mxfp8", 32)),
        # decode: a batch with long contexts (the most bytes)
        ("tree, long batch", _tree(32, 32768, 8, 1, False, 64, 8, 128, 128, "bf16", 64)),
        # decode: the sampled token's log probability and its alternatives
        ("logprobs, one token", _lp(1, 163840, 1, 20, "f32")),
        # scoring a batch of drafts, several candidates each
        ("logprobs, batch", _lp(509, 163840, 4, 8, "f32", ban=77)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("qk", "att", "att", "tree", "tree", "lp"))
    if op == "lp":
        V = _log_int(rng, 1000, 163840)
        T = min(_log_int(rng, 1, 2048), 509 * 163840 // V)
        return _lp(T, V, rng.choice((1, 1, 2, 5)), rng.choice((0, 1, 5, 8, 20)), rng.choice(("f32", "f32", "bf16")),
                   rng.choice((0, 0, 13, V // 3)), rng.choice((0, 0, 1, 8)))
    D, Dv = rng.choice(((64, 64), (128, 128), (128, 128), (192, 128)))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    if op == "qk":
        Hq = Hkv * rng.choice((1, 2, 4, 8))
        T = min(_log_int(rng, 1, 8192), 8192 * 80 * 128 // ((Hq + 2 * Hkv) * D))
        return _qk(T, Hq, Hkv, D, Dv, rng.choice((D, D, D // 2, 32)), rng.choice(("halves", "pairs")),
                   rng.choice(("none", "bf16", "bf16", "mxfp8")), rng.choice((16, 32, 64, 256)),
                   rng.choice((True, False)), rng.choice((4096, 131072, 1000000)), rng.choice((True, True, False)),
                   rng.choice((0, 8, 64)))
    if op == "att":
        Hq = Hkv * rng.choice((1, 2, 4))
        total = _log_int(rng, 1, 6000)
        B = min(rng.choice((1, 1, 2, 4, 9)), total)
        cuts = sorted(rng.sample(range(1, total), B - 1)) if B > 1 else []
        nq = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        later = rng.choice((0, 0, 1))
        nk = [n + later * rng.randrange(0, 2000 // B) for n in nq]
        return _att(",".join(map(str, nq)), ",".join(map(str, nk)), Hq, Hkv, D, Dv, rng.random() < 0.8,
                    rng.choice((0, 0, 3)), rng.choice((0, 8, 64)))
    B = _log_int(rng, 1, 64)
    L = min(_log_int(rng, 16, 32768), 32 * 32768 * 8 * 256 // (B * Hkv * (D + Dv)))
    n = rng.choice((1, 1, 1, 4, 8, 16, 40, 64))
    return _tree(B, L, rng.choice((1, 2, 8)), n, n > 1 and rng.random() < 0.5, Hkv * rng.choice((1, 2, 4, 8)), Hkv, D,
                 Dv, rng.choice(("bf16", "bf16", "mxfp8")), rng.choice((16, 32, 64, 256)))


def _ints(text):
    return [int(v) for v in text.split(",")]


def _lens(c):
    """(cached, drafted) tokens of each sequence of a tree case, by the case alone."""
    rng = random.Random(c["B"] * 1000003 + c["L"])
    lens = [c["L"] if b == 0 else rng.randint(c["L"] // c["spread"], c["L"]) for b in range(c["B"])]
    ns = [c["n"] if b == 0 or not c["ragged"] else rng.randint(1, c["n"]) for b in range(c["B"])]
    return lens, ns


def _pairs(nq, nk, causal):
    """Visible pairs of nq queries and nk keys, the last query at the last key."""
    if not causal:
        return nq * nk
    lo = max(0, nq - nk)                  # queries before the first key see none
    first, n = max(1, nk - nq + 1), nq - lo
    return n * (first + nk) // 2


def work(c):
    if c["op"] == "lp":
        n = c["T"] * c["V"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + c["T"] * (8 * c["M"] + 4 + 8 * c["k"]), "flops": 6 * n}
    if c["op"] == "qk":
        T, q, k, v = c["T"], c["Hq"] * c["D"], c["Hkv"] * c["D"], c["Hkv"] * c["Dv"]
        b = 4 * T * q + 2 * T * k * (2 if c["k_out"] else 1)
        if c["cache"] == "bf16":
            b += 2 * T * (k + 2 * v)
        elif c["cache"] == "mxfp8":
            b += T * (k + k // 32 + 2 * v + v + v // 32)
        return {"bytes": b, "flops": 8 * T * (q + k)}
    Hq, Hkv, dims = c["Hq"], c["Hkv"], c["D"] + c["Dv"]
    if c["op"] == "att":
        nq, nk = _ints(c["nq"]), _ints(c["nk"])
        p = sum(_pairs(a, b, c["causal"]) for a, b in zip(nq, nk))
        return {"bytes": sum(nq) * Hq * (2 * dims + 4) + sum(nk) * Hkv * 2 * dims, "flops": 2 * p * Hq * dims}
    lens, ns = _lens(c)
    keys = sum(a + b for a, b in zip(lens, ns)) * Hkv
    b = keys * (2 * dims if c["cache"] == "bf16" else dims + dims // 32)
    return {"bytes": b + sum(ns) * Hq * (2 * dims + 4),
            "flops": 2 * Hq * dims * sum((a + b) * b for a, b in zip(lens, ns))}


# ---------------------------------------------------------------------------
# Inputs.
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device=DEV, generator=g)


def _pool(kind, pages, heads, page, dim, g):
    """Cache pages of near unit variance: (values, E8M0 bytes or None)."""
    if kind == "bf16":
        p = torch.empty((pages, heads, page, dim), dtype=torch.bfloat16, device=DEV)
        return p.normal_(generator=g), None
    v = _randn(g, pages * heads * page, dim)
    q, s = _mxfp8(v)
    return q.view(pages, heads, page, dim), s.view(pages, heads, page, dim // 32)


def _offsets(ns):
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    c = {k: v for k, v in case.items() if k != "name"}
    return {"qk": _prepare_qk, "att": _prepare_att, "tree": _prepare_tree, "lp": _prepare_lp}[c["op"]](c, g, rng)


def _prepare_qk(c, g, rng):
    T, Hq, Hkv, D, Dv, R, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["Dv"], c["R"], c["page"]
    s = {"case": c}
    wide = _randn(g, T, Hq * D + Hkv * (D + Dv) + c["pad"]).to(torch.bfloat16)   # one projection's rows
    s["q"] = wide[:, :Hq * D].view(T, Hq, D)
    s["k"] = wide[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    s["v"] = wide[:, (Hq + Hkv) * D:(Hq + Hkv) * D + Hkv * Dv].view(T, Hkv, Dv)
    s["gq"] = s["gk"] = None
    if c["norm"]:
        s["gq"], s["gk"] = 1.0 + 0.1 * _randn(g, D), 1.0 + 0.1 * _randn(g, D)
    start = rng.randrange(0, c["far"])
    s["pos"] = (start + torch.arange(T, device=DEV)).to(torch.int32)
    s["freq"] = torch.tensor([500000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float32, device=DEV)
    s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    s["k_out"] = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV) if c["k_out"] else None
    s["kc"] = s["vc"] = s["ks"] = s["vs"] = s["slots"] = None
    if c["cache"] != "none":
        pages = -(-T // page) + 1
        s["kc"], s["ks"] = _pool(c["cache"], pages, Hkv, page, D, g)
        s["vc"], s["vs"] = _pool(c["cache"], pages, Hkv, page, Dv, g)
        order = torch.randperm(pages * page, device=DEV, generator=g)[:T]
        # padding rows have no place
        s["slots"] = torch.where(torch.rand(T, device=DEV, generator=g) < 0.05, -1, order) if T > 1 else order
    return s


def _prepare_att(c, g, rng):
    Hq, Hkv, D, Dv = c["Hq"], c["Hkv"], c["D"], c["Dv"]
    nq, nk = _ints(c["nq"]), _ints(c["nk"])
    Tq, Tk = sum(nq) + c["tail"], sum(nk) + c["tail"]
    s = {"case": c, "cu_q": _offsets(nq), "cu_k": _offsets(nk) if nk != nq else None}
    wide = _randn(g, Tk, Hkv * (D + Dv) + c["pad"]).to(torch.bfloat16)
    s["q"] = _randn(g, Tq, Hq, D).mul_(2.0).to(torch.bfloat16)    # some rows attend to few keys
    s["k"], s["v"] = wide[:, :Hkv * D].view(Tk, Hkv, D), wide[:, Hkv * D:Hkv * (D + Dv)].view(Tk, Hkv, Dv)
    s["out"] = torch.zeros((Tq, Hq, Dv), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((Tq, Hq), dtype=torch.float32, device=DEV)
    return s


def _ancestors(n, rng):
    """Words of a random tree of n drafted tokens: each sees itself and its ancestors."""
    words = []
    for i in range(n):
        up = rng.randrange(-1, i) if i else -1
        words.append((words[up] if up >= 0 else 0) | 1 << i)
    return [w - (1 << 64) if w >> 63 else w for w in words]


def _prepare_tree(c, g, rng):
    Hq, Hkv, D, Dv, page, B = c["Hq"], c["Hkv"], c["D"], c["Dv"], c["page"], c["B"]
    lens, ns = _lens(c)
    s = {"case": c, "T": sum(ns)}
    need = [-(-(a + b) // page) for a, b in zip(lens, ns)]
    total = sum(need) + 3
    s["kc"], s["ks"] = _pool(c["cache"], total, Hkv, page, D, g)
    s["vc"], s["vs"] = _pool(c["cache"], total, Hkv, page, Dv, g)
    order = list(range(total))
    rng.shuffle(order)
    table = []
    for b in range(B):
        table.append([order.pop() for _ in range(need[b])] + [-1] * (max(need) + 1 - need[b]))
    s["pages"] = torch.tensor(table, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu_q"] = s["tree"] = None
    s["n"] = c["n"]
    if c["n"] > 1:
        s["cu_q"] = _offsets(ns)
        s["tree"] = torch.tensor([w for n in ns for w in _ancestors(n, rng)], dtype=torch.int64, device=DEV)
    s["q"] = _randn(g, s["T"], Hq, D).mul_(2.0).to(torch.bfloat16)
    s["out"] = torch.empty((s["T"], Hq, Dv), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((s["T"], Hq), dtype=torch.float32, device=DEV)
    return s


def _prepare_lp(c, g, rng):
    T, V, M, k = c["T"], c["V"], c["M"], c["k"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = {"case": c}
    x = torch.empty((T, V + c["pad"]), dtype=dt, device=DEV)[:, :V]
    # rows from nearly even to sure of one token
    x.copy_(_randn(g, T, V) * torch.empty((T, 1), device=DEV).uniform_(0.5, 4.0, generator=g))
    if c["ban"]:
        x[:, V - c["ban"]:] = NEG           # entries behind the vocabulary's end
    s["x"] = x
    s["ids"] = torch.randint(0, V, (T, M), device=DEV, generator=g).to(torch.int32)
    s["ids"][:, 0] = x.argmax(-1)           # a greedy draft among them
    s["lp"] = torch.empty((T, M), dtype=torch.float32, device=DEV)
    s["ent"] = torch.empty((T,), dtype=torch.float32, device=DEV)
    s["top_ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV) if k else None
    s["top_lp"] = torch.empty((T, k), dtype=torch.float32, device=DEV) if k else None
    return s


# ---------------------------------------------------------------------------
# Plain forms, 32 bits.
def _mxfp8(v):
    """(e4m3 [T][W], E8M0 [T][W/32]): per 32 values the smallest power of two
    2^s, s >= -127, that brings them within +-448."""
    T, W = v.shape
    b = v.view(T, W // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    s = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)   # 448 = 0.875 * 2^9
    q = torch.ldexp(b, -s.unsqueeze(-1)).view(T, W).to(torch.float8_e4m3fn)
    return q, (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(p, s):
    """Cache values in 32 bits."""
    if s is None:
        return p.float()
    e = s.view(torch.uint8).to(torch.int32)
    f = torch.where(e == 0, torch.full_like(e, 1 << 22), e << 23).view(torch.float32)
    f = torch.where(e == 255, torch.zeros_like(f), f)
    return (p.float().view(*s.shape, 32) * f.unsqueeze(-1)).view(p.shape)


def _heads(x, gamma, cos, sin, rot):
    """Norm and rotation of [T][H][D] heads, 32 bits."""
    x = x.float()
    if gamma is not None:
        x = x * (1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)) * gamma
    R = 2 * cos.shape[-1]
    if rot == "halves":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y, x[..., R:]), -1)


def _put(pool, bytes_, slots, rows):
    """Rows [n][heads][dim] into their places of the pages."""
    page = pool.shape[2]
    if bytes_ is None:
        pool[slots // page, :, slots % page] = rows.to(torch.bfloat16)
        return
    n, H, D = rows.shape
    q, e = _mxfp8(rows.reshape(n * H, D))
    pool.view(torch.uint8)[slots // page, :, slots % page] = q.view(torch.uint8).view(n, H, D)
    bytes_.view(torch.uint8)[slots // page, :, slots % page] = e.view(torch.uint8).view(n, H, D // 32)


def _plain_qk(s):
    c = s["case"]
    angle = s["pos"].double().unsqueeze(-1) * s["freq"].double()
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    s["q_out"].copy_(_heads(s["q"], s["gq"], cos, sin, c["rot"]))
    k = _heads(s["k"], s["gk"], cos, sin, c["rot"])
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    if s["slots"] is not None:
        has = s["slots"] >= 0
        _put(s["kc"], s["ks"], s["slots"][has], k[has])
        _put(s["vc"], s["vs"], s["slots"][has], s["v"].float()[has])
    return _outputs_qk(s)


def _outputs_qk(s):
    return {n: s[n] for n in ("q_out", "k_out", "kc", "vc", "ks", "vs") if s[n] is not None}


def _weighted(x, v):
    """(softmax(x) v, log of the sum) over the last axis; rows of -inf only give zeros."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(l == 0, torch.ones_like(l), l)
    return o, (m + torch.log(l)).squeeze(-1)


def _plain_att(s):
    c = s["case"]
    Hq, Hkv, D, Dv = c["Hq"], c["Hkv"], c["D"], c["Dv"]
    nq = s["cu_q"][1:] - s["cu_q"][:-1]
    cu_k = s["cu_q"] if s["cu_k"] is None else s["cu_k"]
    nk = cu_k[1:] - cu_k[:-1]
    B, Tq, Tk = nq.numel(), sum(_ints(c["nq"])), sum(_ints(c["nk"]))
    at = torch.arange(B, device=DEV)
    bq, bk = torch.repeat_interleave(at, nq, output_size=Tq), torch.repeat_interleave(at, nk, output_size=Tk)
    iq = torch.arange(Tq, device=DEV) - s["cu_q"][bq] + nk[bq] - nq[bq]
    ik = torch.arange(Tk, device=DEV) - cu_k[bk]
    see = bq.unsqueeze(1) == bk
    if c["causal"]:
        see &= ik <= iq.unsqueeze(1)
    q = s["q"][:Tq].float().permute(1, 0, 2).reshape(Hkv, Hq // Hkv * Tq, D)
    k, v = s["k"][:Tk].float().permute(1, 2, 0).contiguous(), s["v"][:Tk].float().permute(1, 0, 2).contiguous()
    x = torch.matmul(q, k).mul_(D ** -0.5).view(Hkv, Hq // Hkv, Tq, Tk).masked_fill_(~see, NEG)
    o, lse = _weighted(x.view(Hkv, Hq // Hkv * Tq, Tk), v)
    s["out"][:Tq] = o.view(Hq, Tq, Dv).permute(1, 0, 2)
    s["lse"][:Tq] = lse.view(Hq, Tq).t()
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tree(s):
    c = s["case"]
    Hq, Hkv, D, Dv, B, n, page = c["Hq"], c["Hkv"], c["D"], c["Dv"], c["B"], c["n"], c["page"]
    G, L = Hq // Hkv, c["L"] + n
    pos = torch.arange(L, device=DEV)
    at = s["pages"][:, pos // page].long().clamp(min=0)                             # [B][L]
    k = _values(s["kc"][at, :, pos % page], None if s["ks"] is None else s["ks"][at, :, pos % page])   # [B][L][Hkv][D]
    v = _values(s["vc"][at, :, pos % page], None if s["vs"] is None else s["vs"][at, :, pos % page])
    if s["cu_q"] is None:
        rows, have = torch.arange(B, device=DEV).unsqueeze(1), torch.ones((B, 1), dtype=torch.bool, device=DEV)
        words = torch.ones((B, 1), dtype=torch.int64, device=DEV)
    else:
        i = torch.arange(n, device=DEV)
        have = i < (s["cu_q"][1:] - s["cu_q"][:-1]).unsqueeze(1)
        rows = torch.where(have, s["cu_q"][:-1].unsqueeze(1) + i, 0)
        words = torch.where(have, s["tree"][rows], 0)                              # [B][n]
    j = pos - s["lens"].unsqueeze(1)                                               # [B][L]: place among the drafted
    bit = (words.unsqueeze(2) >> j.clamp(0, 63).unsqueeze(1)) & 1
    see = (j < 0).unsqueeze(1) | ((j >= 0) & (j < 64)).unsqueeze(1) & (bit == 1)   # [B][n][L]
    q = s["q"][rows].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B * Hkv, G * n, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1).reshape(B * Hkv, D, L)).mul_(D ** -0.5)
    x = x.view(B, Hkv * G, n, L).masked_fill_(~see.unsqueeze(1), NEG).view(B * Hkv, G * n, L)
    o, lse = _weighted(x, v.permute(0, 2, 1, 3).reshape(B * Hkv, L, Dv))
    o = o.view(B, Hq, n, Dv).permute(0, 2, 1, 3)
    lse = lse.view(B, Hq, n).permute(0, 2, 1)
    s["out"][rows[have]] = o[have].to(torch.bfloat16)
    s["lse"][rows[have]] = lse[have]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_lp(s):
    x = s["x"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    total = e.double().sum(-1, keepdim=True)
    log = torch.log(total)
    s["lp"].copy_(d.gather(1, s["ids"].long()).double() - log)
    part = torch.where(e > 0, -d * e, torch.zeros_like(e)).double().sum(-1, keepdim=True)
    s["ent"].copy_((log + part / total).squeeze(1))
    if s["top_ids"] is not None:
        k = s["top_ids"].shape[1]
        top = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :k]        # equal ones in order
        s["top_ids"].copy_(top)
        s["top_lp"].copy_(d.gather(1, top).double() - log)
    return _outputs_lp(s)


def _outputs_lp(s):
    return {n: s[n] for n in ("lp", "ent", "top_ids", "top_lp") if s[n] is not None}


# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"qk": _plain_qk, "att": _plain_att, "tree": _plain_tree, "lp": _plain_lp}[op](s)
    import mxfp4_routed_expert_sigmoid_amd as k3
    c = s["case"]
    if op == "qk":
        k3.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], gamma_q=s["gq"], gamma_k=s["gk"], eps=EPS,
                        rot=k3.ROT_HALVES if c["rot"] == "halves" else k3.ROT_PAIRS, q_out=s["q_out"],
                        k_out=s["k_out"], v=None if s["slots"] is None else s["v"], kc=s["kc"], vc=s["vc"],
                        ks=s["ks"], vs=s["vs"], slots=s["slots"])
        return _outputs_qk(s)
    if op == "att":
        k3.attention(s["q"], s["k"], s["v"], s["cu_q"], s["out"], cu_k=s["cu_k"], scale=c["D"] ** -0.5,
                     causal=c["causal"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "tree":
        if "ws" not in s:      # a program keeps its workspace
            s["ws"] = k3.tree_attention_workspace(c["Hq"], c["Hkv"], c["Dv"], s["n"], device=s["q"].device)
        k3.tree_attention(s["q"], s["kc"], s["vc"], s["pages"], s["lens"], s["out"], ks=s["ks"], vs=s["vs"],
                          cu_q=s["cu_q"], max_q=s["n"], tree=s["tree"], scale=c["D"] ** -0.5, lse=s["lse"],
                          workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if "ws" not in s:
        s["ws"] = k3.logprobs_workspace(c["T"], c["V"], c["k"], device=s["x"].device)
    k3.logprobs(s["x"], ids=s["ids"], lp=s["lp"], entropy=s["ent"], top_ids=s["top_ids"], top_lp=s["top_lp"],
                workspace=s["ws"])
    return _outputs_lp(s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits: values before their last rounding.
def _exact_heads(x, gamma, pos, freq, rot):
    x = x.double()
    if gamma is not None:
        ss = (x * x).sum(-1) / x.shape[-1]
        x = x / torch.sqrt(ss + EPS)[..., None] * gamma.double()
    y, half = x.clone(), freq.numel()
    for i in range(half):
        a = pos.double() * freq[i].double()
        lo, hi = (i, i + half) if rot == "halves" else (2 * i, 2 * i + 1)
        z = torch.polar(torch.ones_like(a), a)[:, None] * torch.complex(x[..., lo], x[..., hi])
        y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_put(pool, scales, slots, rows):
    """The pages in 64 bits with the rows in their places: (values over their scale, scale)."""
    page = pool.shape[2]
    out = pool.double()
    if scales is None:
        out[slots // page, :, slots % page] = rows
        return out, None
    sc = torch.exp2(scales.view(torch.uint8).double() - 127)
    n, H, D = rows.shape
    b = rows.view(n, H, D // 32, 32)
    a = b.abs().amax(-1)
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448)).clamp(min=-127)
    out[slots // page, :, slots % page] = (b / torch.exp2(e)[..., None]).view(n, H, D)
    sc[slots // page, :, slots % page] = torch.exp2(e)
    return out, sc


def _exact_rows(q, k, v, see, scale):
    """One head: softmax(scale q k^T where seen) v and the log of its sum; an empty row is zero."""
    w = torch.where(see, (q @ k.T) * scale, torch.full((), NEG, dtype=torch.float64, device=DEV))
    lse = torch.logsumexp(w, -1)
    p = torch.exp(w - torch.where(lse == NEG, torch.zeros_like(lse), lse)[:, None])
    return p @ v, lse


def _exact_attend(s, spans, key_rows, see_of):
    c = s["case"]
    out, lse = s["out"].double().zero_(), s["lse"].double().zero_()
    G = c["Hq"] // c["Hkv"]
    for b, (lo, hi) in enumerate(spans):
        see = see_of(b)
        for h in range(c["Hkv"]):
            k, v = key_rows(b, h)
            for g in range(h * G, h * G + G):
                out[lo:hi, g], lse[lo:hi, g] = _exact_rows(s["q"][lo:hi, g].double(), k, v, see, c["D"] ** -0.5)
    return {"out": out, "lse": lse}


def _exact_att(s):
    c = s["case"]
    nq, nk = _ints(c["nq"]), _ints(c["nk"])
    oq, ok = [sum(nq[:b]) for b in range(len(nq))], [sum(nk[:b]) for b in range(len(nk))]

    def see_of(b):
        full = torch.ones((nq[b], nk[b]), dtype=torch.bool, device=DEV)
        return full.tril(nk[b] - nq[b]) if c["causal"] else full

    return _exact_attend(s, [(o, o + n) for o, n in zip(oq, nq)],
                         lambda b, h: (s["k"][ok[b]:ok[b] + nk[b], h].double(), s["v"][ok[b]:ok[b] + nk[b], h].double()),
                         see_of)


def _exact_tree(s):
    c = s["case"]
    lens, ns = _lens(c)
    first = [sum(ns[:b]) for b in range(c["B"])]
    words = [[1]] * c["B"] if s["tree"] is None else [s["tree"][f:f + n].tolist() for f, n in zip(first, ns)]

    def rows(pool, scales, b, h):
        used = s["pages"][b, :-(-(lens[b] + ns[b]) // c["page"])].long()
        r = pool[used, h].double().flatten(0, 1)
        if scales is not None:
            r = r * torch.exp2(scales[used, h].view(torch.uint8).double() - 127).flatten(0, 1).repeat_interleave(32, -1)
        return r[:lens[b] + ns[b]]

    def see_of(b):
        drafted = [[w >> j & 1 == 1 for j in range(ns[b])] for w in words[b]]
        return torch.cat((torch.ones((ns[b], lens[b]), dtype=torch.bool, device=DEV),
                          torch.tensor(drafted, dtype=torch.bool, device=DEV)), 1)

    return _exact_attend(s, [(f, f + n) for f, n in zip(first, ns)],
                         lambda b, h: (rows(s["kc"], s["ks"], b, h), rows(s["vc"], s["vs"], b, h)), see_of)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "att":
        return _exact_att(s)
    if c["op"] == "tree":
        return _exact_tree(s)
    if c["op"] == "qk":
        out = {"q_out": _exact_heads(s["q"], s["gq"], s["pos"], s["freq"], c["rot"])}
        k = _exact_heads(s["k"], s["gk"], s["pos"], s["freq"], c["rot"])
        if s["k_out"] is not None:
            out["k_out"] = k
        if s["slots"] is not None:
            has = torch.nonzero(s["slots"] >= 0).squeeze(1)
            kc, ks = _exact_put(s["kc"], s["ks"], s["slots"][has], k[has])
            vc, vs = _exact_put(s["vc"], s["vs"], s["slots"][has], s["v"].double()[has])
            out["kc"], out["vc"] = kc, vc
            if ks is not None:
                out["ks"], out["vs"] = ks, vs
        return out
    x = s["x"].double()
    p = torch.log_softmax(x, -1)
    out = {"lp": torch.take_along_dim(p, s["ids"].long(), 1),
           "ent": -torch.special.xlogy(torch.exp(p), torch.exp(p)).sum(-1)}
    if s["top_ids"] is not None:
        # largest first, equal ones by their number: one at a time
        ids = torch.empty(s["top_ids"].shape, dtype=torch.int64, device=DEV)
        left = x.clone()
        number = torch.arange(x.shape[1], device=DEV)
        for j in range(ids.shape[1]):
            best = left.amax(-1, keepdim=True)
            ids[:, j] = torch.where(left == best, number, x.shape[1]).amin(-1)
            left.scatter_(1, ids[:, j:j + 1], float("nan"))
            left = torch.where(torch.isnan(left), torch.full((), NEG, dtype=torch.float64, device=DEV), left)
        out["top_ids"], out["top_lp"] = ids.to(torch.int32), torch.take_along_dim(p, ids, 1)
    return out

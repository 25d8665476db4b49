"""The dense operators around the expert layer, as cases that can be timed and
compared: the residual addition with RMS norm (bf16 tokens or tokens in 8 bits
with a scale per 32), products with MXFP4 matrices, and the gated first half of
a dense MLP.

Where `own` is false `run` computes them in elementary torch operations in 32
bits; where it is true it makes the library's calls. MXFP4 weights are packed
nibbles [N][K/2] (E2M1, low nibble first) with E8M0 bytes [N][K/32]; MXFP8
tokens are e4m3 [T][K] with E8M0 bytes [T][ceil(K/32)].
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
SITU, SWIGLU = 1, 2
B1, B2 = 4.0, 25.0      # SiTU betas
# E2M1 magnitudes by code; bit 3 is the sign
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# Cases.
def _norm(T, H, d, out, pad=0):
    return {"op": "norm", "T": T, "H": H, "d": d, "out": out, "pad": pad}


def _linear(T, N, K, x, out):
    return {"op": "linear", "T": T, "N": N, "K": K, "x": x, "out": out}


def _glu(T, I, K, x, out, act):
    return {"op": "glu", "T": T, "N": I, "K": K, "x": x, "out": out, "act": act}


def listed():
    cases = [
        # decode: the attention output of one token joins the residual stream
        ("norm, one token", _norm(1, 7168, "bf16", "bf16")),
        # a decode batch whose next product takes 8-bit tokens
        ("norm, decode batch to 8 bits", _norm(32, 7168, "f32", "mxfp8")),
        # a narrow odd width in a wider buffer, both forms of the tokens
        ("norm, odd width", _norm(517, 1999, "bf16", "both", 9)),
        # prefill: a long chunk to 8-bit tokens
        ("norm, prefill to 8 bits", _norm(8192, 7168, "bf16", "mxfp8")),
        # decode: a narrow projection of one token (the smallest product)
        ("linear, one token, narrow", _linear(1, 1536, 7168, "bf16", "bf16")),
        # decode: the second half of a dense MLP, added into the stream
        ("linear, one token, down", _linear(1, 7168, 18432, "bf16", "add")),
        # decode: the logits of a few tokens
        ("linear, logits", _linear(4, 163840, 7168, "mxfp8", "f32")),
        # a decode batch through a square projection
        ("linear, batch", _linear(48, 7168, 7168, "mxfp8", "bf16")),
        # a ragged chunk with odd sizes
        ("linear, odd sizes", _linear(301, 1001, 2080, "bf16", "f32")),
        # prefill: the second half of a dense MLP, added into the stream
        ("linear, prefill down", _linear(2048, 7168, 18432, "mxfp8", "add")),
        # decode: the first half of a dense MLP for one token
        ("glu, one token", _glu(1, 18432, 7168, "bf16", "bf16", SITU)),
        # a ragged prefill chunk, 8-bit tokens in and out
        ("glu, ragged prefill", _glu(1000, 6144, 7168, "mxfp8", "mxfp8", SWIGLU)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "glu"))
    if op == "norm":
        H = _log_int(rng, 96, 8192)
        T = _log_int(rng, 1, 8192)
        return _norm(T, H, rng.choice(("none", "bf16", "f32")), rng.choice(("bf16", "mxfp8", "both")),
                     rng.choice((0, 0, 1, 9)))
    T = _log_int(rng, 1, 2048)
    K = 32 * _log_int(rng, 8, 576)
    x = rng.choice(("bf16", "mxfp8"))
    if op == "linear":
        # no more weights, and no more products, than the largest listed cases
        N = min(_log_int(rng, 64, 163840), 163840 * 7168 // K)
        T = min(T, max(1, 2048 * 7168 * 18432 // (N * K)))
        return _linear(T, N, K, x, rng.choice(("bf16", "f32", "add")))
    I = _log_int(rng, 32, 2560)
    return _glu(T, I, K, x, rng.choice(("bf16", "mxfp8")), rng.choice((SITU, SWIGLU)))


def work(c):
    T = c["T"]
    if c["op"] == "norm":
        H, G = c["H"], -(-c["H"] // 32)
        b = 4 * T * H + 4 * H
        if c["d"] != "none":
            b += (2 if c["d"] == "bf16" else 4) * T * H + 4 * T * H   # d read, h written
        b += {"bf16": 2 * T * H, "mxfp8": T * (H + G), "both": 3 * T * H + T * G}[c["out"]]
        return {"bytes": b, "flops": 8 * T * H}
    N, K, mats = c["N"], c["K"], 2 if c["op"] == "glu" else 1
    b = mats * N * (K // 2 + K // 32)
    b += T * (2 * K if c["x"] == "bf16" else K + K // 32)
    b += {"bf16": 2 * T * N, "f32": 4 * T * N, "add": 8 * T * N, "mxfp8": T * (N + -(-N // 32))}[c["out"]]
    return {"bytes": b, "flops": 2 * mats * T * N * K}


# ---------------------------------------------------------------------------
# Inputs.
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _wide(T, W, pad, dtype):
    """A [T][W] view of a buffer whose rows are pad elements wider."""
    return torch.empty((T, W + pad), dtype=dtype, device=DEV)[:, :W]


def _matrix(N, K, g):
    """Packed codes of every value and scales that give rows of about unit norm."""
    packed = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    mid = 127 - round(math.log2(2.93 * math.sqrt(K)))
    scales = torch.randint(mid - 2, mid + 2, (N, K // 32), device=DEV, generator=g).to(torch.uint8)
    return packed, scales


def _tokens(T, K, kind, g):
    """Tokens as a norm leaves them: near unit variance, a few strong channels."""
    v = torch.randn((T, K), device=DEV, generator=g)
    v *= torch.where(torch.rand(K, device=DEV, generator=g) < 0.01, 8.0, 1.0)
    if kind == "bf16":
        return v.to(torch.bfloat16), None
    return _mxfp8(v)


def prepare(case, seed):
    g = _gen(seed)
    c = {k: v for k, v in case.items() if k != "name"}
    T, s = c["T"], {"case": c}
    if c["op"] == "norm":
        H, pad = c["H"], c["pad"]
        h = _wide(T, H, pad, torch.float32)
        h.copy_(torch.randn((T, H), device=DEV, generator=g) * 4.0)
        s["h"] = h
        s["d"] = None
        if c["d"] != "none":
            d = _wide(T, H, pad, torch.bfloat16 if c["d"] == "bf16" else torch.float32)
            s["d"] = d.copy_(torch.randn((T, H), device=DEV, generator=g))
        s["gamma"] = 1.0 + 0.1 * torch.randn(H, device=DEV, generator=g)
        s["x"] = s["q"] = s["qs"] = None
        if c["out"] != "mxfp8":
            s["x"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        if c["out"] != "bf16":
            s["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
            s["qs"] = torch.empty((T, -(-H // 32)), dtype=torch.float8_e8m0fnu, device=DEV)
        return s
    N, K = c["N"], c["K"]
    s["w"] = [_matrix(N, K, g) for _ in range(2 if c["op"] == "glu" else 1)]
    s["x"], s["xs"] = _tokens(T, K, c["x"], g)
    s["outs"] = None
    if c["out"] == "add":
        s["out"] = torch.randn((T, N), device=DEV, generator=g) * 4.0
    elif c["out"] == "mxfp8":
        s["out"] = torch.empty((T, N), dtype=torch.float8_e4m3fn, device=DEV)
        s["outs"] = torch.empty((T, -(-N // 32)), dtype=torch.float8_e8m0fnu, device=DEV)
    else:
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# Plain forms, 32 bits.
def _mxfp8(v):
    """(e4m3 [T][W], E8M0 [T][ceil(W/32)]): per 32 values the smallest power of
    two 2^s, s >= -127, that brings them within +-448."""
    T, W = v.shape
    G = -(-W // 32)
    b = torch.nn.functional.pad(v, (0, 32 * G - W)).view(T, G, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    s = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)   # 448 = 0.875 * 2^9
    q = torch.ldexp(b, -s.unsqueeze(-1)).view(T, 32 * G)[:, :W].contiguous().to(torch.float8_e4m3fn)
    return q, (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _pow2(byte):
    """2^(byte - 127) in 32 bits, 0 where the byte is 255."""
    e = byte.to(torch.int32)
    p = torch.where(e == 0, torch.tensor(1 << 22, dtype=torch.int32, device=e.device), e << 23).view(torch.float32)
    return torch.where(e == 255, torch.zeros_like(p), p)


def _dense(packed, scales):
    """An MXFP4 matrix as fp32 [N][K]."""
    N, half = packed.shape
    lut = torch.tensor(MAGS + tuple(-m for m in MAGS), dtype=torch.float32, device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).view(N, 2 * half)
    w = lut[codes.to(torch.int32)]
    return (w.view(N, -1, 32) * _pow2(scales).unsqueeze(-1)).view(N, 2 * half)


def _values(x, xs):
    """Tokens as fp32 [T][K]."""
    if xs is None:
        return x.float()
    T, K = x.shape
    return (x.float().view(T, K // 32, 32) * _pow2(xs.view(torch.uint8)).unsqueeze(-1)).view(T, K)


def _act(g, u, act):
    sg = 1.0 / (1.0 + torch.exp(-g))
    if act == SITU:
        return (B1 * torch.tanh(g / B1) * sg) * (B2 * torch.tanh(u / B2))
    return g * sg * u


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        h = s["h"]
        out = {}
        if s["d"] is not None:
            h += s["d"]
            out["h"] = h
        ss = h.double().square().mean(-1, keepdim=True)
        v = h * (1.0 / torch.sqrt(ss + EPS)).float() * s["gamma"]
        if s["x"] is not None:
            out["x"] = v.to(torch.bfloat16)
        if s["q"] is not None:
            out["q"], out["qs"] = _mxfp8(v)
        return out
    x = _values(s["x"], s["xs"])
    y = [x @ _dense(*w).t() for w in s["w"]]
    if c["op"] == "glu":
        a = _act(y[0], y[1], c["act"])
        if c["out"] == "mxfp8":
            q, qs = _mxfp8(a)
            return {"q": q, "qs": qs}
        return {"out": a.to(torch.bfloat16)}
    if c["out"] == "add":
        s["out"] += y[0]
        return {"out": s["out"]}
    return {"out": y[0].to(torch.bfloat16) if c["out"] == "bf16" else y[0]}


# ---------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import mxfp4_routed_expert_sigmoid_amd as k3
    c = s["case"]
    if c["op"] == "norm":
        k3.add_norm(s["h"], s["gamma"], EPS, d=s["d"], x=s["x"], q=s["q"], qs=s["qs"])
        out = {} if s["d"] is None else {"h": s["h"]}
        if s["x"] is not None:
            out["x"] = s["x"]
        if s["q"] is not None:
            out["q"], out["qs"] = s["q"], s["qs"]
        return out
    if c["op"] == "glu":
        k3.glu(*s["w"][0], *s["w"][1], s["x"], s["out"], xs=s["xs"], outs=s["outs"], act=c["act"],
               situ_b1=B1, situ_b2=B2)
        return {"out": s["out"]} if s["outs"] is None else {"q": s["out"], "qs": s["outs"]}
    k3.linear(*s["w"][0], s["x"], s["out"], xs=s["xs"], accumulate=c["out"] == "add")
    return {"out": s["out"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits: values before their last rounding.
def _exact_dense(packed, scales):
    p = packed.to(torch.int64)
    code = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=torch.int64, device=p.device)
    code[:, 0::2], code[:, 1::2] = p % 16, p // 16
    m, e = code % 2, (code // 2) % 4          # E2M1: mantissa bit, exponent bits (bias 1)
    mag = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2((e - 1).double()))
    mag = torch.where(code >= 8, -mag, mag)
    b = scales.to(torch.int64).repeat_interleave(32, 1)
    return torch.where(b == 255, torch.zeros_like(mag), mag * torch.exp2((b - 127).double()))


def _exact_tokens(x, xs):
    v = x.double()
    if xs is None:
        return v
    b = xs.view(torch.uint8).to(torch.int64).repeat_interleave(32, 1)[:, :v.shape[1]]
    return torch.where(b == 255, torch.zeros_like(v), v * torch.exp2((b - 127).double()))


def _exact_mxfp8(v):
    """Scales, and the values over them before their rounding to e4m3."""
    T, W = v.shape
    qs = torch.zeros((T, -(-W // 32)), dtype=torch.float64, device=v.device)
    for j in range(qs.shape[1]):
        a = v[:, 32 * j:32 * j + 32].abs().amax(1)
        qs[:, j] = torch.exp2(torch.ceil(torch.log2(a / 448.0)).clamp(min=-127.0))
    return v / qs.repeat_interleave(32, 1)[:, :W], qs


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        h = s["h"].double()
        out = {}
        if s["d"] is not None:
            h = h + s["d"].double()
            out["h"] = h
        inv = torch.rsqrt((h * h).sum(1) / h.shape[1] + EPS)
        v = h * inv[:, None] * s["gamma"].double()[None, :]
        if s["x"] is not None:
            out["x"] = v
        if s["q"] is not None:
            out["q"], out["qs"] = _exact_mxfp8(v)
        return out
    x = _exact_tokens(s["x"], s["xs"])
    y = []
    for packed, scales in s["w"]:
        parts = [torch.matmul(x, _exact_dense(packed[i:i + 8192], scales[i:i + 8192]).t().contiguous())
                 for i in range(0, packed.shape[0], 8192)]
        y.append(torch.cat(parts, 1))
    if c["op"] == "glu":
        g, u = y
        sg = torch.sigmoid(g)
        a = B1 * torch.tanh(g / B1) * sg * B2 * torch.tanh(u / B2) if c["act"] == SITU else g * sg * u
        if c["out"] == "mxfp8":
            q, qs = _exact_mxfp8(a)
            return {"q": q, "qs": qs}
        return {"out": a}
    return {"out": s["out"].double() + y[0] if c["out"] == "add" else y[0]}

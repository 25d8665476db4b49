"""Plain 64-bit statements of attention and what stands around it (not collected
by pytest), with bounds on what the library's arithmetic may be off by. Nothing
here shares code with the library."""
import math

import numpy as np

from dense_ref import e4m3_rne, pow2, E4M3

U32, U16 = 2.0 ** -24, 2.0 ** -8      # half a step of fp32 and of bf16, relative


def bf16(v):
    """bf16 bits of fp64 values (nearest, ties to even; NaN to a NaN)."""
    f = np.asarray(v, np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(f), np.uint16(0x7fc0), r)


def unbf16(b):
    return (np.asarray(b).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def attend(q, k, v, see, scale):
    """One head: (out, lse, bound of out, bound of lse) for queries q [n][D], keys k [N][D], values v [N][Dv] and
    see [n][N].

    Scores are sums of D exact products in fp32, each rounding at most 2^-24 of the magnitude sum, then scaled
    (two roundings); a score that is off by d turns its weight by a factor e^d, numerator and denominator, and the
    exponent's own arithmetic adds 2^-22 and what fp32 holds of |s| log2(e) (the maximum's product is another such
    number). Weights are rounded to bf16 (2^-8) and summed in fp32 (2^-24 each time); so is their product with v. The
    result is rounded to bf16 once."""
    n, N = see.shape
    dv = v.shape[1]
    out, lse = np.zeros((n, dv)), np.full(n, -math.inf)
    tol, ltol = np.zeros((n, dv)), np.zeros(n)
    for i in range(n):
        at = np.nonzero(see[i])[0]
        if not len(at):
            continue
        s = scale * (k[at] @ q[i])
        mag = scale * (np.abs(k[at]) @ np.abs(q[i]))
        ds = ((q.shape[1] + 4) * U32 * mag + 4 * U32 * np.abs(s)).max() + 4 * U32 * np.abs(s).max() + 2.0 ** -22
        m = s.max()
        p = np.exp(s - m)
        l = p.sum()
        out[i] = (p @ v[at]) / l
        lse[i] = m + math.log(l)
        a = (p @ np.abs(v[at])) / l
        steps = (len(at) + 80) * U32
        tol[i] = a * (U16 + 2 * ds + 2 * steps) + U16 * (np.abs(out[i]) + a * (U16 + 2 * ds + 2 * steps)) + 2.0 ** -133
        ltol[i] = ds + steps + 4 * U32 * (abs(lse[i]) + abs(m)) + 4 * U32
    return out, lse, tol, ltol


def check_rows(got, lse, want, want_lse, tol, ltol, what):
    """bf16 results and fp32 lse (or None) against attend's."""
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{what}: out off by {np.nanmax(err)} where {tol.flat[np.nanargmax(err - tol)]} is allowed"
    if lse is not None:
        empty = np.isneginf(want_lse)
        assert (np.isneginf(lse) == empty).all(), f"{what}: lse of empty rows"
        bad = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, want_lse)) > ltol
        assert not bad.any(), f"{what}: lse off"


def heads(x, gamma, eps, pos, freq, pairs):
    """(y, bound of fp32 arithmetic) of heads x [T][H][D]: norm, then rotation of the first 2 len(freq) dimensions.

    fp32: squares of bf16 are exact, D / 2 additions deep at most, then a quotient, a root, an inverse and two products:
    n is off by (D / 4 + 8) 2^-24 relative (the root halves the sum's). The angle is 64-bit but for its reduced
    fraction of a turn: 2^-26 of a turn, 2 pi 2^-26 < 2^-23, and 2^-53 of up to 2^31 / (2 pi) turns twice; sine and
    cosine are within 4 ulp (2^-22); two products and a sum follow (3 * 2^-24)."""
    x = x.astype(np.float64)
    D = x.shape[-1]
    rel = 0.0
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
        rel = (D / 4 + 8) * U32
    y, tol = x.copy(), rel * np.abs(x)
    half = len(freq)
    turn = 2.0 ** -23 + 2.0 ** -22 + 2 * math.pi * 2 * 2.0 ** -53 * (np.abs(pos).max() if len(pos) else 0) + 3 * U32
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        ang = pos.astype(np.float64) * float(freq[i])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        t = (np.abs(x[..., a]) + np.abs(x[..., b])) * (rel + turn)
        tol[..., a] = tol[..., b] = t
    return y, tol


def check_mxfp8(codes, bytes_, y, tol, what):
    """e4m3 codes [..][D] and E8M0 bytes [..][D / 32] of values y known to within tol."""
    v = y.reshape(-1, 32)
    t = tol.reshape(-1, 32)
    q, s = codes.reshape(-1, 32), bytes_.reshape(-1)
    lo, hi = np.maximum(np.abs(v) - t, 0).max(1), (np.abs(v) + t).max(1)
    scale = np.exp2(s.astype(np.float64) - 127)
    assert (lo <= 448 * scale).all(), f"{what}: scale too small"
    assert ((hi > 224 * scale) | (s == 0)).all(), f"{what}: scale not the smallest"
    got = E4M3[q] * scale[:, None]
    # nearest e4m3: half a step, 2^-4 relative, 2^-10 of the scale among the smallest
    err = np.abs(got - v)
    assert (err <= np.maximum(2.0 ** -4 * (np.abs(v) + t), 2.0 ** -10 * scale[:, None]) + t).all(), f"{what}: values"


def mxfp8_pool(v):
    """(codes, bytes) of fp64 values [..][D] as an MXFP8 cache holds them."""
    f = np.asarray(v, np.float64).reshape(-1, 32)
    m = np.abs(f).max(1)
    s = np.full(len(f), -127)
    while (m > 448 * np.exp2(s.astype(float))).any():
        s = s + (m > 448 * np.exp2(s.astype(float)))
    q = e4m3_rne(f / np.exp2(s.astype(float))[:, None])
    return q.reshape(v.shape), (s + 127).astype(np.uint8).reshape(*v.shape[:-1], v.shape[-1] // 32)


def mxfp8_values(q, s):
    return E4M3[q] * np.repeat(pow2(s), 32, -1)


def logprobs(x, ids, k):
    """(lp, entropy, top ids, top lp, bound of lp, bound of entropy) of one row in 64 bits.

    e^(x - m): the difference is rounded (2^-24 of it), the exponential within 2^-22; a thread sums at most 64 of them in
    fp32 (2^-24 each). What is not the maximum is so off by 2^-17 of itself, and 2^-23 of sum |x - m| e^(x - m). A term is
    an fp32 number: one below 2^-126 (x - m below -87.3) counts as 0, in the entropy with its |x - m| < 2^8 for every
    such term that 64 bits tell from 0 beside 2^-126."""
    x = x.astype(np.float64)
    m = x.max()
    with np.errstate(invalid="ignore"):
        d = x - m
        e = np.exp(d)
        dev = np.where(e > 0, -d * e, 0.0).sum()
    s, peak = e.sum(), (x == m).sum()
    lp = d - math.log(s) if s - peak > 1e-3 else d - math.log1p((peak - 1) + e[x != m].sum())
    ent = math.log(s) + dev / s if s - peak > 1e-3 else math.log1p((peak - 1) + e[x != m].sum()) + dev / s
    off = (2.0 ** -17 * (s - peak) + 2.0 ** -23 * dev + len(x) * 2.0 ** -126) / s
    big = np.where(e > 0, d, 0.0) ** 2 @ e + len(x) * 2.0 ** (8 + 23 - 126)
    order = np.lexsort((np.arange(len(x)), -x))[:k]
    at = np.array([lp[i] if 0 <= i < len(x) else np.nan for i in ids])
    return (at, ent, order, lp[order], off,
            off * (1 + dev / s) + (2.0 ** -17 * dev + 2.0 ** -23 * big) / s + U32 * abs(ent) + 2.0 ** -149)

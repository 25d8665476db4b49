"""Plain 64-bit statements of the dense operators (not collected by pytest):
the MXFP4 and MXFP8 formats written out by their definitions, the norm, and
the products. Nothing here shares code with the library."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = math.nan if (e == 15 and m == 7) else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = -v if s else v
    return t


E4M3 = _e4m3_table()


def pow2(byte):
    """2^(byte - 127), 0 for 255."""
    b = np.asarray(byte).astype(np.int64)
    return np.where(b == 255, 0.0, np.exp2((b - 127).astype(np.float64)))


def dense(packed, scales):
    """An MXFP4 matrix [N][K] in 64 bits."""
    codes = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    return E2M1[codes] * np.repeat(pow2(scales), 32, 1)


def tokens8(q, s):
    """MXFP8 tokens [T][W] in 64 bits."""
    return E4M3[q] * np.repeat(pow2(s), 32, 1)[:, :q.shape[1]]


def e4m3_rne(v):
    """e4m3 codes of values within +-448, nearest, ties to the even code;
    NaN for what is not finite. By comparison with every code."""
    v = np.asarray(v, np.float64)
    pos = E4M3[:127]                       # 0 .. 448, ascending
    a = np.abs(v)
    a0 = np.where(np.isfinite(a), a, 0.0)
    hi = np.clip(np.searchsorted(pos, a0), 1, 126)
    dl, dh = a0 - pos[hi - 1], pos[hi] - a0
    c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1)
    c = np.where(np.signbit(v), c | 128, c)
    return np.where(np.isfinite(v), c, 127).astype(np.uint8)


def mxfp8(v):
    """(codes, bytes) of fp32 rows: per 32 values the smallest s >= -127 with
    the largest finite magnitude <= 448 * 2^s."""
    T, W = v.shape
    G = -(-W // 32)
    q, sb = np.empty((T, W), np.uint8), np.empty((T, G), np.uint8)
    for j in range(G):
        b = v[:, 32 * j:32 * j + 32].astype(np.float64)
        a = np.where(np.isfinite(b), np.abs(b), 0.0).max(1)
        s = np.full(T, -127)
        while True:
            low = a > 448.0 * np.exp2(s.astype(np.float64))
            if not low.any():
                break
            s = s + low
        q[:, 32 * j:32 * j + 32] = e4m3_rne(b / np.exp2(s.astype(np.float64))[:, None])
        sb[:, j] = s + 127
    return q, sb


def inv_rms(h, eps):
    """fp32(1 / sqrt(mean h^2 + eps)) per row, and whether no order of a 64-bit
    sum can round it otherwise: H terms of one sign, each exact or rounded
    once, sum to within H 2^-53 in any order (the root halves that), and the
    quotient, the sum with eps, the root and the inverse add less than 8 2^-53."""
    tol = (h.shape[1] + 8) * 2.0 ** -53
    out, sure = np.empty(h.shape[0], np.float32), np.zeros(h.shape[0], bool)
    for t, row in enumerate(h):
        y = 1.0 / math.sqrt(math.fsum(float(a) * float(a) for a in row.astype(np.float64)) / h.shape[1]
                            + float(np.float32(eps)))
        f = np.float32(y)
        mids = [(float(f) + float(np.nextafter(f, np.float32(w)))) / 2 for w in (0.0, np.inf)]
        out[t], sure[t] = f, all(abs(y - m) > tol * y for m in mids)
    return out, sure


def add_norm(h, d, gamma, eps):
    """(h', v fp32, rows that are sure) of fp32 h, d (or None), gamma."""
    h2 = h if d is None else h + d.astype(np.float32)
    inv, sure = inv_rms(h2, eps)
    with np.errstate(invalid="ignore"):
        return h2, (h2 * inv[:, None]).astype(np.float32) * gamma[None, :], sure


def act(g, u, kind, b1=4.0, b2=25.0):
    sg = 1.0 / (1.0 + np.exp(-g))
    return b1 * np.tanh(g / b1) * sg * (b2 * np.tanh(u / b2)) if kind == 1 else g * sg * u

"""GPU tests of what the dense operators make of values and sizes that ordinary
inputs do not have: products of very different sizes in one run of the sum,
infinite tokens, tokens below bf16's range, more rows than a grid has blocks.
Against the 64-bit statements of ``dense_ref``; what is exact is compared bit
for bit."""
import numpy as np
import pytest
import torch

import dense_ref as R
import mxfp4_routed_expert_sigmoid_amd as k3
from gpu_helpers import bf16_rne_np
from test_gpu_dense import ACT_TOL, DEV, _f8, _glu_scaled, _linear, _need, _result, _t

pytestmark = pytest.mark.gpu


def _pack(codes):
    """fp4 codes [N][K] -> packed bytes [N][K / 2]."""
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def _tokens(v, x8):
    """(device tokens, device bytes, values in 64 bits) of values that both types hold (bytes 127)."""
    if x8:
        q = R.e4m3_rne(v)
        s = np.full((v.shape[0], v.shape[1] // 32), 127, np.uint8)
        assert np.array_equal(R.tokens8(q, s), v)
        return _t(q), _t(s), v
    x = _t(v.astype(np.float32)).to(torch.bfloat16)
    assert np.array_equal(x.double().cpu().numpy(), v)
    return x, None, v


# --- products of very different sizes ---------------------------------------
# Every row has up to seven pairs of products 2^10 and -2^10 within runs of 8
# columns, and else products that are multiples of 2^-10 below 2^-3.5: what is
# left of a row is 2^20 times finer than its largest products. Every partial sum, in any
# order, is a multiple of 2^-10 below 7 * 2^10 + 18432 * 2^-3.5 < 2^14, so fp32 sums
# are exact and a sum that keeps fewer bits below its largest product is not.
def _spread(N, K, r, down=0):
    """Weights of a matrix of such rows (scale bytes `down` below 127)."""
    codes = r.integers(0, 16, (N, K))
    big = _big_columns(K)
    sign = r.integers(0, 2, (N, len(big) // 2)) * 8
    codes[:, big[0::2]] = 6 + sign            # +-4
    codes[:, big[1::2]] = 6 + (8 - sign)      # its negative
    return _pack(codes), np.full((N, K // 32), 127 - down, np.uint8)


def _big_columns(K):
    """Pairs of columns within one run of 8 columns of seven blocks (or of all, if fewer)."""
    blocks = np.unique(np.linspace(0, K // 32 - 1, 7).astype(int))
    return np.array([32 * b + o for b in blocks for o in (3, 6)])


def _spread_tokens(T, K, x8, r):
    v = r.integers(-7, 8, (T, K)) * 2.0 ** -9
    v[:, _big_columns(K)] = 256.0
    return _tokens(v, x8)


SPREAD = [(1, 33, 7168), (2, 65, 18432), (3, 65, 18432), (4, 65, 8192), (4, 65, 8224), (1, 33, 32768), (1, 33, 32800),
          (5, 65, 2080), (33, 4137, 1184), (48, 257, 7168), (64, 100, 640), (130, 20001, 160), (300, 4137, 1056)]


@pytest.mark.parametrize("T,N,K", SPREAD)
@pytest.mark.parametrize("x8", [False, True])
def test_linear_sums_keep_32_bits(T, N, K, x8):
    _need()
    r = np.random.default_rng([T, N, K])
    p, s = _spread(N, K, r)
    x, xs, xv = _spread_tokens(T, K, x8, r)
    y = xv @ R.dense(p, s).T                  # exact in 64 bits too
    for out in ("f32", "bf16", "add", "mxfp8"):
        _, o, _, os_, h = _result(out, T, N, 0, r)
        print(f"[linear] T={T} N={N} K={K} x8={x8} out={out}", flush=True)
        k3.linear(_t(p), _t(s), x, o, xs=xs, outs=os_, accumulate=out == "add")
        if out == "mxfp8":
            q, sw = R.mxfp8(y.astype(np.float32))
            assert np.array_equal(_f8(o), q) and np.array_equal(os_.cpu().numpy(), sw)
        elif out == "bf16":
            assert np.array_equal(o.view(torch.int16).cpu().numpy().view(np.uint16), bf16_rne_np(y.astype(np.float32)))
        else:
            assert np.array_equal(o.double().cpu().numpy(), y if h is None else h + y)


@pytest.mark.parametrize("T,N,K", [(1, 33, 7168), (2, 65, 18432), (4, 65, 8224), (33, 257, 1184), (130, 20001, 160),
                                   (600, 2100, 352)])
@pytest.mark.parametrize("x8", [False, True])
def test_glu_sums_keep_32_bits(T, N, K, x8):
    _need()
    r = np.random.default_rng([T, N, K])
    mats = [_spread(N, K, r) for _ in range(2)]
    x, xs, xv = _spread_tokens(T, K, x8, r)
    want = R.act(*(xv @ R.dense(*m).T for m in mats), k3.ACT_SWIGLU)
    for out in ("f32", "bf16"):
        _, o, _, _, _ = _result(out, T, N, 0, r)
        print(f"[glu] T={T} N={N} K={K} x8={x8} out={out}", flush=True)
        k3.glu(*map(_t, mats[0]), *map(_t, mats[1]), x, o, xs=xs, act=k3.ACT_SWIGLU)
        half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= np.abs(want) * (ACT_TOL + half * (1 + ACT_TOL)))


# --- infinite tokens --------------------------------------------------------
# A token t holds one infinity, in block t mod (K / 32) (so every block has one
# where there are tokens enough; the last token holds it in the last column), at a
# column whose weight is zero in no row: its results are infinities with the sign of
# the weights. In MXFP8 the infinity is 448 * 2^127, beyond bf16's range.
def _infinite(T, N, K, x8, r):
    codes = r.integers(0, 16, (N, K))
    s = np.full((N, K // 32), 127, np.uint8)
    v = r.integers(-15, 16, (T, K)).astype(np.float64)
    at = 32 * (np.arange(T) % (K // 32)) + (7 * np.arange(T) + 31) % 32
    at[-1] = K - 1
    cols = np.unique(at)
    codes[:, cols] = np.where(codes[:, cols] & 7, codes[:, cols], 1)
    neg = r.integers(0, 2, T).astype(bool)
    x, xs, _ = _tokens(v, x8)
    rows = np.arange(T)
    if x8:
        q, sb = x.cpu().numpy(), xs.cpu().numpy()
        for t in range(T):
            b = at[t] // 32
            q[t, 32 * b:32 * b + 32], q[t, at[t]], sb[t, b] = 0, 0xfe if neg[t] else 0x7e, 254
        x, xs = _t(q), _t(sb)
    else:
        x[_t(rows), _t(at)] = _t(np.where(neg, -np.inf, np.inf).astype(np.float32)).to(torch.bfloat16)
    p = _pack(codes)
    w = R.dense(p, s)[:, at].T                # [T][N]: the weights at each token's infinity
    return p, s, x, xs, np.where((w < 0) == neg[:, None], np.inf, -np.inf)


INF = [(1, 40, 32), (1, 40, 160), (4, 40, 96), (3, 40, 1056), (4, 66001, 288), (2, 16500, 2080), (5, 45, 160), (9, 45, 288),
       (40, 40, 160), (33, 45, 1056), (66, 45, 2080), (47, 4137, 1184), (130, 20001, 160), (300, 9001, 1056),
       (129, 16640, 2048)]


@pytest.mark.parametrize("T,N,K", INF)
@pytest.mark.parametrize("x8", [False, True])
def test_linear_of_infinite_tokens(T, N, K, x8):
    _need()
    r = np.random.default_rng([T, N, K])
    p, s, x, xs, want = _infinite(T, N, K, x8, r)
    for out in ("f32", "bf16", "add"):
        _, o, _, _, _ = _result(out, T, N, 0, r)
        print(f"[linear] T={T} N={N} K={K} x8={x8} out={out}", flush=True)
        k3.linear(_t(p), _t(s), x, o, xs=xs, accumulate=out == "add")
        assert np.array_equal(o.double().cpu().numpy(), want)
    _, o, _, os_, _ = _result("mxfp8", T, N, 0, r)
    k3.linear(_t(p), _t(s), x, o, xs=xs, outs=os_)
    assert bool((_t(_f8(o)) & 127 == 127).all()) and bool((os_ == 0).all())


@pytest.mark.parametrize("T,N,K", [(1, 40, 160), (3, 40, 1056), (5, 45, 160), (33, 257, 1184), (130, 20001, 160)])
@pytest.mark.parametrize("x8", [False, True])
def test_glu_of_infinite_tokens(T, N, K, x8):
    # SiTU's arms end at +-b1 and +-b2 and its sigmoid at 0 and 1
    _need()
    r = np.random.default_rng([T, N, K])
    p, s, x, xs, y = _infinite(T, N, K, x8, r)
    out = torch.empty((T, N), device=DEV)
    k3.glu(_t(p), _t(s), _t(p), _t(s), x, out, xs=xs)
    assert np.array_equal(out.double().cpu().numpy(), np.where(y > 0, 100.0, 0.0))


# --- tokens below bf16's range ----------------------------------------------
# e4m3 goes down to 2^-9, so a group of byte 0 to 2 holds multiples of 2^-136, which bf16
# (multiples of 2^-133 at least) does not: such a token value is taken within one
# step 2^-133. From byte 3 on every value is a bf16. The weights are about 2^123.
@pytest.mark.parametrize("T,N,K", [(1, 33, 160), (3, 33, 1056), (7, 45, 160), (40, 45, 1056), (130, 20001, 160)])
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 4])
def test_smallest_tokens(T, N, K, byte):
    _need()
    r = np.random.default_rng([T, N, K, byte])
    p = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = np.full((N, K // 32), 250, np.uint8)
    q = R.e4m3_rne(r.integers(-15, 16, (T, K)) * 2.0 ** -9)
    xs = np.full((T, K // 32), byte, np.uint8)
    out = torch.empty((T, N), device=DEV)
    k3.linear(_t(p), _t(s), _t(q), out, xs=_t(xs))
    got, W, xv = out.double().cpu().numpy(), R.dense(p, s), R.tokens8(q, xs)
    want = xv @ W.T
    if byte >= 3:      # multiples of 2^-133 * 2^122, sums below 2^24 of them
        assert np.array_equal(got, want)
    else:
        assert np.all(np.abs(got - want) <= 2.0 ** -133 * np.abs(W).sum(1))


# --- sizes ------------------------------------------------------------------
# a block per tile and blocks of many tiles, on both sides of the borders between them (1024 to 4096 tiles), one unit
# of columns per wave and more
@pytest.mark.parametrize("T,N,K", [(1, 16368, 256), (2, 16400, 2048), (4, 16385, 1056), (1, 32752, 512), (3, 32785, 288),
                                   (2, 65552, 96)])
@pytest.mark.parametrize("x8", [False, True])
def test_few_tokens_at_the_borders_of_long_matrices(T, N, K, x8):
    for out in ("f32", "mxfp8"):
        _linear(T, N, K, x8, out)
        _glu_scaled(T, N, K, x8, out, 1)


@pytest.mark.parametrize("H,want", [(8, "both"), (9, "mxfp8")])
def test_norm_of_more_rows_than_a_grid_holds(H, want):
    # 2^20 blocks: the last rows are a block's second one. Rows repeat every 1021, so each is compared
    # with the same row of a short call
    _need()
    T, R0 = (1 << 20) + 1500, 1021
    r = np.random.default_rng(H)
    h0, d0, gamma = (_t((4 * r.standard_normal(s)).astype(np.float32)) for s in ((R0, H), (R0, H), (H,)))

    def call(h, d):
        t = h.shape[0]
        x = torch.empty((t, H), dtype=torch.bfloat16, device=DEV) if want == "both" else None
        q = torch.empty((t, H), dtype=torch.uint8, device=DEV)
        qs = torch.empty((t, 1), dtype=torch.uint8, device=DEV)
        k3.add_norm(h, gamma, 1e-5, d=d, x=x, q=q, qs=qs)
        return [h, q, qs] + ([x.view(torch.int16)] if x is not None else [])
    short = call(h0.clone(), d0)
    i = torch.arange(T, device=DEV) % R0
    for a, b in zip(short, call(h0[i], d0[i])):
        assert torch.equal(a[i], b)

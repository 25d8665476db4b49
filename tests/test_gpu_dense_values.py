"""GPU tests of what the dense products make of values that ordinary inputs do
not hold: products of very different sizes in one run of the sum. Against the
64-bit statements of ``dense_ref``; what is exact is compared bit for bit."""
import numpy as np
import pytest
import torch

import dense_ref as R
import mxfp4_routed_expert_sigmoid_amd as k3
from gpu_helpers import bf16_rne_np
from test_gpu_dense import ACT_TOL, DEV, _f8, _need, _result, _t

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

"""GPU tests of the dense operators (k3moe_add_norm, k3moe_linear, k3moe_glu)
against the 64-bit statements of ``dense_ref``.

Tolerances. The norm's outputs are decisions both sides take in fp32 from the
same operations, so they must be equal bit for bit (rows whose inverse root
lies next to an fp32 rounding border are left out; none here does). The
products are tested on inputs whose every partial sum is a multiple of one
power of two below 2^24 times it: any order of fp32 sums gives the exact
result, so fp32 outputs must be equal, bf16 ones the rounding of the exact
value. On random inputs an fp32 sum of K exact products is held to
K 2^-24 sum|w x| (K roundings to nearest of sums no larger than that). The
activation adds its own roundings, see ACT_TOL."""
import numpy as np
import pytest
import torch

import dense_ref as R
import mxfp4_routed_expert_sigmoid_amd as k3
from gpu_helpers import bf16_rne_np

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-5
# a = b1 tanh(g / b1) * sg * b2 tanh(u / b2), sg = 1 / (1 + exp(-g)): two tanh
# and an exp of up to 2 ulp each and eight products, quotients and sums of half
# an ulp: under 16 ulp together
ACT_TOL = 16 * 2.0 ** -23
SENT = 77.0


def _need():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _bits(a):
    """fp32 numpy -> bf16 tensor on the device (exact where the values are)."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(torch.bfloat16)


def _padded(T, W, pad, dtype, fill=None):
    """(whole buffer, view [T][W] of it): pad elements behind every row and two
    rows behind the last, all filled with SENT."""
    buf = torch.full((T + 2, W + pad), SENT, device=DEV).to(dtype)
    v = buf[:T, :W]
    if fill is not None:
        v.copy_(fill)
    return buf, v


def _untouched(buf, T, W):
    f = buf.float()
    return bool((f[T:] == f[T, 0]).all()) and bool((f[:, W:] == f[T, 0]).all()) and float(f[T, 0]) > 70


def _f8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# --- norm -------------------------------------------------------------------
def _norm_case(T, H, dk, want, pad=0, scale=4.0, seed=0, poke=None):
    _need()
    r = np.random.default_rng([T, H, seed])
    h = (r.standard_normal((T, H)) * scale).astype(np.float32)
    gamma = (1.0 + 0.1 * r.standard_normal(H)).astype(np.float32)
    d = None
    if dk == "f32":
        d = r.standard_normal((T, H)).astype(np.float32)
    elif dk == "bf16":
        d = _bits(r.standard_normal((T, H))).float().cpu().numpy()
    if poke:
        poke(h, d)
    hb, hv = _padded(T, H, pad, torch.float32, torch.from_numpy(h))
    dt = None if d is None else _padded(T, H, pad, torch.float32 if dk == "f32" else torch.bfloat16,
                                        torch.from_numpy(d))[1]
    xb, x = _padded(T, H, pad, torch.bfloat16) if want != "mxfp8" else (None, None)
    qb, q = _padded(T, H, pad, torch.float8_e4m3fn) if want != "bf16" else (None, None)
    G = -(-H // 32)
    sb = torch.full((T + 2, G + 3), 201, dtype=torch.uint8, device=DEV) if q is not None else None
    print(f"[norm] T={T} H={H} d={dk} {want} pad={pad}", flush=True)
    k3.add_norm(hv, torch.from_numpy(gamma).to(DEV), EPS, d=dt, x=x, q=q, qs=None if sb is None else sb[:T, :G])
    torch.cuda.synchronize()
    h2, v, sure = R.add_norm(h, d, gamma, EPS)
    return dict(T=T, H=H, G=G, h=h, h2=h2, v=v, sure=sure, hb=hb, hv=hv, xb=xb, x=x, qb=qb, q=q, sb=sb)


def _check_norm(o):
    T, H, G = o["T"], o["H"], o["G"]
    assert np.array_equal(o["hv"].cpu().numpy(), o["h2"], equal_nan=True) and _untouched(o["hb"], T, H)
    assert o["sure"].all()
    if o["x"] is not None:
        assert np.array_equal(o["x"].contiguous().view(torch.int16).cpu().numpy().view(np.uint16), bf16_rne_np(o["v"]))
        assert _untouched(o["xb"], T, H)
    if o["q"] is not None:
        q, s = R.mxfp8(o["v"])
        assert np.array_equal(o["sb"][:T, :G].cpu().numpy(), s)
        assert np.array_equal(_f8(o["q"]), q) and _untouched(o["qb"], T, H)
        assert bool((o["sb"][T:] == 201).all()) and bool((o["sb"][:, G:] == 201).all())


@pytest.mark.parametrize("H", [1, 2, 31, 33, 100, 256, 1000, 1999, 2049, 4096, 7168, 8188, 8192, 8196, 8193, 20000])
@pytest.mark.parametrize("dk", ["none", "bf16", "f32"])
def test_norm_widths(H, dk):
    _check_norm(_norm_case(3, H, dk, "both"))


@pytest.mark.parametrize("T,H,dk,want,pad", [
    (1, 7168, "bf16", "bf16", 0), (1, 7168, "f32", "mxfp8", 0), (5, 7168, "bf16", "mxfp8", 4), (5, 7168, "bf16", "both", 1),
    (4, 1999, "f32", "both", 9), (2, 12000, "bf16", "both", 8), (3, 640, "none", "bf16", 3), (2000, 96, "bf16", "both", 0),
    (301, 2048, "f32", "mxfp8", 32)])
def test_norm_rows_strides_and_outputs(T, H, dk, want, pad):
    _check_norm(_norm_case(T, H, dk, want, pad))


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e15])
def test_norm_small_and_large_streams(scale):
    # 1e-30: eps rules the root, the tokens fall below e4m3's range of one
    # group (byte 0 and values that round to zero); 1e15: squares of 1e30
    _check_norm(_norm_case(4, 512, "none", "both", scale=scale))


def test_norm_of_zeros_and_of_what_is_not_finite():
    def poke(h, d):
        h[0] = 0.0
        h[1, 40:72] = 0.0
        h[2, 5] = np.inf
        h[3, 6] = np.nan
    o = _norm_case(5, 512, "none", "both", poke=poke)
    x, q, s = o["x"].float().cpu().numpy(), R.E4M3[_f8(o["q"])], o["sb"][:5, :16].cpu().numpy()
    assert (x[0] == 0).all() and (q[0] == 0).all() and (s[0] == 0).all()
    assert (x[1, 40:72] == 0).all() and s[1, 1] > 0
    # an infinity makes the inverse root 0: it becomes NaN and the rest 0; a NaN spreads over its row
    assert np.isnan(x[2, 5]) and (np.delete(x[2], 5) == 0).all() and np.isnan(q[2, 5]) and s[2, 0] == 0
    assert np.isnan(x[3]).all() and np.isnan(q[3]).all()
    w, sw = R.mxfp8(o["v"][4:])
    assert np.array_equal(_f8(o["q"])[4:], w) and np.array_equal(s[4:], sw)


def test_norm_is_the_steps_norm():
    # the tokens of k3moe_step for the same stream, bit for bit
    _need()
    import synth
    import synth.device as sd
    spec = synth.LayerSpec(hidden=512, inter=256, n_experts=16, topk=4, shared_inter=0, seed=5)
    layer = sd.make_layer(spec, sd.layer_tensors(spec, 0, DEV))
    T = 9
    h = torch.from_numpy(synth.make_residual(spec, T)).to(DEV)
    gamma = torch.from_numpy(synth.make_post_norm(spec)).to(DEV)
    idx = torch.empty((T, 4), dtype=torch.int32, device=DEV)
    w = torch.empty((T, 4), device=DEV)
    a, b = (torch.empty((T, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k3.add_norm(h, gamma, EPS, x=b)
    layer.step(h, gamma, EPS, idx, w, x_out=a)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# --- products ---------------------------------------------------------------
def _weights(N, K, r, kind):
    p = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if kind == "exact":      # three neighbouring scales, some groups dropped
        s = r.choice(np.array([125, 126, 127, 255], np.uint8), (N, K // 32), p=[.3, .3, .3, .1])
    else:
        mid = 127 - round(np.log2(2.93 * np.sqrt(K)))
        s = r.integers(mid - 2, mid + 2, (N, K // 32)).astype(np.uint8)
    return p, s


def _tok(T, K, x8, r, kind):
    """(device tokens, device bytes or None, values in 64 bits)."""
    if x8:
        if kind == "exact":  # integers to 15 in e4m3, times 1/2, 1 or nothing
            q = R.e4m3_rne(r.integers(-15, 16, (T, K)).astype(np.float64))
            s = r.choice(np.array([126, 127, 255], np.uint8), (T, K // 32), p=[.45, .45, .1])
        else:
            q, s = R.mxfp8(r.standard_normal((T, K)).astype(np.float32))
        return (torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), R.tokens8(q, s))
    v = r.integers(-15, 16, (T, K)).astype(np.float32) if kind == "exact" else r.standard_normal((T, K))
    x = _bits(v)
    return x, None, x.double().cpu().numpy()


def _t(a):
    return torch.from_numpy(a).to(DEV)


def _result(kind, T, N, pad, r):
    """(buffer, out, outs buffer, outs, start values)."""
    if kind == "mxfp8":
        b, o = _padded(T, N, pad, torch.float8_e4m3fn)
        G = -(-N // 32)
        sb = torch.full((T + 2, G + 3), 201, dtype=torch.uint8, device=DEV)
        return b, o, sb, sb[:T, :G], None
    if kind == "add":
        h = (r.integers(-1000, 1000, (T, N)) / 8).astype(np.float32)
        b, o = _padded(T, N, pad, torch.float32, torch.from_numpy(h))
        return b, o, None, None, h
    b, o = _padded(T, N, pad, torch.bfloat16 if kind == "bf16" else torch.float32)
    return b, o, None, None, None


def _mx8_close(q, s, want, tol):
    """Codes and bytes q, s against 64-bit values that the kernel's fp32 value
    is within tol (relative) of: the group's scale is the right one for some
    such value, and each code is off by at most half a step beyond tol."""
    W = want.shape[1]
    sc = np.repeat(R.pow2(s), 32, 1)[:, :W]
    amax = np.stack([np.abs(want[:, 32 * j:32 * j + 32]).max(1) for j in range(s.shape[1])], 1)
    p = R.pow2(s)
    assert np.all(amax * (1 - tol) <= 448 * p) and np.all((amax * (1 + tol) > 224 * p) | (s == 0))
    got = R.E4M3[q] * sc
    half = np.maximum(np.abs(want) * 2.0 ** -4, sc * 2.0 ** -10)
    assert np.all(np.abs(got - want) <= half * (1 + tol) + np.abs(want) * tol)


def _linear(T, N, K, x8, out, kind="exact", pad=0, xpad=0, seed=0):
    _need()
    r = np.random.default_rng([T, N, K, x8, seed])
    p, s = _weights(N, K, r, kind)
    x, xs, xv = _tok(T, K, x8, r, kind)
    if xpad:
        x = torch.nn.functional.pad(x, (0, xpad), value=5)[:, :K]
        xs = None if xs is None else torch.nn.functional.pad(xs, (0, 5), value=130)[:, :K // 32]
    b, o, sb, os_, h = _result(out, T, N, pad, r)
    print(f"[linear] T={T} N={N} K={K} x8={x8} out={out} {kind} pad={pad}", flush=True)
    k3.linear(_t(p), _t(s), x, o, xs=xs, outs=os_, accumulate=out == "add")
    torch.cuda.synchronize()
    W = R.dense(p, s)
    want = xv @ W.T if h is None else h + xv @ W.T
    assert _untouched(b, T, N)
    if out == "mxfp8":
        q, sw = R.mxfp8(want.astype(np.float32))
        assert np.array_equal(_f8(o), q) and np.array_equal(os_.cpu().numpy(), sw)
        assert bool((sb[T:] == 201).all()) and bool((sb[:, -3:] == 201).all())
        return
    got = o.double().cpu().numpy()
    if kind == "random":
        half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
        mag = np.abs(xv) @ np.abs(W).T * (K * 2.0 ** -24)
        assert np.all(np.abs(got - want) <= mag * (1 + half) + half * np.abs(want))
    elif out == "bf16":
        assert np.array_equal(o.contiguous().view(torch.int16).cpu().numpy().view(np.uint16),
                              bf16_rne_np(want.astype(np.float32)))
    else:
        assert np.array_equal(got, want)


SHAPES = [(1, 1, 32), (1, 33, 64), (2, 31, 96), (3, 40, 2080), (1, 1000, 7168), (4, 130, 7168), (7, 64, 4128),
          (16, 48, 512), (17, 65, 160), (33, 128, 1056), (48, 257, 1536), (64, 100, 640), (65, 96, 352),
          (130, 257, 224), (129, 384, 1024), (300, 300, 1056), (1, 96, 18432), (257, 130, 2048)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("x8", [False, True])
def test_linear_sizes(T, N, K, x8):
    for out in ("f32", "bf16", "add", "mxfp8"):
        _linear(T, N, K, x8, out)


# wide matrices: many row tiles per block for a few tokens (from 65521 rows, and
# from 16385 to MXFP8), the tile kernel for batches (ragged in every direction)
@pytest.mark.parametrize("T,N,K,out", [
    (1, 65521, 96, "f32"), (4, 66001, 288, "bf16"), (2, 70000, 1056, "add"), (3, 16500, 160, "mxfp8"),
    (130, 20001, 160, "f32"), (257, 9000, 352, "bf16"), (300, 9001, 1056, "add"), (1000, 4129, 640, "mxfp8"),
    (129, 16640, 2048, "bf16"), (70, 33000, 128, "f32"), (2100, 2090, 416, "f32"), (385, 16001, 96, "bf16")])
@pytest.mark.parametrize("x8", [False, True])
def test_linear_wide(T, N, K, out, x8):
    _linear(T, N, K, x8, out, pad=3 if N % 2 else 0)


@pytest.mark.parametrize("T,N,K", [(1, 66000, 96), (4, 16500, 288), (130, 20001, 160), (600, 5000, 352)])
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("out", ["bf16", "mxfp8"])
def test_glu_wide(T, N, K, x8, out):
    _glu_scaled(T, N, K, x8, out, 1)


# every number of 16-token tiles, every last phase and scale run of the streaming kernel
@pytest.mark.parametrize("T", [5, 16, 17, 32, 33, 48, 49, 64, 66])
@pytest.mark.parametrize("K", [32, 96, 128, 1024, 1152, 4128, 16416, 18432])
@pytest.mark.parametrize("x8", [False, True])
def test_linear_streamed(T, K, x8):
    for out in ("f32", "bf16"):
        _linear(T, 45, K, x8, out)


# 130 row blocks: two to four 16-token tiles per block, one phase to a second run of scales, a last block of 9 rows
@pytest.mark.parametrize("T", [32, 47, 61])
@pytest.mark.parametrize("K", [96, 1184, 8736])
@pytest.mark.parametrize("x8", [False, True])
def test_linear_streamed_in_wide_token_blocks(T, K, x8):
    for out in ("f32", "bf16"):
        _linear(T, 4137, K, x8, out, pad=3, xpad=16)


@pytest.mark.parametrize("T", [32, 47, 61])
@pytest.mark.parametrize("K", [96, 1184])
@pytest.mark.parametrize("x8", [False, True])
def test_glu_streamed_in_wide_token_blocks(T, K, x8):
    for out in ("mxfp8", "bf16"):
        _glu_scaled(T, 4137, K, x8, out, 1)


@pytest.mark.parametrize("T,N,K", [(1, 100, 7168), (5, 130, 2080), (48, 257, 1536), (300, 160, 1056), (2048, 256, 512)])
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_random_values(T, N, K, x8, out):
    _linear(T, N, K, x8, out, kind="random")


@pytest.mark.parametrize("T,N,K,pad,xpad", [(1, 40, 96, 3, 16), (5, 41, 256, 1, 16), (40, 96, 512, 7, 32),
                                            (200, 130, 288, 5, 48)])
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16", "add", "mxfp8"])
def test_linear_strides(T, N, K, pad, xpad, x8, out):
    _linear(T, N, K, x8, out, pad=pad, xpad=xpad)


@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 515, 7168), (2, 33, 96), (16, 64, 2080), (33, 96, 512), (65, 40, 640),
                                   (130, 257, 224), (300, 130, 1056)])
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("act", [1, 2])
def test_glu_sizes(T, N, K, x8, act):
    # the activation wants moderate gates: the exact weights, scaled down by a power of two
    for out in ("f32", "bf16", "mxfp8"):
        _glu_scaled(T, N, K, x8, out, act)


def _glu_scaled(T, N, K, x8, out, act, pad=0):
    _need()
    r = np.random.default_rng([T, N, K, x8, act])
    down = 3 + round(np.log2(np.sqrt(K)))     # sums of about 1
    mats = []
    for _ in range(2):
        p, s = _weights(N, K, r, "exact")
        mats.append((p, np.where(s == 255, s, s - down).astype(np.uint8)))
    x, xs, xv = _tok(T, K, x8, r, "exact")
    b, o, sb, os_, _ = _result(out, T, N, pad, r)
    print(f"[glu] T={T} N={N} K={K} x8={x8} out={out} act={act}", flush=True)
    k3.glu(*map(_t, mats[0]), *map(_t, mats[1]), x, o, xs=xs, outs=os_, act=act)
    torch.cuda.synchronize()
    g, u = (xv @ R.dense(*m).T for m in mats)
    want = R.act(g, u, act)
    assert _untouched(b, T, N)
    if out == "mxfp8":
        _mx8_close(_f8(o), os_.cpu().numpy(), want, ACT_TOL)
        assert bool((sb[T:] == 201).all()) and bool((sb[:, -3:] == 201).all())
    else:
        half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
        got = o.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= np.abs(want) * (ACT_TOL + half * (1 + ACT_TOL)))


def test_glu_strided_rows_are_left_alone():
    _glu_scaled(5, 41, 96, False, "mxfp8", 1, pad=7)
    _glu_scaled(140, 41, 96, True, "bf16", 2, pad=3)


@pytest.mark.parametrize("T", [1, 9, 150])
@pytest.mark.parametrize("x8", [False, True])
def test_extreme_scales_and_values(T, x8):
    # byte 0 (2^-127) and large bytes, the values chosen so that results stay in range
    _need()
    N, K = 40, 160
    r = np.random.default_rng(T)
    p = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = np.full((N, K // 32), 0, np.uint8)
    s[:, 1] = 255
    if x8:
        q = R.e4m3_rne(r.integers(-15, 16, (T, K)).astype(np.float64))
        xsb = np.full((T, K // 32), 200, np.uint8)
        xsb[:, 2] = 255
        x, xs, xv = _t(q), _t(xsb), R.tokens8(q, xsb)
    else:
        x = _bits(r.integers(-15, 16, (T, K)) * 2.0 ** 73)
        xs, xv = None, x.double().cpu().numpy()
    out = torch.empty((T, N), device=DEV)
    k3.linear(_t(p), _t(s), x, out, xs=xs)
    assert np.array_equal(out.double().cpu().numpy(), xv @ R.dense(p, s).T)


@pytest.mark.parametrize("T", [3, 40, 200])
@pytest.mark.parametrize("x8", [False, True])
def test_a_token_that_is_not_finite_stays_alone(T, x8):
    _need()
    N, K = 40, 160
    r = np.random.default_rng(T)
    p, s = _weights(N, K, r, "exact")
    x, xs, xv = _tok(T, K, x8, r, "exact")
    bad = T // 2
    if x8:
        xs[bad] = 127
        x[bad, K - 1] = 127           # the NaN code
    else:
        x[bad, K - 1] = float("nan")
    p[:, -1] |= 0x10                  # its weight is not zero
    s[:, -1] = 127
    out = torch.empty((T, N), device=DEV)
    k3.linear(_t(p), _t(s), x, out, xs=xs)
    got = out.double().cpu().numpy()
    assert np.isnan(got[bad]).all()
    keep = np.arange(T) != bad
    assert np.array_equal(got[keep], (xv @ R.dense(p, s).T)[keep])


@pytest.mark.parametrize("T", [2, 6, 20, 200])
@pytest.mark.parametrize("K", [96, 1056, 2080])
def test_what_lies_behind_a_row_is_not_used(T, K):
    # scale bytes behind a row's last block (the next token's first, or padding) are far out of the row's
    # range: read by the kernels in wide loads, they must not reach a result
    _need()
    N = 40
    r = np.random.default_rng([T, K])
    p, s = _weights(N, K, r, "exact")
    q = R.e4m3_rne(r.integers(-15, 16, (T, K)).astype(np.float64))
    q[:, K - 32:] |= 0x78                            # large last blocks: not zeros
    q[:, K - 32:] &= 0xfd
    q[:, :32] = R.e4m3_rne(r.integers(-1, 2, (T, 32)).astype(np.float64))   # (15 * 2^127 would be infinite)
    xsb = np.full((T, K // 32), 127, np.uint8)
    xsb[:, 0] = 254                                  # every row's first block 2^127, its weights dropped
    s[:, 0] = 255
    wide = np.full((T, K // 32 + 16), 254, np.uint8)
    wide[:, :K // 32] = xsb
    want = R.tokens8(q[:, 32:], xsb[:, 1:]) @ R.dense(p, s)[:, 32:].T
    for xs in (_t(xsb), _t(wide)[:, :K // 32]):
        out = torch.empty((T, N), device=DEV)
        k3.linear(_t(p), _t(s), _t(q), out, xs=xs)
        got = out.double().cpu().numpy()
        assert np.array_equal(got, want)


def test_no_tokens():
    _need()
    p, s = (torch.zeros((8, w), dtype=torch.uint8, device=DEV) for w in (16, 1))
    e = lambda w, t: torch.empty((0, w), dtype=t, device=DEV)
    k3.linear(p, s, e(32, torch.bfloat16), e(8, torch.float32))
    k3.glu(p, s, p, s, e(32, torch.bfloat16), e(8, torch.float32))
    k3.add_norm(e(32, torch.float32), torch.ones(32, device=DEV), EPS, x=e(32, torch.bfloat16))


# --- together ---------------------------------------------------------------
def _mlp(T, H, I, x8, r):
    """A dense MLP's tensors: gate, up, down, gamma."""
    mats = []
    for n, k in ((I, H), (I, H), (H, I)):
        p, s = _weights(n, k, r, "random")
        mats.append((p, s))
    gamma = (1 + 0.1 * r.standard_normal(H)).astype(np.float32)
    h = (4 * r.standard_normal((T, H))).astype(np.float32)
    d = r.standard_normal((T, H)).astype(np.float32)
    return mats, gamma, h, d


class _Run:
    """One decoder layer's dense MLP on the stream: h += d, norm, glu, h += W2 a."""

    def __init__(self, T, H, I, x8, mats, gamma):
        self.w = [(_t(p), _t(s)) for p, s in mats]
        self.gamma = _t(gamma)
        e8, s8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
        mk = lambda w, t: torch.empty((T, w), dtype=t, device=DEV)
        self.x8 = x8
        if x8:
            self.x, self.xs, self.a, self.as_ = mk(H, e8), mk(H // 32, s8), mk(I, e8), mk(I // 32, s8)
        else:
            self.x, self.xs, self.a, self.as_ = mk(H, torch.bfloat16), None, mk(I, torch.bfloat16), None

    def __call__(self, h, d, stream=None):
        if self.x8:
            k3.add_norm(h, self.gamma, EPS, d=d, q=self.x, qs=self.xs, stream=stream)
        else:
            k3.add_norm(h, self.gamma, EPS, d=d, x=self.x, stream=stream)
        k3.glu(*self.w[0], *self.w[1], self.x, self.a, xs=self.xs, outs=self.as_, stream=stream)
        k3.linear(*self.w[2], self.a, h, xs=self.as_, accumulate=True, stream=stream)


@pytest.mark.parametrize("T", [1, 6, 70, 260])
@pytest.mark.parametrize("x8", [False, True])
def test_dense_mlp_step(T, x8):
    # each stage against 64 bits on the stage's own input, so that the
    # tolerances are those of one stage
    _need()
    H, I = 512, 1536
    r = np.random.default_rng([T, x8])
    mats, gamma, h0, d0 = _mlp(T, H, I, x8, r)
    run = _Run(T, H, I, x8, mats, gamma)
    h, d = _t(h0.copy()), _t(d0)
    run(h, d)
    torch.cuda.synchronize()
    h2, v, sure = R.add_norm(h0, d0, gamma, EPS)
    assert sure.all()
    if x8:
        q, s = R.mxfp8(v)
        assert np.array_equal(_f8(run.x), q) and np.array_equal(_f8(run.xs), s)
        xv = R.tokens8(q, s)
    else:
        assert np.array_equal(run.x.view(torch.int16).cpu().numpy().view(np.uint16), bf16_rne_np(v))
        xv = run.x.double().cpu().numpy()
    W1, W3, W2 = (R.dense(*m) for m in mats)
    g, u = xv @ W1.T, xv @ W3.T
    want = R.act(g, u, 1)
    # what the sums' errors can move the activation: |da/dg| <= 1.1 * 25 (|a / sg| + |a|), |da/du| <= 4
    K = H
    eg, eu = (np.abs(xv) @ np.abs(W).T * (K * 2.0 ** -24) for W in (W1, W3))
    err = eg * 1.1 * np.minimum(np.abs(u), 25.0) + eu * np.minimum(np.abs(g), 4.0) + np.abs(want) * ACT_TOL + eg * eu
    av = R.tokens8(_f8(run.a), _f8(run.as_)) if x8 else run.a.double().cpu().numpy()
    step = np.repeat(R.pow2(_f8(run.as_)), 32, 1) * 2.0 ** -10 if x8 else 0.0
    half = np.maximum((2.0 ** -4 if x8 else 2.0 ** -8) * (np.abs(want) + err), step)
    assert np.all(np.abs(av - want) <= half + err)
    y = av @ W2.T
    mag = np.abs(av) @ np.abs(W2).T * (I * 2.0 ** -24)
    assert np.all(np.abs(h.double().cpu().numpy() - (h2 + y)) <= mag * (1 + 2.0 ** -24) + 2.0 ** -24 * np.abs(h2 + y))


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("x8", [False, True])
def test_captured_and_replayed(T, x8):
    _need()
    H, I = 512, 640
    r = np.random.default_rng([T, 3])
    mats, gamma, h0, d0 = _mlp(T, H, I, x8, r)
    run = _Run(T, H, I, x8, mats, gamma)
    h, d = _t(h0.copy()), _t(d0)
    run(h, d)                                   # loads the kernels before the capture
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        run(h, d)
    ref = _Run(T, H, I, x8, mats, gamma)
    want, other = _t(h0.copy()), _t(h0.copy())
    h.copy_(want)
    for i in range(4):
        d.copy_(_t(d0 * (i + 1)))
        gr.replay()
        torch.cuda.synchronize()
        ref(want, _t(d0 * (i + 1)))             # eager work between the replays
        ref(other, d)
        torch.cuda.synchronize()
        assert torch.equal(h, want), i


@pytest.mark.parametrize("T", [1, 40, 200])
def test_two_streams_at_once(T):
    _need()
    H, I = 512, 640
    r = np.random.default_rng([T, 4])
    jobs = []
    for j in range(2):
        mats, gamma, h0, d0 = _mlp(T, H, I, j, r)
        jobs.append((_Run(T, H, I, bool(j), mats, gamma), _t(h0), _t(d0)))
    want = []
    for run, h, d in jobs:
        w = h.clone()
        for _ in range(3):
            run(w, d)
        want.append(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        for (run, h, d), s in zip(jobs, streams):
            run(h, d, stream=s)                 # another stream than the current one
    torch.cuda.synchronize()
    for (run, h, d), w in zip(jobs, want):
        assert torch.equal(h, w)


def test_same_call_gives_the_same_bits():
    _need()
    r = np.random.default_rng(9)
    for T in (1, 5, 70, 300):
        p, s = _weights(200, 2080, r, "random")
        x, xs, _ = _tok(T, 2080, True, r, "random")
        outs = []
        for _ in range(3):
            o = torch.empty((T, 200), device=DEV)
            k3.linear(_t(p), _t(s), x, o, xs=xs)
            outs.append(o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_rows_beyond_four_gib():
    # the last rows of a matrix, of the tokens and of the result lie past 2^32 bytes
    _need()
    K, N = 65536, 131104                        # packed: 4.3 GB
    p = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    p[N - 3:] = 0x22                            # ones
    x = torch.ones((1, K), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((1, N), device=DEV)
    k3.linear(p, s, x, out)
    torch.cuda.synchronize()
    assert bool((out[0, N - 3:] == K).all()) and bool((out[0, :N - 3] == 0).all())
    del p, s, x, out
    T, N, K = 70000, 31000, 32                  # out: 8.7 GB
    r = np.random.default_rng(3)
    pw, sw = _weights(N, K, r, "exact")
    x, _, _ = _tok(T, K, False, r, "exact")
    out = torch.empty((T, N), device=DEV)
    k3.linear(_t(pw), _t(sw), x, out)
    torch.cuda.synchronize()
    W = R.dense(pw, sw)
    for t in (0, 34636, 69999):
        assert np.array_equal(out[t].double().cpu().numpy(), x[t].double().cpu().numpy() @ W.T)

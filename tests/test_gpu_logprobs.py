"""k3moe_logprobs against log softmax in 64 bits: sizes, types, strides, ties,
banned tokens, rows that are no distribution."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda:0"


def _run(x, ids=None, k=0, ent=True, ws=None, stream=None):
    T = x.shape[0]
    i = lp = ti = tl = None
    if ids is not None:
        i = torch.tensor(ids, dtype=torch.int32, device=DEV).view(T, -1)
        lp = torch.full(i.shape, 5.0, device=DEV)
    if k:
        ti, tl = torch.full((T, k), -5, dtype=torch.int32, device=DEV), torch.full((T, k), 5.0, device=DEV)
    e = torch.full((T,), 5.0, device=DEV) if ent else None
    k3.logprobs(x, ids=i, lp=lp, entropy=e, top_ids=ti, top_lp=tl, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (lp, e, ti, tl)]


def _check(x, ids, k):
    lp, e, ti, tl = _run(x, ids, k)
    xn = x.float().cpu().numpy()
    for t in range(len(xn)):
        a, ent, order, top, tol, etol = ref.logprobs(xn[t], ids[t], k)
        got = lp[t].astype(float)
        assert np.array_equal(np.isnan(got), np.isnan(a)) and np.array_equal(np.isneginf(got), np.isneginf(a))
        fin = np.isfinite(a)
        got, a = got[fin], a[fin]
        assert (np.abs(got - a) <= tol + ref.U32 * np.abs(a)).all(), (t, got - a, tol)
        assert abs(float(e[t]) - ent) <= etol, (t, e[t], ent, etol)
        if k:
            assert np.array_equal(ti[t], order), (t, ti[t], order)
            fin = np.isfinite(top)
            assert np.array_equal(np.isneginf(tl[t]), np.isneginf(top))
            assert (np.abs(tl[t].astype(float)[fin] - top[fin]) <= tol + ref.U32 * np.abs(top[fin])).all()


def _x(T, V, dtype=torch.float32, pad=0, off=0, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    buf = torch.zeros(T * (V + pad) + off, dtype=dtype, device=DEV)
    x = buf[off:].view(T, V + pad)[:, :V]
    x.copy_(spread * torch.randn((T, V), generator=g))
    return x


def _ids(T, V, M=3, seed=0):
    return np.random.default_rng(seed).integers(0, V, (T, M)).tolist()


@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 257, 4095, 4096, 4097, 16385, 50001, 163840])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabularies(V, dtype):
    _check(_x(3, V, dtype), _ids(3, V), min(V, 8))


@pytest.mark.parametrize("T,V", [(600, 1000), (700, 16000), (530, 17001), (60, 163840)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_batches(T, V, dtype):
    _check(_x(T, V, dtype), _ids(T, V, 2), 5)


@pytest.mark.parametrize("k", [1, 2, 20, 63, 64])
@pytest.mark.parametrize("T", [2, 600])
def test_top_counts(T, k):
    _check(_x(T, 5000, seed=k), _ids(T, 5000, 1), k)


@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (3, 5), (4, 4), (8, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignments(pad, off, dtype):
    _check(_x(4, 4999, dtype, pad, off), _ids(4, 4999), 6)
    _check(_x(520, 4999, dtype, pad, off), _ids(520, 4999, 1), 6)


@pytest.mark.parametrize("k", [1, 7, 64])
@pytest.mark.parametrize("T", [1, 600])
def test_ties_go_to_the_lower_number(T, k):
    """Constant rows, a few values only, zeros of both signs: more elements reach the bound than a list holds."""
    V = 9001
    x = torch.zeros((T, V), device=DEV)
    _check(x, _ids(T, V, 1), k)
    x[:, ::2] = -0.0
    _check(x, _ids(T, V, 1), k)
    x[:, 5000:7000] = 1.0
    x[:, 17] = 1.0
    _check(x, _ids(T, V, 1), k)
    _check(torch.randint(0, 3, (T, V), device=DEV).to(torch.bfloat16), _ids(T, V, 1), k)


def test_banned_tokens():
    V = 20000
    x = _x(3, V)
    x[0, 100:] = float("-inf")                       # whole chunks without a token
    x[1, :19990] = float("-inf")
    x[2, 1:] = float("-inf")                         # one token only: sure of it
    _check(x, [[0, 99, 100], [5, 19990, 19999], [0, 1, 2]], 32)
    lp, e, _, _ = _run(x, [[0], [0], [0]])
    assert lp[2, 0] == 0.0 and e[2] == 0.0 and lp[1, 0] == -np.inf


@pytest.mark.parametrize("gap", [5.0, 12.0, 20.0, 60.0, 200.0])
def test_rows_nearly_sure_of_one_token(gap):
    """The probability that is left keeps its digits."""
    x = _x(2, 9000, spread=0.5)
    x[:, 4321] = gap + 9.0
    _check(x, [[4321, 0], [4321, 8999]], 3)


def test_ids_outside_have_no_probability():
    x = _x(2, 100)
    lp, _, _, _ = _run(x, [[-1, 100, 3], [2 ** 31 - 1, -2 ** 31, 99]])
    assert np.array_equal(np.isnan(lp), [[True, True, False], [True, True, False]])


def test_rows_that_are_no_distribution():
    x = _x(5, 6000)
    x[0] = float("-inf")
    x[1, 77] = float("nan")
    x[2, 5000] = float("inf")
    x[3] = float("nan")
    lp, e, ti, tl = _run(x, [[1]] * 5, 4)
    assert np.isnan(lp[:4]).all() and np.isnan(e[:4]).all() and np.isnan(tl[:4]).all()
    assert np.isfinite(lp[4]).all() and np.isfinite(e[4]) and np.isfinite(tl[4]).all()
    assert ti[0].tolist() == [0, 1, 2, 3] and ti[2, 0] == 5000 and ti[3].tolist() == [0, 1, 2, 3]
    clean = x[1].clone()
    clean[77] = float("-inf")
    assert ti[1].tolist() == torch.topk(clean, 4)[1].tolist()


def test_each_result_alone():
    x = _x(3, 5000)
    ids = _ids(3, 5000)
    lp, e, ti, tl = _run(x, ids, 4)
    assert np.array_equal(_run(x, ids, 0, ent=False)[0], lp)
    assert np.array_equal(_run(x)[1], e)
    a = _run(x, None, 4, ent=False)
    assert np.array_equal(a[2], ti) and np.array_equal(a[3], tl)


def test_same_bits_streams_and_graphs():
    x = _x(40, 30000)
    ws = k3.logprobs_workspace(40, 30000, 5, device=DEV)
    ws.fill_(0xff)
    want = _run(x, _ids(40, 30000), 5)
    for w, g in zip(want, _run(x, _ids(40, 30000), 5, ws=ws)):
        assert np.array_equal(w, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for w, g in zip(want, _run(x, _ids(40, 30000), 5, stream=s)):
        assert np.array_equal(w, g)
    ids = torch.zeros((40, 1), dtype=torch.int32, device=DEV)
    lp, ti, tl = torch.zeros((40, 1), device=DEV), torch.zeros((40, 5), dtype=torch.int32, device=DEV), torch.zeros((40, 5), device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        k3.logprobs(x, ids=ids, lp=lp, top_ids=ti, top_lp=tl, workspace=ws)
    for step in range(3):
        x.normal_()
        ids += 7
        got = [torch.zeros_like(t) for t in (lp, ti, tl)]
        k3.logprobs(x, ids=ids, lp=got[0], top_ids=got[1], top_lp=got[2])
        lp.zero_(), ti.zero_(), tl.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (lp, ti, tl)))


def test_rows_beyond_32_bits():
    T, V = 7000, 163840
    if torch.cuda.mem_get_info()[0] < T * V * 4 + 2 ** 32:
        pytest.skip("not enough device memory")
    x = torch.zeros((T, V), device=DEV)
    x[T - 1].normal_()
    ids = torch.full((T, 1), 5, dtype=torch.int32, device=DEV)
    lp, ti, tl = torch.zeros((T, 1), device=DEV), torch.zeros((T, 1), dtype=torch.int32, device=DEV), torch.zeros((T, 1), device=DEV)
    k3.logprobs(x, ids=ids, lp=lp, top_ids=ti, top_lp=tl)
    a, _, order, top, tol, _ = ref.logprobs(x[T - 1].cpu().numpy(), [5], 1)
    assert abs(float(lp[T - 1, 0]) - a[0]) <= tol + ref.U32 * abs(a[0]) and int(ti[T - 1, 0]) == order[0]
    assert int(ti[T - 2, 0]) == 0 and abs(float(lp[0, 0]) + np.log(V)) < 1e-5


def test_a_workspace_serves_fewer_rows():
    """160 rows of 32000 take half the chunks that 159 take."""
    V = 32000
    ws = k3.logprobs_workspace(160, V, 5, device=DEV)
    for T in (160, 159, 81, 80, 1):
        x, ids = _x(T, V, seed=T), _ids(T, V, 1)
        ws.fill_(0xff)
        for w, g in zip(_run(x, ids, 5), _run(x, ids, 5, ws=ws)):
            assert np.array_equal(w, g)
        for w, g in zip(_run(x, ids, 2), _run(x, ids, 2, ws=ws)):
            assert np.array_equal(w, g)

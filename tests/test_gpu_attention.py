"""k3moe_attention against its formula in 64 bits: head widths and groups,
lengths around the tiles, chunks, strides, empty rows, masked infinities."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda:0"
BF = torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


def _cu(ns):
    return torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device=DEV)


def _inputs(nq, nk, Hq, Hkv, D, Dv, seed=0, tail=0, pad=0, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(nq) + tail, sum(nk) + tail
    q = (sharp * torch.randn((Tq, Hq * D + pad), generator=g)).to(BF).to(DEV)[:, :Hq * D].view(Tq, Hq, D)
    w = torch.randn((Tk, Hkv * (D + Dv) + pad), generator=g).to(BF).to(DEV)
    return q, w[:, :Hkv * D].view(Tk, Hkv, D), w[:, Hkv * D:Hkv * (D + Dv)].view(Tk, Hkv, Dv)


def _check(q, k, v, nq, nk, causal, out, lse, scale, heads=None):
    Hq, Hkv = q.shape[1], k.shape[1]
    qn, kn, vn, on = _np(q), _np(k), _np(v), _np(out)
    ln = None if lse is None else _np(lse)
    a = b = 0
    for n, N in zip(nq, nk):
        i, j = np.arange(n)[:, None], np.arange(N)[None, :]
        see = (j <= i + N - n) if causal else np.ones((n, N), bool)
        for h in heads or range(Hq):
            kv = h // (Hq // Hkv)
            want = ref.attend(qn[a:a + n, h], kn[b:b + N, kv], vn[b:b + N, kv], see, scale)
            ref.check_rows(on[a:a + n, h], None if ln is None else ln[a:a + n, h], *want, f"{n}x{N} head {h}")
        a, b = a + n, b + N


def _case(nq, nk, Hq, Hkv, D, Dv, causal=True, seed=0, tail=0, pad=0, sharp=1.0, scale=None, heads=None, with_lse=True):
    q, k, v = _inputs(nq, nk, Hq, Hkv, D, Dv, seed, tail, pad, sharp)
    Tq = q.shape[0]
    out = torch.full((Tq, Hq * Dv + pad), 5.0, dtype=BF, device=DEV)[:, :Hq * Dv].view(Tq, Hq, Dv)
    lse = torch.full((Tq, Hq), 5.0, device=DEV) if with_lse else None
    k3.attention(q, k, v, _cu(nq), out, cu_k=None if list(nq) == list(nk) else _cu(nk), scale=scale, causal=causal, lse=lse)
    torch.cuda.synchronize()
    _check(q, k, v, nq, nk, causal, out, lse, D ** -0.5 if scale is None else scale, heads)
    assert (out[sum(nq):] == 5.0).all() and (lse is None or (lse[sum(nq):] == 5.0).all()), "rows of no sequence"


DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
def test_lengths(D, Dv, n):
    _case([n], [n], 2, 1, D, Dv)


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_packed(D, Dv, causal):
    _case([1, 70, 0, 33, 129, 2, 64], [1, 70, 0, 33, 129, 2, 64], 4, 2, D, Dv, causal, tail=3, pad=8)


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_more_tiles_than_cus(D, Dv, causal):
    """Two blocks on most CUs."""
    _case([257, 1, 130, 64], [257, 40, 700, 64], 96, 8, D, Dv, causal, heads=[0, 37, 95], tail=2)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (12, 4)])
def test_groups(Hq, Hkv):
    _case([40, 90], [40, 90], Hq, Hkv, 64, 64, pad=16)


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_and_empty_rows(D, Dv, causal):
    """More keys than queries, fewer (the first queries see none when causal), and no key at all."""
    _case([17, 130, 5, 9], [300, 131, 0, 4], 2, 2, D, Dv, causal)


def test_many_sequences():
    ns = [(7 * b) % 41 for b in range(200)]
    _case(ns, ns, 2, 1, 64, 64, heads=[1])


@pytest.mark.parametrize("sharp,scale", [(30.0, None), (1.0, 3.0), (1.0, 1e-3)])
def test_sharp_and_flat_rows(sharp, scale):
    _case([150], [150], 2, 1, 128, 128, sharp=sharp, scale=scale)


def test_rising_scores_raise_the_maximum_in_every_tile():
    n, D = 300, 64
    q, k, v = _inputs([n], [n], 1, 1, D, D)
    q.fill_(0.0), k.fill_(0.0)
    q[:, 0, 0], k[:, 0, 0] = 8.0, torch.arange(n, device=DEV).to(BF)      # s = j: 11.5 powers of two per 8 keys
    out, lse = torch.empty((n, 1, D), dtype=BF, device=DEV), torch.empty((n, 1), device=DEV)
    for sign in (1.0, -1.0):
        k3.attention(q, k * sign, v, _cu([n]), out, lse=lse)
        _check(q, k * sign, v, [n], [n], True, out, lse, D ** -0.5)


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("Hq", [2, 80])
def test_what_is_not_seen_has_no_influence(D, Dv, Hq):
    """NaN and infinities in keys and values behind a query, and in the other sequences' rows."""
    nq = [100, 3, 140]
    q, k, v = _inputs(nq, nq, Hq, 1, D, Dv)
    bad = [float("nan"), float("inf"), float("-inf")]
    clean, lse = torch.empty((sum(nq), Hq, Dv), dtype=BF, device=DEV), torch.empty((sum(nq), Hq), device=DEV)
    k3.attention(q, k, v, _cu(nq), clean, lse=lse)
    for b in bad:
        k2, v2 = k.clone(), v.clone()
        k2[60:100], v2[60:100] = b, b                                     # seen by queries 60 .. 99 of the first
        v2[103 + 77, 0, 5] = b                                            # one value, seen from query 77 on
        out, l2 = torch.empty_like(clean), torch.empty_like(lse)
        k3.attention(q, k2, v2, _cu(nq), out, lse=l2)
        torch.cuda.synchronize()
        assert torch.equal(out[:60], clean[:60]) and torch.equal(l2[:60], lse[:60])
        assert not torch.isfinite(out[60:100].float()).any()
        assert torch.equal(out[100:103], clean[100:103]) and torch.equal(l2[100:], lse[100:])
        third, want = out[103:].float(), clean[103:].float()
        assert not torch.isfinite(third[77:, :, 5]).any()
        if b == b:
            assert (third[77:, :, 5] == b).all()                          # an infinity weighs in as one
        third[77:, :, 5] = want[77:, :, 5] = 0
        assert torch.equal(third, want)


def test_scores_that_are_not_finite():
    q, k, v = _inputs([90], [90], 1, 1, 64, 64)
    q[20] = float("nan")
    q[30], k[:, :, :] = float("inf"), k.abs() + 1.0                       # every score +inf: no distribution
    q[40] = float("-inf")                                                 # every score -inf: nothing left
    out, lse = torch.empty((90, 1, 64), dtype=BF, device=DEV), torch.empty((90, 1), device=DEV)
    k3.attention(q, k, v, _cu([90]), out, lse=lse)
    o = out.float()
    assert torch.isnan(o[20]).all() and torch.isnan(o[30]).all() and (o[40] == 0).all() and lse[40] == float("-inf")
    rest = [i for i in range(90) if i not in (20, 30, 40)]
    assert torch.isfinite(o[rest]).all()


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [
    ([1], [512], 2), ([1], [4097], 1),                  # one token: 4 parts and 16
    ([100], [1000], 4), ([130], [1024], 8),             # rows behind the sequence's; a last tile that nearly all is
    ([1, 0, 3, 129], [0, 0, 5000, 700], 2),             # rows without keys, a sequence without rows
    ([700], [600], 1),                                  # causal: rows that see nothing, tiles without keys
    ([33, 300], [4000, 20], 3)])                        # parts that only one sequence has
def test_few_queries_split_their_keys(D, Dv, causal, nq, nk, H):
    assert k3._attention_bytes(len(nq), sum(nq), sum(nk), 2 * H, Dv) > 0
    _case(nq, nk, 2 * H, H, D, Dv, causal)


def test_split_results_agree_with_whole_ones_and_repeat():
    q, k, v = _inputs([200], [3001], 8, 2, 128, 128, 8)
    cq, ck = _cu([200]), _cu([3001])
    ws = k3.attention_workspace(1, 200, 3001, 8, 128, device=DEV)
    ws.fill_(255)                                       # what it holds has no influence

    def run(w):
        out, lse = torch.empty_like(q), torch.empty(200, 8, device=DEV)
        k3.attention(q, k, v, cq, out, cu_k=ck, lse=lse, workspace=w)
        return out, lse

    a, b, c = run(ws), run(ws), run(None)
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))
    out, lse = torch.empty_like(q), torch.empty(200, 8, device=DEV)
    p = lambda t: t.data_ptr()
    assert k3.lib().k3moe_attention(p(q), q.stride(0), p(k), k.stride(0), p(v), v.stride(0), p(cq), p(ck), 1, 200, 3001, 8, 2,
                                    128, 128, 128 ** -0.5, 1, p(out), out.stride(0), p(lse), None, 0,
                                    torch.cuda.current_stream().cuda_stream) == 0
    _check(q, k, v, [200], [3001], True, out, lse, 128 ** -0.5)
    with pytest.raises(k3.K3MoeError):
        run(ws[:1000])
    with pytest.raises((ValueError, TypeError)):
        run(ws.cpu())


def test_split_not_finite():
    """A row all of whose scores are -inf in one part, or in every one; NaN and infinities where they are not seen."""
    q, k, v = _inputs([2], [2000], 2, 1, 128, 128, 9)
    k, v = k.contiguous(), v.contiguous()
    q[0] = 1.0
    q[1] = torch.where(torch.arange(128, device=DEV) == 0, 1.0, 0.0).to(BF)
    k[:600, 0, 0] = -float("inf")
    k[1999], v[1999, 0, :5] = float("nan"), float("inf")    # the last key: only row 1 sees it
    out, lse = torch.empty(2, 2, 128, dtype=BF, device=DEV), torch.empty(2, 2, device=DEV)
    k3.attention(q, k, v, _cu([2]), out, cu_k=_cu([2000]), lse=lse)
    assert out[0].isfinite().all() and lse[0].isfinite().all() and out[1].isnan().all() and lse[1].isnan().all()
    k[:, 0, 0] = -float("inf")
    k[1999], v[1999] = k[1998], v[1998]
    k3.attention(q, k, v, _cu([2]), out, cu_k=_cu([2000]), lse=lse)
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_offsets_are_held_to_the_tensors():
    """Offsets behind the rows, falling ones and negative ones are cut, not followed."""
    q, k, v = _inputs([50], [50], 1, 1, 64, 64)
    out = torch.full((50, 1, 64), 5.0, dtype=BF, device=DEV)
    for cu in ([0, 90, 70], [-5, 20, 10], [60, 70, 80]):
        k3.attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()


def test_same_bits_streams_and_graphs():
    nq, nk = [40, 300, 1], [90, 300, 500]
    q, k, v = _inputs(nq, nk, 4, 2, 128, 128)
    cq, ck = _cu(nq), _cu(nk)
    a, b = (torch.zeros((sum(nq), 4, 128), dtype=BF, device=DEV) for _ in range(2))
    k3.attention(q, k, v, cq, a, cu_k=ck)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k3.attention(q, k, v, cq, b, cu_k=ck, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        k3.attention(q, k, v, cq, b, cu_k=ck)
    for step in range(3):
        q.normal_()
        cq[1] -= 1 + step               # other lengths in the same graph
        ck[1] += 2
        k3.attention(q, k, v, cq, a, cu_k=ck)
        b.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_split_calls_share_a_workspace_in_two_graphs():
    cases = []
    for D, Dv, nq, nk, H in ((128, 128, [200], [3001], 4), (192, 128, [5, 90], [2000, 800], 2), (128, 128, [1], [9000], 8)):
        q, k, v = _inputs(nq, nk, 2 * H, H, D, Dv, seed=len(cases))
        cases.append((q, k, v, _cu(nq), _cu(nk), torch.zeros((sum(nq), 2 * H, Dv), dtype=BF, device=DEV)))
    ws = k3.attention_workspace(1, 1, 9000, 16, 128, device=DEV)      # one size for all
    ws.fill_(255)

    def run(c, out, w=None, stream=None):
        k3.attention(c[0], c[1], c[2], c[3], out, cu_k=c[4], workspace=w, stream=stream)

    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, c[5], ws)
        graphs.append(g)
    for step in range(3):
        for c in cases:
            c[0].normal_()
            c[5].zero_()
        cases[0][3][1] -= step                                        # other lengths in the same graph
        for g in graphs:
            g.replay()
        want = [torch.empty_like(c[5]).copy_(c[5]) for c in cases]
        eager = [torch.zeros_like(c[5]) for c in cases]
        for c, o in zip(cases, eager):
            run(c, o, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, eager))
    s = torch.cuda.Stream()
    other = [torch.zeros_like(c[5]) for c in cases]
    s.wait_stream(torch.cuda.current_stream())
    for c, o in zip(cases, other):                                    # two streams at once, a workspace each
        run(c, o, None, s)
        run(c, c[5].zero_(), None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c[5]) for a, b, c in zip(other, eager, cases))


def test_rows_beyond_32_bits():
    """Keys more than 2^32 bytes behind the first ones."""
    T, W = 40000, 65536
    if torch.cuda.mem_get_info()[0] < T * W * 2 + 2 ** 30:
        pytest.skip("not enough device memory")
    wide = torch.zeros((T, W), dtype=BF, device=DEV)
    wide[:, :384].normal_()
    q, k, v = (wide[:, 128 * i:128 * i + 128].view(T, 1, 128) for i in range(3))
    n = 200
    cq = torch.tensor([T - n, T], dtype=torch.int32, device=DEV)
    ck = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    out, lse = torch.zeros((T, 1, 128), dtype=BF, device=DEV), torch.zeros((T, 1), device=DEV)
    k3.attention(q, k, v, cq, out, cu_k=ck, lse=lse)
    rows = [0, 77, 199]
    qn, kn, vn = _np(q[T - n:])[rows, 0], _np(k)[:, 0], _np(v)[:, 0]
    see = np.arange(T)[None, :] <= np.array(rows)[:, None] + T - n
    want = ref.attend(qn, kn, vn, see, 128 ** -0.5)
    ref.check_rows(_np(out[T - n:])[rows, 0], _np(lse[T - n:])[rows, 0], *want, "far rows")


def test_a_workspace_serves_smaller_calls():
    """Made for a call that is not split, used by smaller ones that are."""
    ws = k3.attention_workspace(1, 3000, 3000, 32, 128, device=DEV)
    for nq, nk in ((3000, 3000), (64, 2999), (1, 600), (64, 100)):
        q, k, v = _inputs([nq], [nk], 32, 4, 128, 128, seed=nq)
        ws.fill_(0xff)
        a, b = torch.zeros_like(q), torch.zeros_like(q)
        k3.attention(q, k, v, _cu([nq]), a, cu_k=_cu([nk]), workspace=ws)
        k3.attention(q, k, v, _cu([nq]), b, cu_k=_cu([nk]))
        assert torch.equal(a, b) and a.float().abs().sum() > 0


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("nq,nk,H", [(1, 256, 8), (1, 320, 8), (1, 383, 8), (1, 384, 8), (1, 511, 8), (128, 511, 32)])
def test_a_given_workspace_changes_nothing(D, Dv, nq, nk, H):
    """Around the fewest keys that are split: the same bits with a workspace given and without."""
    _case([nq], [nk], H, H // 4, D, Dv, heads=[0, H - 1])
    q, k, v = _inputs([nq], [nk], H, H // 4, D, Dv)
    ws = k3.attention_workspace(1, 128, 5000, H, Dv, device=DEV)
    a, b = (torch.zeros((nq, H, Dv), dtype=BF, device=DEV) for _ in range(2))
    k3.attention(q, k, v, _cu([nq]), a, cu_k=_cu([nk]))
    k3.attention(q, k, v, _cu([nq]), b, cu_k=_cu([nk]), workspace=ws)
    assert torch.equal(a, b)

"""k3moe_qk_norm_rope against its formula in 64 bits: widths, head counts,
rotations, strides, positions, both kinds of cache, places outside it."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda:0"
BF = torch.bfloat16


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _case(T, Hq, Hkv, D, Dv, R, pairs, cache, page=16, norm=True, pad=0, far=4096, seed=0, in_place=False, k_out=True,
          stream=None):
    g = torch.Generator().manual_seed(seed)
    W = (Hq + Hkv) * D + Hkv * Dv + pad
    wide = (torch.randn((T, W), generator=g) * torch.exp2(torch.randint(-6, 7, (T, 1), generator=g).float())).to(BF).to(DEV)
    q = wide[:, :Hq * D].view(T, Hq, D) if T else wide.new_empty((0, Hq, D))
    k = wide[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D) if T else wide.new_empty((0, Hkv, D))
    v = wide[:, (Hq + Hkv) * D:(Hq + Hkv) * D + Hkv * Dv].view(T, Hkv, Dv) if T else wide.new_empty((0, Hkv, Dv))
    qn, kn, vn = (ref.unbf16(_bits(t)) for t in (q, k, v))
    gq = (1 + 0.2 * torch.randn(D, generator=g)).to(DEV) if norm else None
    gk = (1 + 0.2 * torch.randn(D, generator=g)).to(DEV) if norm else None
    pos = (torch.randint(0, far, (T,), generator=g) - far // 8).to(torch.int32).to(DEV)
    freq = torch.tensor([10000.0 ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float32, device=DEV) if R else None
    a = dict(gamma_q=gq, gamma_k=gk, eps=1e-5, rot=k3.ROT_PAIRS if pairs else k3.ROT_HALVES)
    a["q_out"] = q if in_place else torch.zeros((T, Hq, D), dtype=BF, device=DEV)
    a["k_out"] = (k if in_place else torch.zeros((T, Hkv, D), dtype=BF, device=DEV)) if k_out else None
    pages = T // page + 2
    slots = None
    if cache:
        slots = torch.randperm(pages * page, generator=g)[:T]
        drop = torch.rand(T, generator=g) < 0.2
        slots = torch.where(drop, torch.where(torch.rand(T, generator=g) < 0.5, -1, pages * page + 3), slots)
        a["v"], a["slots"] = v, slots.to(DEV)
        if cache == "bf16":
            a["kc"] = torch.full((pages, Hkv, page, D), 7.0, dtype=BF, device=DEV)
            a["vc"] = torch.full((pages, Hkv, page, Dv), 7.0, dtype=BF, device=DEV)
        else:
            for n, d in (("k", D), ("v", Dv)):
                a[n + "c"] = torch.full((pages, Hkv, page, d), 9, dtype=torch.uint8, device=DEV)
                a[n + "s"] = torch.full((pages, Hkv, page, d // 32), 9, dtype=torch.uint8, device=DEV)
    k3.qk_norm_rope(q, k, pos, freq, stream=stream, **a)
    torch.cuda.synchronize()
    p, f = pos.cpu().numpy(), freq.cpu().numpy() if R else np.zeros(0)
    gnp = [None, None] if not norm else [gq.cpu().numpy().astype(float), gk.cpu().numpy().astype(float)]
    yq, tq = ref.heads(qn, gnp[0], 1e-5, p, f, pairs)
    yk, tk = ref.heads(kn, gnp[1], 1e-5, p, f, pairs)

    def near(got, y, t, what):
        assert (np.abs(got - y) <= ref.U16 * (np.abs(y) + t) + t + 2.0 ** -134).all(), what
    near(ref.unbf16(_bits(a["q_out"])), yq, tq, "q_out")
    if k_out:
        near(ref.unbf16(_bits(a["k_out"])), yk, tk, "k_out")
    if cache:
        s = slots.numpy()
        ok = (s >= 0) & (s < pages * page)
        at = s[ok]
        rest = np.ones((pages, page), bool)
        rest[at // page, at % page] = False
        if cache == "bf16":
            kc, vc = _bits(a["kc"]), _bits(a["vc"])
            near(ref.unbf16(kc[at // page, :, at % page]), yk[ok], tk[ok], "kc")
            assert np.array_equal(ref.unbf16(vc[at // page, :, at % page]), vn[ok])
            for c in (kc, vc):
                assert (c.transpose(0, 2, 1, 3)[rest] == 0x40e0).all(), "other places"
        else:
            for n, y, t in (("k", yk, tk), ("v", vn, 0 * vn)):
                c, b = a[n + "c"].cpu().numpy(), a[n + "s"].cpu().numpy()
                ref.check_mxfp8(c[at // page, :, at % page], b[at // page, :, at % page], y[ok], t[ok], n)
                assert (c.transpose(0, 2, 1, 3)[rest] == 9).all() and (b.transpose(0, 2, 1, 3)[rest] == 9).all()
    return a


@pytest.mark.parametrize("D,Dv,R", [(64, 64, 64), (128, 128, 128), (192, 128, 64), (128, 64, 0), (256, 256, 256),
                                    (8, 8, 0), (16, 40, 16), (72, 72, 48), (96, 32, 96), (248, 8, 16)])
@pytest.mark.parametrize("pairs", [False, True])
def test_widths(D, Dv, R, pairs):
    _case(13, 6, 3, D, Dv, R, pairs, "bf16", pad=8)


@pytest.mark.parametrize("T", [0, 1, 2, 7, 65, 700])
@pytest.mark.parametrize("cache", [None, "bf16", "mxfp8"])
def test_token_counts(T, cache):
    _case(T, 8, 2, 128, 128, 64, False, cache, page=32)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (64, 8), (96, 1), (33, 11)])
@pytest.mark.parametrize("cache", ["bf16", "mxfp8"])
def test_head_counts(Hq, Hkv, cache):
    _case(3, Hq, Hkv, 64, 96, 64, True, cache)


@pytest.mark.parametrize("far", [16, 2 ** 20, 2 ** 30])
@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(far, pairs):
    """Angles of 2^30 radians: an fp32 product would be off by half a turn and more."""
    _case(33, 2, 1, 128, 128, 128, pairs, None, far=far)


@pytest.mark.parametrize("norm", [True, False])
def test_in_place_and_without_norm(norm):
    _case(21, 4, 2, 128, 128, 128, False, "bf16", norm=norm, in_place=True, pad=16)
    _case(21, 4, 2, 64, 64, 32, True, "mxfp8", norm=norm, k_out=False)


def test_other_stream_and_graph():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _case(9, 4, 2, 128, 128, 128, False, "bf16", stream=s)
    q = torch.randn((5, 4, 64), device=DEV).to(BF)
    k = torch.randn((5, 2, 64), device=DEV).to(BF)
    pos, f = torch.arange(5, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV)
    qo, ko, want = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    k3.qk_norm_rope(q, k, pos, f, q_out=qo, k_out=ko)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        k3.qk_norm_rope(q, k, pos, f, q_out=qo, k_out=ko)
    for step in range(3):
        q.normal_()
        pos += 3
        k3.qk_norm_rope(q, k, pos, f, q_out=want)
        qo.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want)


def test_values_that_are_not_finite_stay_in_their_heads():
    q = torch.randn((2, 4, 64), device=DEV).to(BF)
    k = torch.randn((2, 2, 64), device=DEV).to(BF)
    v = torch.randn((2, 2, 64), device=DEV).to(BF)
    k[0, 0, 5], k[1, 1, 3], v[1, 0, 33] = float("inf"), float("nan"), float("inf")
    kc, vc = (torch.zeros((1, 2, 16, 64), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((1, 2, 16, 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    qo, g = torch.empty_like(q), torch.ones(64, device=DEV)
    k3.qk_norm_rope(q, k, torch.arange(2, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV), gamma_q=g, gamma_k=g,
                    q_out=qo, v=v, kc=kc, vc=vc, ks=ks, vs=vs, slots=torch.tensor([3, 4], device=DEV))
    kv, vv = kc.view(torch.float8_e4m3fn).float(), vc.view(torch.float8_e4m3fn).float()
    assert torch.isfinite(qo.float()).all()
    bad = torch.isnan(kv).any(-1)[0]
    assert bad[0, 3] and bad[1, 4] and not bad[1, 3] and not bad[0, 4]
    nan = torch.isnan(vv)
    assert nan.sum() == 1 and nan[0, 0, 4, 33]      # an infinity is held as NaN, its neighbours as what they are


def test_a_cache_beyond_32_bits():
    pages, Hkv, page, D = 40000, 4, 64, 256
    if torch.cuda.mem_get_info()[0] < 2 * pages * Hkv * page * D * 2 + 2 ** 30:
        pytest.skip("not enough device memory")
    kc = torch.zeros((pages, Hkv, page, D), dtype=BF, device=DEV)
    vc = torch.zeros((pages, Hkv, page, 64), dtype=BF, device=DEV)
    assert kc.numel() * 2 > 2 ** 32
    k = torch.randn((2, Hkv, D), device=DEV).to(BF)
    v = torch.randn((2, Hkv, 64), device=DEV).to(BF)
    at = torch.tensor([pages * page - 1, (pages - 7) * page + 5], device=DEV)
    k3.qk_norm_rope(k, k, None, None, v=v, kc=kc, vc=vc, slots=at)
    for t in range(2):
        n, r = int(at[t]) // page, int(at[t]) % page
        assert torch.equal(kc[n, :, r], k[t]) and torch.equal(vc[n, :, r], v[t])
    assert int(torch.count_nonzero(kc[:pages - 7])) == 0


@pytest.mark.parametrize("D", [64, 128, 256, 72])
@pytest.mark.parametrize("eps", [1e-5, 1e-40])
def test_heads_of_any_magnitude(D, eps):
    """Squares beyond fp32, squares below it, and heads of zeros, beside ordinary ones in the same wave."""
    g = torch.Generator().manual_seed(D)
    size = torch.tensor([1.0, 1e25, 3e37, 1e-18, 1e-25, 1e-37, 0.0, 1e18, 1e20, 1.0])
    k = (torch.randn((3, 10, D), generator=g).clamp(-4, 4) * size[None, :, None]).to(BF).to(DEV)
    gamma = (1 + 0.2 * torch.randn(D, generator=g)).to(DEV)
    out = torch.full_like(k, 5.0)
    k3.qk_norm_rope(k, k, None, None, gamma_q=gamma, gamma_k=gamma, eps=eps, q_out=out)
    torch.cuda.synchronize()
    eps = float(np.float32(eps))
    y, tol = ref.heads(ref.unbf16(_bits(k)), gamma.cpu().numpy().astype(float), eps, np.zeros(3), np.zeros(0), False)
    got = ref.unbf16(_bits(out))
    assert (np.abs(got - y) <= ref.U16 * (np.abs(y) + tol) + tol + 2.0 ** -133).all(), np.isfinite(got).all((0, 2))

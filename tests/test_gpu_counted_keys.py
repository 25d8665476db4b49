"""Every key counts once, at any length. With keys of zero every weight is 1,
and with values that are 1 in one dimension per run of 16 keys and else 0 every
sum is a whole number that fp32 holds: a result is the share of the keys seen
that belong to its dimension, rounded to bf16 (2^-8), behind an inverse and a
product (2^-24 each, the inverse within an ulp); the lse is the logarithm of
their number, a logarithm within an ulp, a sum and a product. Sixteen keys that
are lost or counted twice are 5 % of a dimension and more."""
import math

import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref
from test_gpu_attention import BF, DEV, DIMS, _cu
from test_gpu_tree import Case, _tree

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def _near(out, lse, see, Dv, what):
    """out [n][Dv] and lse [n] of rows that see the keys of see [n][N]."""
    of = np.arange(see.shape[1]) // 16 % Dv
    count = see @ (of[:, None] == np.arange(Dv)[None, :]).astype(np.float64)
    n = see.sum(1)
    want = count / np.maximum(n, 1)[:, None]
    assert (np.abs(out - want) <= (ref.U16 + 4 * ref.U32) * want).all(), what
    for i, m in enumerate(n):
        if m:
            assert abs(lse[i] - math.log(m)) <= 8 * ref.U32 * (1 + math.log(m)), (what, i)
        else:
            assert lse[i] == -math.inf, (what, i)


def _ones(N, Dv):
    v = np.zeros((N, Dv))
    v[np.arange(N), np.arange(N) // 16 % Dv] = 1.0
    return v


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("group,ns", [(4, [1, 1, 1]), (4, [3, 8, 1]), (4, [12, 0, 16]), (4, [40, 17, 64])])
def test_drafted_tokens(D, Dv, x8, group, ns):
    lens = [20000, 9, 7003]
    c = Case(lens, ns, 2 * group, 2, D, Dv, page=64, x8=x8, words=_tree(ns))
    for b, (a, n) in enumerate(zip(lens, ns)):
        p = np.arange(a + n)
        c.k[c.table[b, p // c.page], :, p % c.page] = 0.0
        c.v[c.table[b, p // c.page], :, p % c.page] = _ones(a + n, Dv)[:, None, :]
    for name in ("k", "v"):
        x = getattr(c, name)
        if x8:
            q, s = ref.mxfp8_pool(np.where(np.isnan(x), 0.0, x))
            q[np.isnan(x)] = 0x7f
            c.cache[name + "c"], c.cache[name + "s"] = torch.tensor(q, device=DEV), torch.tensor(s, device=DEV)
        else:
            c.cache[name + "c"] = torch.tensor(ref.bf16(x).view(np.int16), device=DEV).view(BF)
    out, lse = c.run()
    torch.cuda.synchronize()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    first = 0
    for b, n in enumerate(ns):
        for h in range(2 * group):
            _near(o[first:first + n, h], l[first:first + n, h], c.see(b), Dv, f"sequence {b} head {h}")
        first += n


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [([1], [40000], 4), ([200], [9000], 2), ([33, 300], [4000, 20], 2), ([3000], [3000], 2),
                                     ([1, 700, 0, 2047, 129], [1, 700, 5, 2047, 129], 16)])
def test_prompts(D, Dv, causal, nq, nk, H):
    q = torch.randn((sum(nq), H, D), device=DEV).to(BF)
    k = torch.zeros((sum(nk), 1, D), dtype=BF, device=DEV)
    v = torch.tensor(np.concatenate([_ones(N, Dv) for N in nk]), device=DEV).to(BF).view(sum(nk), 1, Dv)
    out, lse = torch.empty((sum(nq), H, Dv), dtype=BF, device=DEV), torch.empty((sum(nq), H), device=DEV)
    k3.attention(q, k, v, _cu(nq), out, cu_k=_cu(nk), causal=causal, lse=lse)
    torch.cuda.synchronize()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    a = 0
    for n, N in zip(nq, nk):
        i, j = np.arange(n)[:, None], np.arange(N)[None, :]
        see = (j <= i + N - n) if causal else np.ones((n, N), bool)
        for h in {0, H - 1}:
            _near(o[a:a + n, h], l[a:a + n, h], see, Dv, f"{n}x{N} head {h}")
        a += n

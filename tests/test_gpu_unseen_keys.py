"""What a row does not see leaves its bits alone, however large: keys that only
other rows of the same block see."""
import math

import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
from test_gpu_attention import DIMS, _cu, _inputs
from test_gpu_tree import Case

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda:0"


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("nq,nk,key", [(128, 128, 120), (300, 300, 250), (300, 700, 690), (20, 3000, 2990)])
def test_a_large_key_of_later_queries(D, Dv, nq, nk, key):
    q, k, v = _inputs([nq], [nk], 4, 2, D, Dv, seed=4)

    def run(k):
        out, lse = torch.zeros((nq, 4, Dv), dtype=torch.bfloat16, device=DEV), torch.zeros((nq, 4), device=DEV)
        k3.attention(q, k, v, _cu([nq]), out, cu_k=_cu([nk]), lse=lse)
        return out, lse

    first = key - (nk - nq)                       # the first query that sees the key
    out, lse = run(k)
    for f in (8.0, -8.0, 60.0, -60.0):
        large = k.clone()
        large[key] *= f
        o2, l2 = run(large)
        assert torch.equal(o2[:first], out[:first]) and torch.equal(l2[:first], lse[:first]), f
        assert not torch.equal(l2[first:], lse[first:])


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("group,n,ctx", [(2, 6, 60100), (4, 16, 30100), (4, 20, 70), (4, 32, 1000), (8, 16, 9050)])
def test_a_large_key_of_a_sibling(D, Dv, x8, group, n, ctx):
    """Drafted tokens that see the context and themselves: one's large key, every other one's bits."""
    c = Case([333, ctx], [n, n], 2 * group, 2, D, Dv, page=64, x8=x8, words=[1 << i for i in range(n)] * 2)
    out, lse = c.run()
    at = ctx + n // 2                               # a drafted token of the second sequence
    page, row = c.table[1, at // c.page], at % c.page
    rest = [i for i in range(2 * n) if i != n + n // 2]
    for f in (3, 6):                                # times 8 and 64
        keep = dict(c.cache)
        if x8:
            c.cache["ks"] = c.cache["ks"].clone()
            c.cache["ks"][page, :, row] += f
        else:
            c.cache["kc"] = c.cache["kc"].clone()
            c.cache["kc"][page, :, row] *= 2.0 ** f
        o2, l2 = c.run()
        c.cache = keep
        assert torch.equal(o2[rest], out[rest]) and torch.equal(l2[rest], lse[rest]), f
        assert not torch.equal(l2[n + n // 2], lse[n + n // 2])


def _huge(n_keys, D, rows, low, high):
    """Queries and keys with scores of 1, but for `low` at the keys low and `high` at the keys high (times the scale 2:
    beyond fp32): q = (1, 2^62, 0 ..), k = (0.5, 0 or +-1.35 * 2^65, 0 ..)."""
    q, k = torch.zeros(rows, D), torch.zeros(n_keys, D)
    q[:, 0], q[:, 1] = 1.0, 2.0 ** 62
    k[:, 0] = 0.5
    k[low, 1], k[high, 1] = -1.375 * 2.0 ** 65, 1.375 * 2.0 ** 65
    return q.to(torch.bfloat16), k.to(torch.bfloat16)


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("rows,n_keys", [(300, 300), (4, 3000)])
@pytest.mark.parametrize("first", [0, 70])
def test_scores_beyond_fp32_count_as_infinities(D, Dv, rows, n_keys, first):
    """Below it: a weight of 0, also where a whole tile is. Above it: the row is no distribution."""
    low = list(range(first, first + 150))
    q, k = _huge(n_keys, D, rows, low, [n_keys - 1])
    v = torch.randn(n_keys, 1, Dv, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    q, k = q.view(rows, 1, D).to(DEV), k.view(n_keys, 1, D).to(DEV)
    out, lse = torch.zeros((rows, 1, Dv), dtype=torch.bfloat16, device=DEV), torch.zeros((rows, 1), device=DEV)
    k3.attention(q, k, v, _cu([rows]), out, cu_k=_cu([n_keys]), lse=lse, scale=2.0)
    torch.cuda.synchronize()
    assert torch.isnan(out[-1].float()).all() and torch.isnan(lse[-1]).all()      # the last query sees the last key
    keep = torch.ones(n_keys, dtype=torch.bool)
    keep[low] = False
    for i in range(0, rows - 1, max(1, rows // 60)):
        seen = keep.clone()
        seen[i + n_keys - rows + 1:] = False
        n = int(seen.sum())
        if not n:
            assert (out[i] == 0).all() and lse[i] == -float("inf"), i
            continue
        want = v[seen.to(DEV), 0].double().mean(0)
        # n weights of 1, each sum of them within n 2^-24, and the rounding of the result to bf16
        assert ((out[i, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + n * 2.0 ** -23 * 5).all(), i
        assert abs(float(lse[i]) - 1 - math.log(n)) <= n * 2.0 ** -24 + 2.0 ** -20, i


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("group,n", [(2, 4), (8, 16)])
def test_drafts_scores_beyond_fp32_count_as_infinities(D, Dv, group, n):
    c = Case([9000, 300], [n, n], 2 * group, 2, D, Dv, page=64, words=[1 << i for i in range(n)] * 2)
    at = [9000 + n, 300 + n]
    lows = [list(range(0, 200)) + list(range(4000, 4400)), list(range(64, 192))]
    for b in range(2):
        q, k = _huge(at[b], D, n, lows[b], [at[b] - 1])
        p = torch.arange(at[b])
        page = torch.tensor(c.table[b, (p // c.page).numpy()]).long().to(DEV)
        kc = c.cache["kc"]
        kc[page, :, (p % c.page).to(DEV)] = k.to(DEV)[:, None, :]
        c.q[b * n:(b + 1) * n] = q.to(DEV)[:, None, :]
    out = torch.zeros((2 * n, 2 * group, Dv), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((2 * n, 2 * group), device=DEV)
    k3.tree_attention(c.q, pages=c.pages, lens=c.dlens, out=out, cu_q=c.cu, max_q=n, lse=lse, scale=2.0,
                      tree=torch.tensor(c.words, device=DEV), **c.cache)
    torch.cuda.synchronize()
    for b in range(2):
        last = (b + 1) * n - 1
        assert torch.isnan(out[last].float()).all() and torch.isnan(lse[last]).all()
        m = at[b] - n - len(lows[b]) + 1                  # the context that counts, and the token itself
        l = lse[b * n:last].double()
        assert ((l - 1 - math.log(m)).abs() <= m * 2.0 ** -24 + 2.0 ** -20).all()
        assert torch.isfinite(out[b * n:last].float()).all()

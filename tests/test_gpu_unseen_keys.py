"""What a row does not see leaves its bits alone, however large: keys that only
other rows of the same block see."""
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

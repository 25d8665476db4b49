"""Workspace sizes serve every smaller call. No GPU: only sizes are asked for."""
import ctypes

import pytest

import mxfp4_routed_expert_sigmoid_amd as k3


@pytest.mark.parametrize("V", [1, 4096, 8192, 8193, 32000, 163840, 2 ** 23, 2 ** 24])
@pytest.mark.parametrize("k", [0, 1, 20, 64])
def test_logprobs_sizes_do_not_fall(V, k):
    """Rows take shorter chunks, and so more of them, below a number of rows."""
    if k > V:
        pytest.skip("no such call")
    n = ctypes.c_size_t()
    last = [0] * 3
    for T in range(0, 800):
        for i, kk in enumerate((k, k // 2, 0)):
            assert k3.lib().k3moe_logprobs_workspace_size(T, V, kk, ctypes.byref(n)) == 0
            assert n.value >= last[i], T
            last[i] = n.value
        assert last[0] >= last[1] >= last[2]


@pytest.mark.parametrize("heads", [1, 8, 32, 96, 255, 256, 257])
@pytest.mark.parametrize("v_dim", [64, 128])
def test_an_attention_size_serves_every_smaller_call(heads, v_dim):
    """A call that is not split by itself may be larger than one that is."""
    sizes = [(1, 8192, 8192), (7, 4264, 4264), (64, 64, 70000), (3, 1024, 4096), (1, 1, 300)]
    for seqs, Tq, Tk in sizes:
        most = k3._attention_bytes(seqs, Tq, Tk, heads, v_dim)
        for s in {1, 2, seqs}:
            for q in {1, 64, 129, Tq}:
                for k in {1, 255, 512, 4096, Tk}:
                    if s <= seqs and q <= Tq and k <= Tk:
                        assert k3._attention_bytes(s, q, k, heads, v_dim) <= most, (seqs, Tq, Tk, s, q, k)
    assert k3._attention_bytes(1, 8192, 8192, 32, v_dim) >= k3._attention_bytes(1, 64, 4096, 32, v_dim) > 0


@pytest.mark.parametrize("v_dim,most", [(64, 18e6), (128, 35e6)])
def test_a_tree_workspace_is_what_its_variants_use(v_dim, most):
    """Two ends of 256 runs of 128 rows, or of 512 of 32, each of v_dim + 2 numbers."""
    assert 2 * 256 * 128 * (v_dim + 2) * 4 <= k3._tree_bytes(8, 2, v_dim, 64) <= most

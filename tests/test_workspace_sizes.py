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

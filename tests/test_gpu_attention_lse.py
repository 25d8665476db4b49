"""The attention checks again with a NaN in lse counted as wrong: a comparison
that asks whether |lse - want| exceeds its bound is never true of one. And what
offsets that are held to the tensors define."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref
import test_gpu_attention as prompts
from test_gpu_attention import BF, DEV, DIMS, _inputs
from test_gpu_tree import Case, _tree


def needs_gpu(f):
    return pytest.mark.gpu(pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")(f))


@pytest.fixture
def strict(monkeypatch):
    """ref.check_rows, with every number inside its bound."""
    plain = ref.check_rows

    def check(got, lse, want, want_lse, tol, ltol, what):
        plain(got, lse, want, want_lse, tol, ltol, what)
        empty = np.isneginf(want_lse)
        assert (empty | (np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, want_lse)) <= ltol)).all(), f"{what}: lse"

    monkeypatch.setattr(ref, "check_rows", check)


def test_a_nan_is_wrong(strict):
    one = np.ones((1, 1)), np.ones(1), np.ones((1, 1)), np.full(1, 1e-6)
    ref.check_rows(np.ones((1, 1)), np.ones(1), *one, "right")
    with pytest.raises(AssertionError):
        ref.check_rows(np.ones((1, 1)), np.full(1, np.nan), *one, "wrong")


@needs_gpu
@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [([1, 70, 0, 33, 129], [1, 70, 0, 33, 129], 4), ([17, 130, 5, 9], [300, 131, 0, 4], 2),
                                     ([100], [1000], 4), ([1, 0, 3, 129], [0, 0, 5000, 700], 2), ([700], [600], 2)])
def test_prompts(strict, D, Dv, causal, nq, nk, H):
    prompts._case(nq, nk, H, H // 2, D, Dv, causal)


@needs_gpu
@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("ns", [[1, 1, 0, 1], [4, 8, 1, 2], [16, 3, 11, 9], [40, 1, 0, 64]])
def test_drafted_tokens(strict, D, Dv, x8, ns):
    c = Case([100, 0, 333, 3000], ns, 8, 2, D, Dv, x8=x8, words=_tree(ns))
    c.check(*c.run(), heads=[0, 3, 7])


@needs_gpu
def test_rows_that_held_offsets_define():
    """Offsets are held to 0 .. 50 each; a sequence whose end is then in front of its start has no rows (the last case:
    50 .. 0, then 0 .. 50)."""
    q, k, v = _inputs([50], [50], 1, 1, 64, 64)
    for cu, n in (([0, 90, 70], 50), ([-5, 20, 10], 20), ([60, 70, 80], 0), ([0, 50, 7], 50), ([2 ** 31 - 1, -2 ** 31, 50], 50)):
        out, lse = torch.full((50, 1, 64), 5.0, dtype=BF, device=DEV), torch.full((50, 1), 5.0, device=DEV)
        k3.attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), out, lse=lse)
        torch.cuda.synchronize()
        assert (out[n:] == 5.0).all() and (lse[n:] == 5.0).all(), cu
        if n:
            prompts._check(q[:n], k[:n], v[:n], [n], [n], True, out[:n], lse[:n], 64 ** -0.5)

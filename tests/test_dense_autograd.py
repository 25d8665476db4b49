"""The dense operators write tensors that autograd may know of: a result that
requires grad is refused, and what a call wrote counts as changed, so that a
backward pass that saved it raises instead of using the new values."""
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
from test_dense_abi import _z

BF, U8 = torch.bfloat16, torch.uint8


def _tracked(*shape, dtype=torch.float32):
    t = _z(*shape, dtype=dtype)
    t.t.requires_grad_()
    return t


def _calls(mk, track):
    """(name of the tracked result, the call) with `track` making that tensor and `mk` the others."""
    w, s = mk(40, 32, dtype=U8), mk(40, 2, dtype=U8)
    x = mk(3, 64, dtype=BF)
    h, d, g = mk(3, 64), mk(3, 64), mk(64)
    yield "h", lambda: k3.add_norm(track(3, 64), g, 1e-5, d=d, x=x)
    yield "x", lambda: k3.add_norm(h, g, 1e-5, d=d, x=track(3, 64, dtype=BF))
    yield "out", lambda: k3.linear(w, s, x, track(3, 40, dtype=BF))
    yield "h of +=", lambda: k3.linear(w, s, x, track(3, 40), accumulate=True)
    yield "a", lambda: k3.glu(w, s, w, s, x, track(3, 40))


@pytest.mark.parametrize("i", range(5))
def test_results_that_require_grad_are_refused(monkeypatch, i):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the call was made"))
    _, call = list(_calls(_z, _tracked))[i]
    with pytest.raises(ValueError, match="requires grad"):
        call()


def _gpu(*shape, dtype=torch.float32):
    return torch.ones(shape, device="cuda:0").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(5))
def test_written_tensors_count_as_changed(i):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    leaf = torch.ones((), device="cuda:0", requires_grad=True)
    y = []

    def saved(*shape, dtype=torch.float32):
        t = _gpu(*shape, dtype=dtype)
        y.append((leaf * t).sum())          # saves t for the gradient of leaf
        return t
    _, call = list(_calls(_gpu, saved))[i]
    call()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y[-1].backward()


@pytest.mark.gpu
def test_a_norm_without_results_is_the_librarys_refusal():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with pytest.raises(k3.K3MoeError):
        k3.add_norm(_gpu(3, 64), _gpu(64), 1e-5)


@pytest.mark.gpu
def test_results_may_require_grad_where_none_is_recorded():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = _gpu(3, 64).requires_grad_()
    v = h._version
    with torch.no_grad():
        k3.add_norm(h, _gpu(64).requires_grad_(), 1e-5, d=_gpu(3, 64), x=_gpu(3, 64, dtype=BF))
    assert bool((h == 2).all()) and h._version > v
    with torch.inference_mode():
        x = _gpu(3, 64, dtype=BF)
        k3.add_norm(h, _gpu(64), 1e-5, x=x)
    assert bool((x.float() == 1).all())

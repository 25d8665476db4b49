"""Which stream a workspace belongs to that a call makes itself: the stream that
uses it. The caching allocator gives a freed block out again in the order of
the stream that it was allocated on; a block of another stream could be written
by one call while an earlier call's kernels still read it. No GPU: the
allocation and the streams are stand-ins."""
import contextlib
import types

import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3


class _Stream:
    cuda_stream = 7


class _Bytes:
    """A workspace that remembers the stream it was made under."""

    def __init__(self, n, on):
        self.n, self.on = n, on

    def data_ptr(self):
        return 0x1010

    def numel(self):
        return self.n

    def record_stream(self, stream):
        pytest.fail("a block of another stream is marked instead of one of this stream")


@pytest.fixture
def current(monkeypatch):
    """[the current stream], with torch's streams and allocation replaced."""
    now = [_Stream()]

    @contextlib.contextmanager
    def under(stream):
        if stream is None:                       # as torch's own: no change
            yield
            return
        before, now[0] = now[0], stream
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: _Bytes(n, now[0]))
    return now


@pytest.mark.parametrize("other", [False, True])
def test_scratch_of_the_functions(current, other):
    stream = _Stream() if other else None
    want = stream or current[0]
    ws, at, n = k3._scratch(None, lambda: 1000, torch.device("cuda:0"), stream)
    assert ws.on is want and at % 256 == 0 and n >= 1000
    assert current[0] is not stream
    mine = _Bytes(5000, None)
    assert k3._scratch(mine, lambda: pytest.fail("not needed"), torch.device("cuda:0"), stream)[0] is mine


@pytest.mark.parametrize("other", [False, True])
def test_scratch_of_a_layer(current, other):
    stream = _Stream() if other else None
    want = stream or current[0]
    layer = types.SimpleNamespace(device=torch.device("cuda:0"), workspace_size=lambda T: 100 * T)
    layer.workspace = lambda T: k3.Layer.workspace(layer, T)
    assert k3.Layer._call_ws(layer, None, 3, stream).on is want
    mine = _Bytes(5000, None)
    assert k3.Layer._call_ws(layer, mine, 3, stream) is mine

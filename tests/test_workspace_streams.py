"""A workspace that the binding allocates belongs to the stream that the call runs on (CPU: the
library is replaced by one that only counts calls, streams by names)."""
import contextlib

import pytest
import torch

from embedding_lookup_feature_amd import embcore as ec
from embedding_lookup_feature_amd import tower as tw


class FakeLibrary:
    """Every size query answers 4096, every call succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return lambda *a: self.calls.append(name) or ec.EL_OK


@pytest.fixture
def streams(monkeypatch):
    """The stream on which each torch.empty of the binding was made ("current" outside of any)."""
    at, made, lib = ["current"], [], FakeLibrary()

    @contextlib.contextmanager
    def enter(s):
        at.append(s)
        yield
        at.pop()

    class Stream:
        def __init__(self, name):
            self.cuda_stream = 7
            self.name = name

    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(at[-1]) or real(*a, **k))
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: f"handle {ptr}")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream("current"))
    monkeypatch.setattr(ec, "lib", lambda: lib)
    monkeypatch.setattr(tw, "lib", lambda: lib)
    monkeypatch.setattr(ec, "_dev", lambda t, name: t.data_ptr())
    monkeypatch.setattr(ec, "_rows", lambda t, name: (t.data_ptr(), t.shape[0], t.stride(0)))
    monkeypatch.setattr(tw, "_mat", lambda t, name, shape, dtype: (None, shape[1]) if t is None else (t.data_ptr(), shape[1]))

    return made, lib, Stream


def device_like(t):
    """`t` as far as the bindings' own checks look at it."""
    class T(torch.Tensor):
        is_cuda = True
    return t.as_subclass(T)


B, F, Z = torch.bfloat16, torch.float32, torch.zeros
CALLS = {
    "dense_fwd": lambda **k: tw.dense_fwd(Z(4, 8, dtype=B), Z(8, 8, dtype=B), None, Z(4, 8, dtype=B), **k),
    "dense_bwd": lambda **k: tw.dense_bwd(Z(4, 8, dtype=B), Z(8, 8, dtype=B), Z(4, 8, dtype=B), Z(8, 8), **k),
    "group_norm_fwd": lambda **k: tw.group_norm_fwd(Z(4, 8), None, None, Z(4, 8), Z(2, 1), Z(2, 1), positions=2, groups=1, **k),
    "group_norm_bwd": lambda **k: tw.group_norm_bwd(Z(4, 8), Z(4, 8), None, None, Z(2, 1), Z(2, 1), Z(4, 8), None, None,
                                                    positions=2, groups=1, **k),
    "linear_bwd": lambda **k: ec.linear_bwd(Z(4, 8, dtype=B), Z(8, 8, dtype=B), Z(4, 8, dtype=B), Z(8, 8), Z(8), **k),
    "bce_logits": lambda **k: ec.bce_logits(device_like(Z(4, dtype=B)), Z(4), Z(1), device_like(Z(4, dtype=B)), **k),
}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_workspace_is_taken_on_the_calls_stream(streams, call):
    made, lib, Stream = streams
    side = Stream("side")
    for given, want in ((None, "current"), (side, side), (0x1234, "handle 4660"), (0, "default")):
        made.clear()
        CALLS[call](stream=given)
        assert made == [want], (given, made)
    # a workspace of the caller's is used as it is
    ws = Z(4096, dtype=torch.uint8)
    made.clear()
    CALLS[call](stream=side, workspace=ws)
    assert made == [] and len(lib.calls) == 5

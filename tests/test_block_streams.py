"""The block binding's streams and workspaces (CPU: the library is replaced by one that only counts
calls, streams by names): a workspace that the binding allocates belongs to the stream that the call
runs on, and a call runs with its operands' device current."""
import contextlib

import pytest
import torch

from embedding_lookup_feature_amd import block as bk
from embedding_lookup_feature_amd import embcore as ec

B, Z = torch.bfloat16, torch.zeros


class FakeLibrary:
    """Every size query answers 4096, every call succeeds and keeps the stream it was given."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return lambda *a: self.streams.append(a[-1]) or ec.EL_OK


@pytest.fixture
def fake(monkeypatch):
    at, made, lib, devices, current = ["current"], [], FakeLibrary(), [], [0]

    @contextlib.contextmanager
    def enter(s):
        at.append(s)
        yield
        at.pop()

    @contextlib.contextmanager
    def on_device(i):
        devices.append(i)
        yield

    class Stream:
        def __init__(self, name):
            self.cuda_stream, self.name = 7, name

    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(at[-1]) or real(*a, **k))
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: f"handle {ptr}")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(bk, "lib", lambda: lib)
    monkeypatch.setattr(bk, "_device", lambda t, name: -1)  # host tensors stand for device -1
    monkeypatch.setattr(bk, "_current_device", lambda: -1 + current[0])
    return made, lib, Stream, devices, current


def calls():
    nm = bk.BlockNorm(8)
    x8, w4 = bk.Checkpoint(4, 8, "cpu"), bk.Fp4(8, 8, "cpu")
    z = lambda: Z(4, 8, dtype=B)  # noqa: E731
    return {
        "block_norm_bwd": lambda **k: bk.block_norm_bwd(nm, z(), z(), dh=z(), pre_stats=Z(4, 2), **k),
        "dense_bwd_ckpt": lambda **k: bk.dense_bwd_ckpt(x8, Z(8, 8, dtype=B), z(), Z(8, 8), **k),
        "dense_fwd_fp4": lambda **k: bk.dense_fwd_fp4(z(), w4, None, z(), **k),
    }


@pytest.mark.parametrize("call", ["block_norm_bwd", "dense_bwd_ckpt", "dense_fwd_fp4"])
def test_workspace_is_taken_on_the_calls_stream(fake, call):
    made, lib, Stream, devices, current = fake
    run = calls()[call]
    side = Stream("side")
    for given, want in ((None, "current"), (side, side), (0x1234, "handle 4660"), (0, "default")):
        made.clear()
        run(stream=given)
        assert made == [want], (given, made)
    ws = Z(4096, dtype=torch.uint8)
    made.clear()
    run(stream=side, workspace=ws)
    assert made == [] and len(lib.streams) == 5 and devices == []


def test_a_call_runs_on_its_operands_device(fake):
    made, lib, Stream, devices, current = fake
    nm = bk.BlockNorm(8)
    bk.block_norm_fwd(nm, Z(4, 8), None, Z(4, 8))
    assert devices == [] and lib.streams == [99]  # the operands' device, its current stream
    current[0] = 3  # another device is current
    bk.block_norm_fwd(nm, Z(4, 8), None, Z(4, 8))
    assert devices == [-1] and lib.streams == [99, 99]

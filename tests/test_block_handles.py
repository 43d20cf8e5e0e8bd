"""The binding's handles follow the tensors they were made of (CPU: the library is replaced by one that
keeps what it was given): one whose storage was replaced is never read where it used to lie."""
import gc

import pytest
import torch

from embedding_lookup_feature_amd import block as bk
from embedding_lookup_feature_amd import embcore as ec


class KeepingLibrary:
    """Every size query answers 0, every call succeeds and keeps its arguments."""

    def __init__(self):
        self.args = None

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 0

        def call(*a):
            self.args = a
            return ec.EL_OK

        return call


@pytest.fixture
def lib(monkeypatch):
    L = KeepingLibrary()
    monkeypatch.setattr(bk, "lib", lambda: L)
    monkeypatch.setattr(bk, "_device", lambda t, name: t.get_device())  # host tensors stand for device -1
    monkeypatch.setattr(bk, "_current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    return L


def norm_call(lib, nm):
    bk.block_norm_fwd(nm, torch.zeros(4, 8), None, torch.zeros(4, 8))
    return lib.args[0]._obj


@pytest.mark.parametrize("name", bk.PARAMS)
def test_block_norm_follows_its_parameters(lib, name):
    t = torch.ones(8)
    nm = bk.BlockNorm(8, post="rms", **{name: t})
    assert getattr(norm_call(lib, nm), name) == t.data_ptr()
    first = lib.args[0]._obj
    old = t.data_ptr()
    t.data = torch.full((8,), 2.0)
    assert getattr(norm_call(lib, nm), name) == t.data_ptr() != old
    assert getattr(first, name) == old, "a structure that a call may still read is not changed"
    gc.collect()
    assert getattr(norm_call(lib, nm), name) == t.data_ptr()
    same = norm_call(lib, nm)
    assert same is norm_call(lib, nm)  # nothing is built again while nothing moves


@pytest.mark.parametrize("new", [torch.ones(7), torch.ones(9), torch.ones(8, dtype=torch.float64), torch.ones(8).half(),
                                 torch.ones(16)[::2], torch.ones(1).expand(8)], ids=str)
def test_block_norm_refuses_another_form_of_a_parameter(lib, new):
    t = torch.ones(8)
    nm = bk.BlockNorm(8, pre_gamma=t)
    norm_call(lib, nm)
    t.data = new
    lib.args = None
    for _ in range(2):
        with pytest.raises(ValueError, match="pre_gamma must hold 8 contiguous values"):
            norm_call(lib, nm)
    assert lib.args is None
    t.data = torch.ones(8)
    assert norm_call(lib, nm).pre_gamma == t.data_ptr()


@pytest.mark.parametrize("kind", ["Checkpoint", "Fp4"])
def test_packed_arrays_keep_their_memory(lib, kind):
    p = getattr(bk, kind)(4, 40, "cpu")
    pack = bk.ckpt_pack if kind == "Checkpoint" else bk.fp4_pack
    pack(torch.zeros(4, 40), p)
    first = lib.args[-3:-1]
    assert first == (p.codes.data_ptr(), p.scales.data_ptr())
    p.codes.fill_(7), p.scales.fill_(9)
    assert bool((p.codes == 7).all()) and bool((p.scales == 9).all()), "written in place"
    for name in ("codes", "scales"):
        v = getattr(p, name)
        v.data = torch.zeros(1, dtype=torch.uint8)  # other storage for the view
        w = getattr(p, name)
        w.set_(torch.zeros(1, dtype=torch.uint8))
        with pytest.raises(AttributeError):
            setattr(p, name, v)
    gc.collect()
    pack(torch.zeros(4, 40), p)
    assert lib.args[-3:-1] == first and bool((p.codes == 7).all()) and bool((p.scales == 9).all())
    assert p.nbytes == p.codes.numel() + p.scales.numel() > 100


@pytest.mark.parametrize("kind", ["Checkpoint", "Fp4"])
def test_packed_arrays_follow_storage_that_grew(lib, kind):
    p = getattr(bk, kind)(4, 40, "cpu")
    p.codes.fill_(7)
    grown = p.codes
    grown.resize_(1 << 20)  # the storage that the array shares moves
    (bk.ckpt_pack if kind == "Checkpoint" else bk.fp4_pack)(torch.zeros(4, 40), p)
    assert lib.args[-3] == grown.data_ptr() == p.codes.data_ptr() and bool((p.codes == 7).all())


def test_a_dropout_step_on_another_device_is_refused(lib):
    class Elsewhere:  # a tensor on device 1, beside host tensors that stand for device -1
        device = "cuda:1"

        def get_device(self):
            return 1

    d = bk.tw.Dropout(0.5, 1)
    ck, z = bk.Checkpoint(4, 8, "cpu"), torch.zeros(4, 8, dtype=torch.bfloat16)
    w, dw = torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(8, 8)
    calls = [lambda: bk.ckpt_act_dropout_fwd(ck, z, dropout=d), lambda: bk.ckpt_act_dropout_bwd(z, ck, z.clone(), dropout=d),
             lambda: bk.dense_bwd_ckpt(ck, w, z, dw, dx=z.clone(), dzb=z.clone(), dropout=d)]
    for call in calls:
        d.step, lib.args = None, None
        call()
        assert lib.args is not None
        d.step, lib.args = Elsewhere(), None
        with pytest.raises(ValueError, match="step must be on device -1, got cuda:1"):
            call()
        assert lib.args is None

"""The tower operators' entry points: exported, and bad arguments refused on the host before
anything reaches a GPU (no compute call is made here)."""
import ctypes

import pytest

from embedding_lookup_feature_amd import embcore as ec
from embedding_lookup_feature_amd import tower as tw

INVALID, UNSUPPORTED, WORKSPACE, OK = ec.EL_ERR_INVALID_ARG, ec.EL_ERR_UNSUPPORTED, ec.EL_ERR_WORKSPACE, ec.EL_OK
A = 0x7F0000000000  # fake, aligned: every call below ends at its checks
BIG = 1 << 40


def drop(p, step=0):
    return ctypes.byref(tw.ElDropout(p, 1, 2, step or None))


def test_library_exports_every_declared_function():
    L = tw.lib()
    names = tw.header_functions()
    assert set(names) == {"el_act_dropout_fwd", "el_act_dropout_bwd", "el_dense_fwd_workspace_bytes",
                          "el_dense_bwd_workspace_bytes", "el_dense_fwd", "el_dense_bwd",
                          "el_group_norm_fwd_workspace_bytes", "el_group_norm_bwd_workspace_bytes",
                          "el_group_norm_fwd", "el_group_norm_bwd"}
    for n in names:
        assert hasattr(L, n), n


ADF = dict(x=A, ldx=64, r=None, ldr=0, M=8, N=64, act=2, drop=None, y=A, ldy=64, dt=ec.EL_BF16)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=A + 1), INVALID), (dict(x=A + 2, dt=ec.EL_F32), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=63), INVALID), (dict(ldy=-64), INVALID), (dict(r=A, ldr=63), INVALID),
    (dict(r=A + 1, ldr=64), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(act=4), INVALID),
    (dict(dt=3), INVALID), (dict(dt=-5), INVALID), (dict(drop=drop(-0.1)), INVALID), (dict(drop=drop(1.5)), INVALID),
    (dict(drop=drop(float("nan"))), INVALID), (dict(drop=drop(0.5, A + 4)), INVALID), (dict(ldx=1 << 40), INVALID),
    (dict(M=2**31 - 1, N=64, ldx=64, ldy=64), UNSUPPORTED), (dict(M=0, x=None, y=None), OK),
])
def test_act_dropout_fwd_refusals(change, status):
    a = {**ADF, **change}
    rc = tw.lib().el_act_dropout_fwd(a["x"], a["ldx"], a["r"], a["ldr"], a["M"], a["N"], a["act"], a["drop"], a["y"],
                                     a["ldy"], a["dt"], None)
    assert rc == status
    if status != OK:
        assert "el_act_dropout_fwd" in ec.el_last_error()


@pytest.mark.parametrize("dy,x,dx,act,ld,status", [
    (None, A, A, 1, 64, INVALID), (A, None, A, 1, 64, INVALID), (A, A, None, 1, 64, INVALID), (A, A, A, 9, 64, INVALID),
    (A, A, A, 1, 8, INVALID), (A, A + 1, A, 1, 64, INVALID),
])
def test_act_dropout_bwd_refusals(dy, x, dx, act, ld, status):
    assert tw.lib().el_act_dropout_bwd(dy, ld, x, ld, 4, 64, act, None, dx, ld, ec.EL_F16, None) == status
    assert "el_act_dropout_bwd" in ec.el_last_error()


DF = dict(x=A, ldx=32, M=4, K=32, w=A, bias=A, N=16, act=1, drop=None, r=None, ldr=0, pre=None, ldp=0, y=A, ldy=16,
          dt=ec.EL_BF16, ws=A, wsn=BIG)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(bias=A + 2), INVALID),
    (dict(w=A + 1), INVALID), (dict(ldx=31), INVALID), (dict(ldy=15), INVALID), (dict(r=A, ldr=15), INVALID),
    (dict(pre=A, ldp=15), INVALID), (dict(pre=A + 1, ldp=16), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID),
    (dict(N=0), INVALID), (dict(act=4), INVALID), (dict(dt=ec.EL_F32), UNSUPPORTED), (dict(dt=77), INVALID),
    (dict(drop=drop(2.0)), INVALID), (dict(K=1 << 16, N=1 << 15, ldx=1 << 16, ldy=1 << 15), UNSUPPORTED),
    (dict(M=0, x=None, y=None), OK),
])
def test_dense_fwd_refusals(change, status):
    a = {**DF, **change}
    rc = tw.lib().el_dense_fwd(a["x"], a["ldx"], a["M"], a["K"], a["w"], a["bias"], a["N"], a["act"], a["drop"], a["r"],
                               a["ldr"], a["pre"], a["ldp"], a["y"], a["ldy"], a["dt"], a["ws"], a["wsn"], None)
    assert rc == status
    if status != OK:
        assert "el_dense_fwd" in ec.el_last_error()


DB = dict(x=A, ldx=32, M=4, K=32, w=A, N=16, dz=A, ldz=16, dres=None, ldr=0, dx=A, lddx=32, act=1, drop=None, pre=A,
          ldp=32, dzb=A, ldb=32, dw=A, db=A, dt=ec.EL_BF16, ws=A, wsn=BIG)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(dz=None), INVALID), (dict(dw=None), INVALID),
    (dict(pre=None), INVALID), (dict(dx=None), INVALID), (dict(dx=None, dzb=None, dres=A, ldr=32), INVALID),
    (dict(ldz=15), INVALID), (dict(lddx=31), INVALID), (dict(ldp=31), INVALID), (dict(ldb=31), INVALID),
    (dict(dres=A, ldr=31), INVALID), (dict(dw=A + 2), INVALID), (dict(db=A + 1), INVALID), (dict(act=5), INVALID),
    (dict(dt=ec.EL_F32), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(wsn=1), WORKSPACE),
    (dict(M=-2), INVALID), (dict(drop=drop(-1.0)), INVALID),
])
def test_dense_bwd_refusals(change, status):
    a = {**DB, **change}
    rc = tw.lib().el_dense_bwd(a["x"], a["ldx"], a["M"], a["K"], a["w"], a["N"], a["dz"], a["ldz"], a["dres"], a["ldr"],
                               a["dx"], a["lddx"], a["act"], a["drop"], a["pre"], a["ldp"], a["dzb"], a["ldb"], a["dw"],
                               a["db"], a["dt"], a["ws"], a["wsn"], None)
    assert rc == status
    assert "el_dense_bwd" in ec.el_last_error()


GN = dict(x=A, ldx=64, B=3, S=5, C=64, G=8, ln=None, gm=A, bt=A, eps=1e-5, act=3, y=A, ldy=64, mean=A, rstd=A,
          dt=ec.EL_F32, ws=A, wsn=BIG)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(G=0), INVALID), (dict(G=7), INVALID), (dict(C=0), INVALID), (dict(B=-1), INVALID), (dict(S=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(act=4), INVALID), (dict(dt=9), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(x=A + 2), INVALID), (dict(ln=A + 2), INVALID), (dict(gm=A + 1), INVALID), (dict(mean=A + 2), INVALID),
    (dict(B=1 << 22, G=64), UNSUPPORTED), (dict(S=100_000, ws=None), WORKSPACE), (dict(S=100_000, wsn=16), WORKSPACE),
    (dict(B=0, x=None, y=None, mean=None, rstd=None), OK),
])
def test_group_norm_fwd_refusals(change, status):
    a = {**GN, **change}
    rc = tw.lib().el_group_norm_fwd(a["x"], a["ldx"], a["B"], a["S"], a["C"], a["G"], a["ln"], a["gm"], a["bt"], a["eps"],
                                    a["act"], a["y"], a["ldy"], a["mean"], a["rstd"], a["dt"], a["ws"], a["wsn"], None)
    assert rc == status
    if status != OK:
        assert "el_group_norm_fwd" in ec.el_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(x=None), INVALID), (dict(mean=None), INVALID),
    (dict(lddy=63), INVALID), (dict(lddx=63), INVALID), (dict(dg=A + 2), INVALID), (dict(G=3), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsn=8), WORKSPACE),
])
def test_group_norm_bwd_refusals(change, status):
    a = {**dict(dy=A, lddy=64, x=A, ldx=64, B=3, S=5, C=64, G=8, mean=A, rstd=A, dx=A, lddx=64, dg=A, db=A, ws=A, wsn=BIG),
         **change}
    rc = tw.lib().el_group_norm_bwd(a["dy"], a["lddy"], a["x"], a["ldx"], a["B"], a["S"], a["C"], a["G"], None, None, None,
                                    a["mean"], a["rstd"], 2, a["dx"], a["lddx"], a["dg"], a["db"], ec.EL_BF16, a["ws"],
                                    a["wsn"], None)
    assert rc == status
    assert "el_group_norm_bwd" in ec.el_last_error()


def test_workspace_queries_are_host_pure_and_bounded():
    L = tw.lib()
    for fn in (tw.dense_fwd_workspace_bytes, tw.dense_bwd_workspace_bytes):
        assert fn(0, 8, 8) == 0 and fn(-1, 8, 8) == 0 and fn(8, 0, 8) == 0 and fn(8, 8, -3) == 0
        assert fn(2**31 - 1, 2**31 - 1, 2**31 - 1) == 0
    for fn in (tw.group_norm_fwd_workspace_bytes, tw.group_norm_bwd_workspace_bytes):
        assert fn(0, 1, 8, 1) == 0 and fn(1, 1, 8, 3) == 0 and fn(1, 1, 8, 0) == 0
        assert fn(2**31 - 1, 2**31 - 1, 2**31 - 1, 1) == 0
        assert fn(1, 2**31 - 1, 1 << 24, 1 << 24) >= 0
    # a long sample is cut into chunks; a short one stays in registers
    assert tw.group_norm_fwd_workspace_bytes(65536, 26, 128, 8) == 0
    assert tw.group_norm_fwd_workspace_bytes(2, 50_000, 256, 32) > 0
    assert tw.dense_bwd_workspace_bytes(65536, 1024, 1024) >= 4 * 1024 * 1024
    assert L is not None


def test_python_binding_refuses_mismatched_tensors():
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="act must be"):
        tw._act("tanh")
    with pytest.raises(ValueError, match="device tensor"):
        tw.act_dropout_fwd(x, x)
    with pytest.raises(ValueError, match="step"):
        tw.Dropout(0.1, 1, step=torch.zeros(2, dtype=torch.int64))

"""The gated tower step (the residual block's operators together, next to the embedding core): each
operator's outputs inside the model against its plain 64-bit form on the model's own buffers, with the
bounds of tests/block_plain.py, so that a wrong operand, mask or gradient on the way shows."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from embedding_lookup_feature_amd import gated, synth
from tests import block_plain as bp
from tests import tower_plain as tp
from tests.test_block_gpu import codes_of
from tests.test_tower_gpu import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
EPS = np.float64(np.float32(1e-5))


def build(batch, rows, **kw):
    wl = synth.WORKLOADS["train_step"].scaled(name=f"gated{batch}", batch=batch, rows=(rows,) * 26)
    W, ro = synth.make_tables(wl, DEV)
    idx, off = synth.make_indices(wl, DEV)
    tables, bags = elf.Tables(W, ro), elf.Bags(idx, off, batch)
    model = gated.GatedDLRMStep(wl, tables, DEV, **kw)
    return wl, tables, bags, model, synth.make_dense(wl, DEV, k_pad=model.k_pad), synth.make_labels(wl, DEV)


def kept(ckpt):
    return bp.values(*codes_of(ckpt, False), ckpt.cols, False)


def test_every_operator_in_the_step_matches_its_plain_form():
    p, seed, width, step, scale = 0.2, 99, 160, 7, 0.5
    wl, tables, bags, m, dense, labels = build(96, 40, width=width, blocks=1, p=p, seed=seed, scale=scale)
    B, F, D = wl.batch, wl.num_tables, wl.dim
    m.gammas.add_(0.2 * torch.randn(m.gammas.numel(), device=DEV, generator=torch.Generator(DEV).manual_seed(1)))
    m.step.fill_(step)
    m.forward(dense, bags)
    h_last, a_fwd, z = np64(m.h), np64(m.a), np64(m.z)
    # forward: gated pooled vectors, then the tower
    emb = np64(m.emb).reshape(B * F, D)
    gates = np64(m.gates)
    ry, ey, _, _ = tp.dense_fwd(np64(m.h_bot[-1]), np64(m.gate.w[0]), np64(m.gate.b[0]), "none", None, None, BF)
    tp.check(m.gates, (ry, ey), "gates")
    ref = bp.block_norm_fwd(None, emb, gates, "rms", "rms", np64(m.g_pool), None, None, None, "sigmoid", F, 1.0, EPS, BF)
    tp.check(m.vectors, ref["y"], "vectors")
    tp.check(m.pool_stats, ref["post_stats"], "pool_stats")
    ref = bp.block_norm_fwd(np64(m.s[0]), None, None, "none", "rms", None, None, np64(m.g_pre[0]), None, "none", 1, scale, EPS, BF)
    tp.check(m.pre_stats[0], ref["pre_stats"], "pre_stats0")
    h0 = torch.empty_like(m.h)
    elf.block_norm_fwd(m.seams[0], m.s[0], None, h0)
    tp.check(h0, ref["h"], "h0")
    h0 = np64(h0)
    assert (kept(m.h8[0]) == bp.rounded(h0, False)).all() and (kept(m.z8[0]) == bp.rounded(z, False)).all()
    mask = tp.drop_factors(B, width, p, seed, (1 << 48) + step)
    w1 = np64(m.top.w[1])
    ry, ey, rz, ez = tp.dense_fwd(h0, w1, np64(m.top.b[1]), "gelu", mask, None, BF)
    tp.check(m.a, (ry, ey), "a")
    tp.check(m.z, (rz, ez), "z")
    ref = bp.block_norm_fwd(np64(m.s[0]), a_fwd, None, "rms", "rms", np64(m.g_post[0]), None, np64(m.g_pre[1]), None, "none", 1,
                            scale, EPS, BF)
    for got, k in ((m.s[1], "y"), (m.h, "h"), (m.post_stats[0], "post_stats"), (m.pre_stats[1], "pre_stats")):
        tp.check(got, ref[k], k)
    # backward
    m.backward(dense, labels)
    zq = kept(m.z8[0])
    tp.check(m.a, tp.act_dropout_fwd(zq, "gelu", mask, None, BF), "a from 8 bits")
    dh = torch.empty_like(m.dh)
    elf.linear_bwd(torch.from_numpy(h_last).to(BF).to(DEV), m.top.w[-1], m.dlogit, torch.empty_like(m.top.dw[-1]), m.top.db[-1].clone(),
                   dx=dh, workspace=m.lin_ws)
    ref = bp.block_norm_bwd(None, np64(dh), np64(m.s[1]), np64(m.a), None, "rms", "rms", np64(m.g_post[0]), None,
                            np64(m.g_pre[1]), None, "none", 1, scale, np64(m.post_stats[0]), np64(m.pre_stats[1]), BF)
    for got, k in ((m.ds[0], "dx"), (m.da, "df"), (m.dg_post[0], "dpost_gamma"), (m.dg_pre[1], "dpre_gamma")):
        tp.check(got, ref[k], k)
    tp.check(m.dz, tp.act_dropout_bwd(np64(m.da), zq, "gelu", mask, BF), "dz")
    ref = tp.dense_bwd(kept(m.h8[0]), w1, np64(m.dz), None, None, "none", None, BF)
    for got, k in ((m.top.dw[1], "dw"), (m.top.db[1], "db"), (m.dh, "dx")):
        tp.check(got, ref[k], k)
    ref = bp.block_norm_bwd(np64(m.ds[0]), np64(m.dh), np64(m.s[0]), None, None, "none", "rms", None, None, np64(m.g_pre[0]),
                            None, "none", 1, scale, None, np64(m.pre_stats[0]), BF)
    tp.check(m.ds[1], ref["dx"], "ds0")
    tp.check(m.dg_pre[0], ref["dpre_gamma"], "dg_pre0")
    ref = tp.dense_bwd(np64(m.inter), np64(m.top.w[0]), np64(m.ds[1]), None, None, "none", None, BF)
    for got, k in ((m.top.dw[0], "dw"), (m.dout, "dx")):
        tp.check(got, ref[k], k)
    ref = bp.block_norm_bwd(np64(m.demb).reshape(B * F, D), None, None, emb, gates, "rms", "rms", np64(m.g_pool), None, None,
                            None, "sigmoid", F, 1.0, np64(m.pool_stats), None, BF)
    for got, k in ((m.dvec, "df"), (m.dgates, "dgate"), (m.dg_pool, "dpost_gamma")):
        tp.check(got, ref[k], k)
    ref = tp.dense_bwd(np64(m.h_bot[-1]), np64(m.gate.w[0]), np64(m.dgates), np64(m.dx0), None, "none", None, BF)
    for got, k in ((m.gate.dw[0], "dw"), (m.gate.db[0], "db"), (m.dx0_all, "dx")):
        tp.check(got, ref[k], k)


def test_serving_matches_its_plain_form():
    width = 96
    wl, tables, bags, m, dense, labels = build(77, 30, width=width, blocks=1, p=0.0)
    m.pack()
    logits = m.serve(dense, bags).clone()
    w = [bp.rounded(np64(v), True) for v in m.top.w_master[:-1]]
    x = bp.rounded(np64(m.inter), True)
    tp.check(m.s[0], bp.dense_fp4(x, w[0], np64(m.top.b[0]), "none", None, BF), "s0")
    h0 = torch.empty_like(m.h)
    elf.block_norm_fwd(m.seams[0], m.s[0], None, h0)
    tp.check(m.a, bp.dense_fp4(bp.rounded(np64(h0), True), w[1], np64(m.top.b[1]), "gelu", None, BF), "a")
    ref = bp.block_norm_fwd(np64(m.s[0]), np64(m.a), None, "rms", "rms", np64(m.g_post[0]), None, np64(m.g_pre[1]), None, "none",
                            1, 0.5, EPS, BF)
    tp.check(m.h, ref["h"], "h")
    assert torch.equal(logits, m.serve(dense, bags))


def test_steps_reproduce_and_move_every_parameter():
    runs = []
    for _ in range(2):
        wl, tables, bags, m, dense, labels = build(512, 200, width=256, blocks=3, p=0.1)
        before = [v.clone() for v in (m.bottom.master, m.gate.master, m.top.master, m.gammas)]
        ws = elf.alloc_workspace(tables, bags)
        run = []
        for _ in range(4):
            m.train_step(dense, bags, labels, ws)
            run.append(float(m.loss))
        assert int(m.step) == 4 and all(np.isfinite(run))
        assert all(not torch.equal(a, b) for a, b in zip(before, (m.bottom.master, m.gate.master, m.top.master, m.gammas)))
        runs.append(run)
    assert runs[0] == runs[1]


def test_the_command_runs(capsys):
    gated.main(["--steps", "2", "--batch", "300", "--rows", "50"])
    out = capsys.readouterr().out
    assert "step 0: loss" in out and "step 1: loss" in out and "served in 4 bits" in out

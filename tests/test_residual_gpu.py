"""The residual tower step (every tower operator together, next to the embedding core): each
operator's outputs inside the model against its plain 64-bit form on the model's own buffers, with
the bounds of tests/tower_plain.py, so that a wrong operand, mask or gradient on the way shows."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from embedding_lookup_feature_amd import residual, synth
from tests import tower_plain as tp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def build(batch, rows, **kw):
    wl = synth.WORKLOADS["train_step"].scaled(name=f"residual{batch}", batch=batch, rows=(rows,) * 26)
    W, ro = synth.make_tables(wl, DEV)
    idx, off = synth.make_indices(wl, DEV)
    tables, bags = elf.Tables(W, ro), elf.Bags(idx, off, batch)
    model = residual.ResidualDLRMStep(wl, tables, DEV, **kw)
    return wl, W, ro, idx, off, tables, bags, model, synth.make_dense(wl, DEV, k_pad=model.k_pad), synth.make_labels(wl, DEV)


def np64(t):
    return t.detach().double().cpu().numpy()


def test_every_operator_in_the_step_matches_its_plain_form():
    p, pf, seed, width, groups, step = 0.2, 0.1, 99, 128, 8, 7
    wl, W, ro, idx, off, tables, bags, m, dense, labels = build(96, 40, width=width, blocks=1, p=p, p_features=pf,
                                                                seed=seed, groups=groups)
    B, F, D, bf = wl.batch, wl.num_tables, wl.dim, torch.bfloat16
    m.gn.add_(0.2 * torch.randn(2 * D, device=DEV, generator=torch.Generator(DEV).manual_seed(1)))
    m.step.fill_(step)
    m.forward(dense, bags)
    m.backward(dense, labels)
    mask = lambda M, N, q, layer: tp.drop_factors(M, N, q, seed, (layer << 48) + step)  # noqa: E731
    emb, gm, bt = np64(m.emb).reshape(B * F, D), np64(m.gamma), np64(m.beta)
    # forward
    ry, ey, rm, rr = tp.gn_fwd(emb, F, groups, None, gm, bt, 1e-5, "none", bf)
    tp.check(m.normed, (ry, ey), "normed")
    tp.check(m.mean, rm, "mean")
    tp.check(m.rstd, rr, "rstd")
    ff = mask(B * F, D, pf, 0)
    tp.check(m.vectors, tp.act_dropout_fwd(np64(m.normed), "none", ff, None, bf), "vectors")
    x, masks = [np64(m.inter), np64(m.h_top[0])], [mask(B, width, p, 1), mask(B, width, p, 2)]
    for i in range(2):
        w, b = np64(m.top.w[i]), np64(m.top.b[i])
        ry, ey, rz, ez = tp.dense_fwd(x[i], w, b, "gelu", masks[i], x[i] if i else None, bf)
        tp.check(m.h_top[i], (ry, ey), f"h{i}")
        tp.check(m.pre[i], (rz, ez), f"pre{i}")
    # backward: dh[0], dz[0] belong to the block, dh[1], dz[1] to the first layer
    tp.check(m.dz[0], tp.act_dropout_bwd(np64(m.dh[0]), np64(m.pre[1]), "gelu", masks[1], bf), "dz1")
    ref = tp.dense_bwd(x[1], np64(m.top.w[1]), np64(m.dz[0]), np64(m.dh[0]), np64(m.pre[0]), "gelu", masks[0], bf)
    for name, got, key in (("dw1", m.top.dw[1], "dw"), ("db1", m.top.db[1], "db"), ("dh0", m.dh[1], "dx"), ("dz0", m.dz[1], "dzb")):
        tp.check(got, ref[key], name)
    ref = tp.dense_bwd(x[0], np64(m.top.w[0]), np64(m.dz[1]), None, None, "none", None, bf)
    for name, got, key in (("dw0", m.top.dw[0], "dw"), ("db0", m.top.db[0], "db"), ("dout", m.dout, "dx")):
        tp.check(got, ref[key], name)
    dx0, demb = torch.empty_like(m.dx0), torch.empty_like(m.demb)
    elf.dot_interact_bwd(m.h_bot[-1], m.vectors.view_as(m.emb), m.dout, dx0, demb)
    tp.check(m.dnormed, tp.act_dropout_bwd(np64(demb).reshape(B * F, D), None, "none", ff, bf), "dnormed")
    ref = tp.gn_bwd(np64(m.dnormed), emb, F, groups, None, gm, bt, np64(m.mean), np64(m.rstd), "none", bf)
    tp.check(m.demb, ref["dx"], "demb")
    tp.check(m.dgn[:D], ref["dgamma"], "dgamma")
    tp.check(m.dgn[D:], ref["dbeta"], "dbeta")


def test_steps_reduce_the_loss_and_reproduce():
    losses = []
    for _ in range(2):
        wl, W, ro, idx, off, tables, bags, m, dense, labels = build(512, 200, width=256, blocks=3, p=0.1)
        ws = elf.alloc_workspace(tables, bags)
        run = []
        for _ in range(12):
            m.train_step(dense, bags, labels, ws)
            run.append(float(m.loss))
        assert int(m.step) == 12
        logits = m.forward(dense, bags, train=False).clone()
        assert torch.equal(logits, m.forward(dense, bags, train=False))
        losses.append(run)
    assert losses[0] == losses[1]
    assert min(losses[0][-3:]) < losses[0][0]


def test_the_command_runs(capsys):
    residual.main(["--steps", "2", "--batch", "300", "--rows", "50"])
    out = capsys.readouterr().out
    assert "step 0: loss" in out and "step 1: loss" in out


@pytest.mark.parametrize("p", [0.0, 0.1])
def test_training_fits_a_batch(p):
    """80 steps at the demonstration's rate on one batch leave less than a tenth of the first loss
    (with p = 0 nothing in it is random), and the fitted model separates the labels."""
    wl, W, ro, idx, off, tables, bags, m, dense, labels = build(512, 200, width=256, blocks=3, p=p, p_features=p / 2)
    m.wl = wl.scaled(name="fit", lr=0.001)
    ws = elf.alloc_workspace(tables, bags)
    m.train_step(dense, bags, labels, ws)
    first = float(m.loss)
    for _ in range(79):
        m.train_step(dense, bags, labels, ws)
    assert float(m.loss) < first / 10
    right = (m.forward(dense, bags, train=False)[:, 0].float() > 0) == (labels > 0.5)
    assert float(right.float().mean()) > 0.95

"""The plain 64-bit forms of the residual block's operators against differences and the formats'
definitions (CPU): what the GPU tests hold the kernels to."""
import numpy as np
import pytest
import torch

from tests import block_plain as bp


def test_format_numbers():
    assert bp.E4M3[-1] == 448 and bp.E4M3[1] == 2.0**-9 and bp.E4M3[8] == 2.0**-6
    assert list(bp.E2M1) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (t == bp.E4M3).all()


@pytest.mark.parametrize("fp4", [False, True])
def test_pack_picks_the_nearest_number(fp4):
    r = np.random.default_rng(1)
    x = r.normal(size=(40, 70)) * 2.0 ** r.integers(-140, 120, size=(40, 1))
    x[3, :32] = 0
    code, byte = bp.pack(x, fp4)
    v = bp.values(code, byte, 70, fp4)
    top = 6.0 if fp4 else 448.0
    table = bp.E2M1 if fp4 else bp.E4M3
    for i in range(0, 40, 7):
        for j in range(70):
            s = 2.0 ** (int(byte[i, j // 32]) - 127)
            best = min(abs(abs(x[i, j]) - t * s) for t in table)
            assert abs(v[i, j] - x[i, j]) == best
            blk = np.abs(x[i, j // 32 * 32:j // 32 * 32 + 32]).max()
            assert blk <= top * s and (byte[i, j // 32] == 1 or blk > top * s / 2)
    assert (np.signbit(v) == np.signbit(x)).all()


def test_pack_special_values():
    x = np.ones((2, 64))
    x[0, 5], x[0, 6], x[1, 40] = np.nan, np.inf, -np.inf
    c8, b8 = bp.pack(x, False)
    v = bp.values(c8, b8, 64, False)
    assert np.isnan(v[0, [5, 6]]).all() and np.isnan(v[1, 40]) and np.isnan(v).sum() == 3
    v = bp.rounded(x, True)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 32:]).all() and np.isnan(v).sum() == 64


def test_torch_rounds_e4m3_the_same_way():
    x = np.random.default_rng(2).normal(size=(64, 32)).astype(np.float32)
    x[:, 0] = 448.0  # scale 1
    code, byte = bp.pack(x.astype(np.float64), False)
    x[:, 1:] = np.clip(x[:, 1:] * 64, -448, 448)
    code, byte = bp.pack(x.astype(np.float64), False)
    assert (byte == 127).all()
    assert (torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy() == code).all()


def _diff(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("act,rows", [("none", 1), ("sigmoid", 3), ("sigmoid", 100), (None, 2)])
def test_block_norm_gradients_match_differences(post, pre, act, rows):
    r = np.random.default_rng(5)
    M, C, scale, eps = 8, 11, 0.7, 1e-3
    R = -(-M // rows)
    v = dict(x=r.normal(size=(M, C)), f=r.normal(size=(M, C)), gate=r.normal(size=(R, C)) if act else None,
             gp=1 + r.normal(size=C), bp=r.normal(size=C), gq=1 + r.normal(size=C), bq=r.normal(size=C))
    cy, ch = r.normal(size=(M, C)), r.normal(size=(M, C))

    def loss(**k):
        w = {**v, **k}
        o = bp.block_norm_fwd(w["x"], w["f"], w["gate"], post, pre, w["gp"], w["bp"], w["gq"], w["bq"], act or "none", rows,
                              scale, eps, torch.float32)
        return float((o["y"][0] * cy).sum() + (o["h"][0] * ch).sum())

    o = bp.block_norm_fwd(v["x"], v["f"], v["gate"], post, pre, v["gp"], v["bp"], v["gq"], v["bq"], act or "none", rows,
                          scale, eps, torch.float32)
    ps = o["post_stats"][0] if post != "none" else None
    g = bp.block_norm_bwd(cy, ch, o["y"][0], v["f"], v["gate"], post, pre, v["gp"], v["bp"], v["gq"], v["bq"], act or "none",
                          rows, scale, ps, o["pre_stats"][0], torch.float32)
    names = dict(x="dx", f="df", gate="dgate", gp="dpost_gamma", bp="dpost_beta", gq="dpre_gamma", bq="dpre_beta")
    for k, n in names.items():
        if v[k] is None:
            continue
        d = r.normal(size=v[k].shape)
        grad = (g[n][0] * d).sum()
        assert abs(_diff(lambda a: loss(**{k: a}), v[k], d) - grad) < 1e-6 * (1 + np.abs(g[n][0] * d).sum()), n

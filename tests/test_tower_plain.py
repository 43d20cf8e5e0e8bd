"""The plain 64-bit forms of the tower operators against published vectors and differences
(CPU): what the GPU tests hold the kernels to."""
import numpy as np
import pytest

from tests import tower_plain as tp


@pytest.mark.parametrize("ctr,key,out", [
    # known answers published with the generator (philox4x32, 10 rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(ctr, key, out):
    got = tp.philox4x32_10([np.array([c], np.uint64) for c in ctr], key)
    assert tuple(int(v[0]) for v in got) == out


def test_drop_factors_keep_the_mean():
    for p in (0.1, 0.5, 0.9):
        f = tp.drop_factors(400, 501, p, 0x123456789ABC, 7)
        kept = np.mean(f > 0)
        assert abs(kept - (1 - p)) < 5 * np.sqrt(p * (1 - p) / f.size) + 2.0**-17
    assert (tp.drop_factors(5, 9, 0.0, 1, 1) == 1).all() and (tp.drop_factors(5, 9, 1.0, 1, 1) == 0).all()


def _diff(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_gradients_match_differences(kind):
    r = np.random.default_rng(3)
    M, K, N = 7, 5, 11
    x, w, b, res = r.normal(size=(M, K)), r.normal(size=(N, K)), r.normal(size=N), r.normal(size=(M, N))
    f, co = tp.drop_factors(M, N, 0.3, 5, 6), r.normal(size=(M, N))
    import torch
    fwd = lambda x, w, b: float((tp.dense_fwd(x, w, b, kind, f, res, torch.float32)[0] * co).sum())  # noqa: E731
    z = tp.dense_fwd(x, w, b, kind, f, res, torch.float32)[2]
    dz = tp.act_dropout_bwd(co, z, kind, f, torch.float32)[0]
    g = tp.dense_bwd(x, w, dz, None, None, "none", None, torch.float32)
    for grad, at, fn in ((g["dx"][0], x, lambda v: fwd(v, w, b)), (g["dw"][0], w, lambda v: fwd(x, v, b)),
                         (g["db"][0], b, lambda v: fwd(x, w, v))):
        d = r.normal(size=at.shape)
        assert abs(_diff(fn, at, d) - (grad * d).sum()) < 1e-6 * (1 + np.abs(grad * d).sum())


@pytest.mark.parametrize("kind", ["none", "gelu", "silu", "relu"])
@pytest.mark.parametrize("lengths", [None, [0, 3, 4]])
def test_group_norm_gradients_match_differences(kind, lengths):
    import torch
    r = np.random.default_rng(4)
    B, S, C, G = 3, 4, 6, 2
    ln = None if lengths is None else np.array(lengths)
    x, gm, bt, co = r.normal(size=(B * S, C)), 1 + r.normal(size=C), r.normal(size=C), r.normal(size=(B * S, C))
    fwd = lambda x, gm, bt: float((tp.gn_fwd(x, S, G, ln, gm, bt, 1e-5, kind, torch.float32)[0] * co).sum())  # noqa: E731
    mean, rstd, _, _ = tp.gn_stats(x, S, G, ln, 1e-5)
    g = tp.gn_bwd(co, x, S, G, ln, gm, bt, mean, rstd, kind, torch.float32)
    for grad, at, fn in ((g["dx"][0], x, lambda v: fwd(v, gm, bt)), (g["dgamma"][0], gm, lambda v: fwd(x, v, bt)),
                         (g["dbeta"][0], bt, lambda v: fwd(x, gm, v))):
        d = r.normal(size=at.shape)
        assert abs(_diff(fn, at, d) - (grad * d).sum()) < 1e-6 * (1 + np.abs(grad * d).sum())

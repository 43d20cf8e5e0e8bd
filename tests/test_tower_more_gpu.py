"""More sizes of the tower operators on the GPU, against the plain 64-bit forms and bounds of
tests/tower_plain.py: the kernel forms and loops that tests/test_tower_gpu.py's sizes do not reach."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from tests import test_tower_gpu as base

pytestmark = pytest.mark.gpu
DEV = "cuda"

# more samples than 512 workgroups' worth: one workgroup has a sample's statistics
WHOLE = [
    # B, S, C, G, ld, dtype, act, lengths, affine
    (300, 40, 520, 8, 520, "bf16", "silu", "mixed", True),   # groups across vectors
    (260, 9, 1888, 32, 1888, "bf16", "gelu", None, True),    # wide: one row of threads
    (260, 70, 257, 1, 259, "f32", "silu", "mixed", True),    # odd rows, one group
    (257, 45, 400, 40, 400, "f16", "gelu", "mixed", False),  # groups of 10 channels
    (258, 200, 128, 128, 128, "f32", "none", "mixed", True),  # one channel per group
    (520, 30, 2048, 1, 2048, "f16", "none", "zero", True),
]


@pytest.mark.parametrize("case", WHOLE, ids=lambda c: "-".join(map(str, c)))
def test_group_norm_whole_samples(case):
    base.test_group_norm(case)


def test_dense_bwd_of_the_longest_batch():
    """2^31 - 1 rows: the last slice of the reduction ends where a 32-bit sum would have passed 2^31,
    and no row behind the last is read.  A few rows count, the others are zeros."""
    M, K, N = 2**31 - 1, 8, 8
    x = torch.zeros((M + 1, K), dtype=torch.bfloat16, device=DEV)
    dz = torch.zeros((M + 1, N), dtype=torch.bfloat16, device=DEV)
    at = [0, 1, 63, 2**23 - 1, 2**23, 2**30, 2**31 - 2**23 - 1, 2**31 - 2**23, M - 64, M - 1]
    rng = np.random.default_rng(0)
    xs, zs = rng.integers(-8, 9, (len(at), K)), rng.integers(-8, 9, (len(at), N))
    x[at], dz[at] = (torch.from_numpy(v).to(torch.bfloat16).to(DEV) for v in (xs, zs))
    x[M], dz[M] = float("nan"), float("nan")  # behind the last row
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    elf.dense_bwd(x[:M], w=torch.ones(N, K, dtype=torch.bfloat16, device=DEV), dz=dz[:M], dw=dw, db=db, workspace=ws)
    assert (dw.cpu().numpy() == zs.T @ xs).all() and (db.cpu().numpy() == zs.sum(0)).all()

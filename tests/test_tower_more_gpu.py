"""More sizes of the tower operators on the GPU, against the plain 64-bit forms and bounds of
tests/tower_plain.py: the kernel forms and loops that tests/test_tower_gpu.py's sizes do not reach."""
import pytest

from tests import test_tower_gpu as base

pytestmark = pytest.mark.gpu

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

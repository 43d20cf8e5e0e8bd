"""More of the residual block's operators on the GPU: the largest batches, and sums that have to be exact."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from tests.test_tower_gpu import DEV, DT

pytestmark = pytest.mark.gpu


def test_block_norm_shared_gates_of_more_than_2_to_the_30_rows():
    """M + gate_rows passes 2^31; two gate rows, the second of one row.  Small whole numbers: exact."""
    M, C = (1 << 30) + 3, 1
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dy, f, df, gate, dgate = z(M, C), z(M, C), z(M, C), z(2, C), z(2, C)
    f.fill_(1.0)
    dy[::65537] = 1.0
    dy[-1] = 4.0
    gate[0], gate[1] = 2.0, 3.0
    ones = -(-M // 65537)  # rows of dy that hold 1 (the last is not one of them)
    assert (M - 1) % 65537 != 0
    nm = elf.BlockNorm(C, post="none", pre="rms", gate_rows=M - 1)
    dgamma, dbeta = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    elf.block_norm_bwd(nm, None, None, dy=dy, f=f, gate=gate, df=df, dgate=dgate, dpost_gamma=dgamma, dpost_beta=dbeta)
    assert dgamma.item() == dbeta.item() == 2 * ones + 12
    assert torch.equal(dgate.cpu(), torch.tensor([[float(ones)], [4.0]]).bfloat16())
    assert bool((df[:-1] == 2 * dy[:-1]).all()) and df[-1].item() == 12.0

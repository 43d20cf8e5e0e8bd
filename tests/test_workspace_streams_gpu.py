"""Calls on another stream without a workspace of the caller's (GPU): what the current stream
allocates and fills right after the call is not the memory that the call still works in."""
import pytest
import torch

import embedding_lookup_feature_amd as elf

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(*s, dt=torch.bfloat16):
    return torch.randn(*s, device=DEV, generator=torch.Generator(DEV).manual_seed(sum(s))).to(dt)


def dense_fwd(stream):
    x, w, y = randn(4099, 479), randn(1001, 479), torch.empty(4099, 1001, dtype=torch.bfloat16, device=DEV)  # copied operands
    return (lambda: elf.dense_fwd(x, w, None, y, act="silu", stream=stream)), [y], elf.dense_fwd_workspace_bytes(4099, 479, 1001)


def dense_bwd(stream):
    M, K, N = 5000, 250, 264
    x, w, dz, dx = randn(M, K), randn(N, K), randn(M, N), torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    return (lambda: elf.dense_bwd(x, w, dz, dw, db, dx=dx, stream=stream)), [dx, dw, db], elf.dense_bwd_workspace_bytes(M, K, N)


def linear_bwd(stream):
    M, K, N = 5000, 256, 264
    x, w, dz, dx = randn(M, K), randn(N, K), randn(M, N), torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    return (lambda: elf.linear_bwd(x, w, dz, dw, db, dx=dx, stream=stream)), [dx, dw, db], elf.linear_bwd_workspace_bytes(M, K, N)


def group_norm(stream):
    B, S, C, G = 2, 5000, 64, 8
    x, dy = randn(B * S, C), randn(B * S, C).flip(0).contiguous()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    st, dp = [torch.empty(B, G, device=DEV) for _ in range(2)], [torch.empty(C, device=DEV) for _ in range(2)]

    def call():
        elf.group_norm_fwd(x, None, None, y, *st, positions=S, groups=G, act="silu", stream=stream)
        elf.group_norm_bwd(dy, x, None, None, *st, dx, *dp, positions=S, groups=G, act="silu", stream=stream)

    return call, [y, dx, *st, *dp], elf.group_norm_fwd_workspace_bytes(B, S, C, G)


@pytest.mark.parametrize("make", [dense_fwd, dense_bwd, linear_bwd, group_norm], ids=lambda f: f.__name__)
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_current_streams_allocations_do_not_reach_the_workspace(make, handle):
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    call, outs, need = make(None)
    assert need > 0, "the case needs a workspace"
    call()
    want = [t.clone() for t in outs]
    call, outs, need = make(given)
    filler = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # work of some milliseconds in front of the call
        for _ in range(40):
            filler.fill_(1)
    call()
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255) for n in (need, need, need // 2 + 512)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    assert all(bool((t == 255).all()) for t in junk)

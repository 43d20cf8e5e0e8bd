"""What the tower operators' size queries promise over whole ranges of sizes (CPU: the queries are
host-pure, no compute call is made here)."""
import random

import pytest

from embedding_lookup_feature_amd import tower as tw

MIB = 1 << 20


def test_group_norm_forward_workspace_is_bounded():
    """At most 8 MiB for up to 2048 channels, whatever the batch and the positions."""
    r = random.Random(7)
    shapes = [(1492, 9, 1888, 32), (1182, 11, 1696, 32), (704, 10, 1824, 32)]
    for _ in range(60_000):
        C = max(1, round(2 ** r.uniform(0, 11)))
        G = r.choice([g for g in (1, 2, 3, 4, 8, 16, 32, C) if C % g == 0])
        shapes.append((round(2 ** r.uniform(0, 18)), round(2 ** r.uniform(0, 14)), C, G))
    for s in shapes:
        assert tw.group_norm_fwd_workspace_bytes(*s) <= 8 * MIB, s


def test_workspaces_of_the_measured_range_fit_a_programs_buffers():
    """The buffers that perf/operators.py gives its calls hold for every size that it draws."""
    op = pytest.importorskip("perf.operators")
    give = {"group_norm_fwd": 8 * MIB, "group_norm_train": 64 * MIB, "dense_fwd": 160 * MIB, "dense_bwd": 512 * MIB}
    r = random.Random(11)
    for _ in range(60_000):
        c = op.draw(r)
        if c["op"].startswith("group_norm"):
            a = (c["M"], c["S"], c["C"], c["G"])
            need = tw.group_norm_fwd_workspace_bytes(*a)
            if c["op"] == "group_norm_train":
                need = max(need, tw.group_norm_bwd_workspace_bytes(*a))
        elif c["op"].startswith("dense"):
            a = (c["M"], c["K"], c["N"])
            need = (tw.dense_fwd_workspace_bytes if c["op"] == "dense_fwd" else tw.dense_bwd_workspace_bytes)(*a)
        else:
            continue
        assert need <= give[c["op"]], (c["op"], a, need)

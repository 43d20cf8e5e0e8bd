"""Tables, bags and dropout steps follow their tensors (CPU: host tensors stand for device ones, no call is made): one
whose storage was replaced is never read where it used to lie."""
import pytest
import torch

from embedding_lookup_feature_amd import embcore as ec
from embedding_lookup_feature_amd import tower as tw


@pytest.fixture(autouse=True)
def host(monkeypatch):
    def dev(t, name):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    monkeypatch.setattr(ec, "_dev", dev)


def tables():
    w, ro = torch.zeros(10, 8), torch.tensor([0, 4, 10])
    return w, ro, ec.Tables(w, ro)


def bags():
    i, o = torch.zeros(6, dtype=torch.int32), torch.arange(7, dtype=torch.int32)
    return i, o, ec.Bags(i, o, 3)


def test_tables_follow_their_tensors():
    w, ro, t = tables()
    first = t.c
    assert (first.base, first.row_offset, first.total_rows, first.num_tables, first.dim, first.max_rows) == \
        (w.data_ptr(), ro.data_ptr(), 10, 2, 8, 6)
    assert t.c is first and (t.num_tables, t.dim) == (2, 8)
    old = w.data_ptr()
    w.data = torch.ones(10, 8)
    assert t.c.base == w.data_ptr() != old and first.base == old, "a structure that a call may still read is not changed"
    ro.data = ro.data.clone()
    c = t.c
    assert (c.base, c.row_offset, c.total_rows, c.num_tables, c.dim, c.dtype, c.max_rows) == \
        (w.data_ptr(), ro.data_ptr(), 10, 2, 8, ec.EL_F32, 6)


def test_bags_follow_their_tensors():
    i, o, b = bags()
    assert (b.c.indices, b.c.offsets, b.c.batch, b.c.nnz) == (i.data_ptr(), o.data_ptr(), 3, 6)
    i.data, o.data = i.data.clone(), o.data.clone()
    assert (b.c.indices, b.c.offsets, b.c.batch, b.c.nnz) == (i.data_ptr(), o.data_ptr(), 3, 6)
    e = ec.Bags(torch.zeros(0, dtype=torch.int32), o, 3)
    assert not e.c.indices and e.c.nnz == 0


@pytest.mark.parametrize("new", [torch.zeros(9, 8), torch.zeros(11, 8), torch.zeros(8, 10), torch.zeros(10, 8).half(),
                                 torch.zeros(10, 16)[:, :8], torch.zeros(80)], ids=lambda t: f"{list(t.shape)} {t.dtype} {t.stride()}")
def test_another_form_is_refused(new):
    w, ro, t = tables()
    w.data = new
    for _ in range(2):
        with pytest.raises(ValueError, match="weight must"):
            t.c
    w.data = torch.zeros(10, 8)
    assert t.c.base == w.data_ptr()


def test_fewer_indices_are_refused():
    i, o, b = bags()
    i.data = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="indices must stay \\[6\\]"):
        b.c


def test_dropout_follows_its_step():
    step = torch.zeros(1, dtype=torch.int64)
    d = tw.Dropout(0.25, 7, 9, step)
    first = d.c
    assert (first.p, first.seed, first.offset, first.step) == (0.25, 7, 9, step.data_ptr()) and d.c is first
    step += 1
    assert d.c is first
    step.data = torch.zeros(1, dtype=torch.int64)
    assert (d.c.p, d.c.seed, d.c.offset, d.c.step) == (0.25, 7, 9, step.data_ptr()) and d.c.step != first.step
    step.data = torch.zeros(1)
    with pytest.raises(ValueError, match="step must stay"):
        d.c
    none = tw.Dropout(0.25, 7)
    assert none.c is none.c and not none.c.step


def test_tables_read_the_largest_table_again_where_row_offset_moved():
    w, ro, t = tables()
    assert t.c.max_rows == t.max_rows == 6
    w.data = torch.ones(10, 8)
    assert t.c.max_rows == 6
    ro.data = torch.tensor([0, 1, 10])
    assert t.c.max_rows == t.max_rows == 9
    given = ec.Tables(w, ro, max_rows=10)
    ro.data = torch.tensor([0, 5, 10])
    assert given.c.max_rows == given.max_rows == 10 and t.c.max_rows == 5

"""The paged batch's own bookkeeping, on a stand-in for the handle (no GPU)."""
import pytest

torch = pytest.importorskip("torch")


class Handle:
    _dev = "cpu"

    def __init__(self):
        self.planned = []

    def paged_plan(self, cu_q, k_lens, table, q_tokens, kv_heads, page_tokens, n_pages, mask_block, cu_groups=None, shared=None):
        self.note(cu_q, k_lens, table, cu_groups, shared)
        return self

    def paged_replan(self, plan, cu_q, k_lens, table, cu_groups=None, shared=None):
        self.note(cu_q, k_lens, table, cu_groups, shared)

    def note(self, *x):
        assert all(y is None or y.dtype == torch.int32 for y in x)
        self.planned.append([None if y is None else y.tolist() for y in x])


def batch(**kw):
    from video_dit_long_gb300.packed import PagedBatch
    h = Handle()
    return h, PagedBatch(h, [1, 2], [10, 20], [[0, 1], [2, 3]], 8, 2, 16, 4, 1, **kw)


def test_steps():
    h, b = batch(groups=[(2, 9)])
    b.next([1, 1], [11, 21])
    b.next(lens=torch.tensor([0, 4, 4], dtype=torch.int32))
    b.next(k_lens=torch.tensor([5, 6]), table=[[3, 2], [1, 0]], shared=[4])
    assert h.planned == [[[0, 1, 3], [10, 20], [[0, 1], [2, 3]], [0, 2], [9]],
                         [[0, 1, 2], [11, 21], [[0, 1], [2, 3]], [0, 2], [9]],
                         [[0, 4, 4], [11, 21], [[0, 1], [2, 3]], [0, 2], [9]],
                         [[0, 4, 4], [5, 6], [[3, 2], [1, 0]], [0, 2], [4]]]


def test_the_batch_has_tensors_of_its_own():
    from video_dit_long_gb300.packed import PagedBatch
    mine = [torch.tensor(x, dtype=torch.int32) for x in ([0, 1, 3], [10, 20], [[0, 1], [2, 3]])]
    b = PagedBatch(Handle(), *mine, 8, 2, 16, 4, 1)
    b.next([5, 5], [30, 40], [[9, 9], [9, 9]])
    assert [x.tolist() for x in mine] == [[0, 1, 3], [10, 20], [[0, 1], [2, 3]]]


@pytest.mark.parametrize("kw", [dict(lens=[1]), dict(lens=[1, 2, 3]), dict(k_lens=5), dict(k_lens=[1.0, 2.0]), dict(k_lens=[[1, 2]]),
                                dict(table=[[0], [1]]), dict(table=[0, 1]), dict(shared=[3])])
def test_what_would_broadcast_or_does_not_fit_is_refused(kw):
    """And nothing of the same call is taken over."""
    h, b = batch()
    with pytest.raises(ValueError):
        b.next(**{"k_lens": [7, 8], **kw})
    assert len(h.planned) == 1 and b.k_lens.tolist() == [10, 20]

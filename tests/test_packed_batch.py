"""The packed batch's own bookkeeping, on a stand-in for the handle (no GPU)."""
import pytest

torch = pytest.importorskip("torch")


class Handle:
    _dev = "cpu"

    def __init__(self):
        self.planned = []

    def packed_plan(self, cu_q, cu_k, q_tokens, k_tokens, kv_heads, mask_block):
        self.planned.append(cu_q.tolist())
        return self

    def packed_replan(self, plan, cu_q, cu_k):
        self.planned.append(cu_q.tolist())


def batch(lens):
    from video_dit_long_gb300.packed import PackedBatch
    h = Handle()
    return h, PackedBatch(h, lens, 100, 2, 1)


def test_other_lengths_as_offsets_or_as_a_list():
    h, b = batch([10, 20, 30])
    b.set_offsets(torch.tensor([0, 5, 5, 60], dtype=torch.int32))
    b.set_offsets(torch.tensor([1, 2, 3, 4]))
    b.set_offsets([7, 0, 8])
    assert h.planned == [[0, 10, 30, 60], [0, 5, 5, 60], [1, 2, 3, 4], [0, 7, 7, 15]]


@pytest.mark.parametrize("offsets", [torch.tensor(5, dtype=torch.int32), torch.tensor([5], dtype=torch.int32),
                                     torch.tensor([0, 5, 60], dtype=torch.int32), torch.tensor([[0, 5, 6, 60]]),
                                     torch.tensor([0.0, 5.0, 6.0, 60.0]), [7, 8], [1, 2, 3, 4]])
def test_offsets_that_would_broadcast_or_do_not_fit_are_refused(offsets):
    """One number would fill every offset and plan a batch of empty sequences."""
    h, b = batch([10, 20, 30])
    with pytest.raises(ValueError):
        b.set_offsets(offsets)
    assert h.planned == [[0, 10, 30, 60]] and b.offsets.tolist() == [0, 10, 30, 60]

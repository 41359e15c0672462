"""Numbers that a batch's int32 tensors cannot hold are refused, not cut off (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from .test_paged_batch import Handle, batch  # noqa: E402

GOOD = dict(lens=[1, 2], k_lens=[10, 20], table=[[0, 1], [2, 3]])
BAD = [dict(lens=[1, 2.5]), dict(lens=torch.tensor([0.0, 1.0, 3.0])), dict(lens=[1, 2 ** 32 + 1]), dict(k_lens=[10.5, 20]),
       dict(k_lens=torch.tensor([10.0, 20.0])), dict(k_lens=[10, 2 ** 32 + 20]), dict(k_lens=[10, -2 ** 31 - 1]),
       dict(table=[[0.0, 1], [2, 3]]), dict(table=[[0, 1], [2, 2 ** 32 + 3]])]


@pytest.mark.parametrize("kw", BAD + [dict(groups=[(1, 8.5)]), dict(groups=[(1.5, 8)]), dict(groups=[(1, 2 ** 32 + 8)])])
def test_at_the_start(kw):
    from video_dit_long_gb300.packed import PagedBatch
    h = Handle()
    with pytest.raises(ValueError):
        PagedBatch(h, **{**GOOD, **kw}, tokens=8, kv_heads=2, page_tokens=16, n_pages=4)
    assert not h.planned


@pytest.mark.parametrize("kw", BAD + [dict(shared=[8.5]), dict(shared=[2 ** 32])])
def test_at_the_next_step(kw):
    """And nothing of the same call is taken over."""
    h, b = batch(groups=[(2, 9)])
    with pytest.raises(ValueError):
        b.next(**{"k_lens": [7, 8], **kw})
    assert len(h.planned) == 1 and b.k_lens.tolist() == [10, 20]


def test_the_largest_that_fit():
    h, b = batch()
    b.next([0, 2 ** 31 - 1], torch.tensor([2 ** 31 - 1, -2 ** 31]), [[2 ** 31 - 1, -1], [-2 ** 31, 0]])
    assert h.planned[1] == [[0, 0, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31], [[2 ** 31 - 1, -1], [-2 ** 31, 0]], None, None]


@pytest.mark.parametrize("lens", [[1, 2.5], [1, 2 ** 32]])
def test_lengths_of_packed_sequences(lens):
    from video_dit_long_gb300.packed import PackedBatch
    with pytest.raises(ValueError):
        PackedBatch._offsets(lens)
    assert PackedBatch._offsets([1, 0, 4]).tolist() == [0, 1, 1, 5] and PackedBatch._offsets([]).tolist() == [0]

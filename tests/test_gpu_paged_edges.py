"""Calls over pages at the borders of what they take: lengths that are none, plans of other calls, shared prefixes over
every kind of copy, calls of different data at once."""
import pytest

from .test_gpu_paged_attention import Step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("Lk", [-1, -2 ** 31, -2 ** 31 + 1, -2 ** 31 + 89, 2 ** 31 - 1])
def test_a_length_that_is_none_gives_no_token_a_place(Lk):
    """Lengths so far below zero that their difference from the new tokens leaves an int included."""
    b = Step([90, 200], [90, 200], 4, 2, 1, seed=13)
    bad = torch.tensor([Lk, 200], dtype=torch.int32, device="cuda")
    T = b.q.shape[0]
    b.plan.buffer.zero_()
    b.h.paged_replan(b.plan, b.cu_q, bad, b.table)
    b.forward()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_INVALID_ARG
    assert bool((b.out == 7.0).all()) and bool((b.lse == 7.0).all())
    slot = b.plan.buffer[-4 * T:].view(torch.int32)  # the last part of a plan: each row's place in the pool
    assert bool((slot[:b.pad + 90] == -1).all()) and bool((slot[b.pad + 290:] == -1).all())
    i = torch.arange(200, device="cuda")
    assert torch.equal(slot[b.pad + 90:b.pad + 290], b.table[1, i // b.page] * b.page + (i % b.page).int())
    b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table)
    b.forward().check()

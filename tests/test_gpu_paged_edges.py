"""Calls over pages at the borders of what they take: lengths that are none, plans of other calls, shared prefixes over
every kind of copy, calls of different data at once."""
import pytest

from .test_gpu_paged_attention import Step
from .test_gpu_paged_layer import EPS, Streams, pages_for

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


@pytest.mark.parametrize("by_head,qk", [(False, "f16"), (True, "bf16")])
def test_a_layer_goes_on_with_its_pools(by_head, qk):
    """From the batch that reads the prompts to the one of single tokens, without a second pair of pools."""
    from video_dit_long_gb300.packed import PagedAttention, PagedBatch
    page, prompts = 16, [70, 200, 33]
    st = Streams(3, 220, 6, 2, 5, 1)
    table, n_pages = pages_for([x + 5 for x in prompts], page, 5)
    read = PagedBatch(st.h, prompts, prompts, table, sum(prompts), 2, page, 20 * n_pages, 1)
    layer = PagedAttention(read, *st.w, EPS, qk=qk, by_head=by_head)
    layer.forward(*st.step(prompts, prompts, sum(prompts)))
    st.h.sync()
    st.check(layer, prompts, prompts)
    now = [x + 1 for x in prompts]
    batch = PagedBatch(st.h, [1] * 3, now, table, 4, 2, page, 20 * n_pages, 1)
    before = torch.cuda.memory_allocated()
    step = PagedAttention(batch, *st.w, EPS, qk=qk, k_cache=layer.k_cache, v_cache=layer.v_cache)
    assert torch.cuda.memory_allocated() - before < layer.k_cache.numel() * 2
    for _ in range(3):
        step.out.zero_()
        step.forward(*st.step([1] * 3, now, 4))
        st.h.sync()
        st.check(step, [1] * 3, now)
        now = [x + 1 for x in now]
        batch.next(k_lens=now)
    with pytest.raises(ValueError):
        PagedAttention(batch, *st.w, EPS, qk=qk, k_cache=layer.k_cache[1:], v_cache=layer.v_cache)
    with pytest.raises(ValueError):
        PagedAttention(batch, *st.w, EPS, qk="bf16" if qk == "f16" else "f16", k_cache=layer.k_cache, v_cache=layer.v_cache)

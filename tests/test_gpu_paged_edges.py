"""Calls over pages at the borders of what they take: lengths that are none, plans of other calls, shared prefixes over
every kind of copy, calls of different data at once."""
import pytest

from . import packed_ref as R
from .test_gpu_paged_append import Step as Append
from .test_gpu_paged_attention import GROUPS, Step, laid
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


@pytest.mark.parametrize("case", GROUPS)
@pytest.mark.parametrize("page,order", [(16, "heads"), (16, (1, 0, 2)), (32, (2, 1, 0)), (48, "tokens"), (64, "tokens"),
                                        (64, "heads"), (112, "tokens"), (128, "tokens"), (128, (2, 0, 1)), (384, "heads")])
def test_shared_prefixes_over_every_kind_of_copy(case, page, order):
    """Boxes of 16 and 32 tokens by groups of 8 and, in orders of the pool that groups cannot say, by rows; larger ones."""
    q, k, groups = case
    b = Step(q, k, 6, 2, 1, page=page, seed=30, groups=groups, order=order if order == "heads" else "tokens")
    if isinstance(order, tuple):
        b.k_cache, b.v_cache = laid(b.k_cache, order), laid(b.v_cache, order)
    b.forward().check().again_the_same()


@pytest.mark.parametrize("page", [48, 64, 128])
@pytest.mark.parametrize("copies", [False, True])
def test_groups_dealt_out_over_every_kind_of_copy(page, copies):
    """More streams than are cut into stretches, two groups among them, one whose streams have copies of the prefix."""
    q = [1, 2, 0, 1] * 280
    k = [30 + s % 7 for s in range(40)] + [1500 + s for s in range(60)] + [40] * 1020
    Step(q, k, 4, 2, 1, page=page, seed=31, groups=[(40, 0), (60, 1490)], copies=copies).forward().check().again_the_same()


def test_two_steps_of_different_data_at_once():
    """One plan and table, two streams, queries and pools of their own: each call's results are its own."""
    lens = [1] * 8, [2100 + n for n in range(8)]
    a, b = (Step(*lens, 8, 4, 1, seed=19, groups=[(8, 2000)]) for _ in "ab")
    g = torch.Generator(device="cuda").manual_seed(32)
    b.q[b.pad:-b.pad] = torch.randn(b.q[b.pad:-b.pad].shape, generator=g, device="cuda").to(b.q.dtype)
    b.k_cache.neg_()
    b.v_cache.mul_(0.5)
    b.k, b.v = [-x for x in b.k], [x * 0.5 for x in b.v]
    want = []
    for x in (a, b):
        x.forward().check()
        want.append((x.out.clone(), x.lse.clone()))
    assert not torch.equal(want[0][0], want[1][0])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        torch.cuda.synchronize()
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                x.out.fill_(7.0)
                x.lse.fill_(7.0)
                x.ws.fill_(255)
                x.h.paged_forward(a.plan, x.q, x.k_cache, x.v_cache, x.out, x.lse, workspace=x.ws)
        torch.cuda.synchronize()
        for x, (out, lse) in zip((a, b), want):
            x.h.sync()
            assert torch.equal(x.out, out) and torch.equal(x.lse, lse)


def test_two_appends_of_different_data_at_once():
    """One plan, two streams, tokens and pools of their own, cleared in every round."""
    b = Append([700, 1, 77], [900, 40, 77], 24, 8, page=16, seed=8)
    n = slice(b.pad, b.q.shape[0] - b.pad)
    g = torch.Generator(device="cuda").manual_seed(33)
    other = b.qkv.clone()
    other[n] = torch.randn(other[n].shape, generator=g, device="cuda").to(torch.bfloat16)
    made = []
    for x in (b.qkv, other):
        pools = [torch.full_like(t, 7.0) for t in (b.k_cache, b.v_cache, b.q_out)]
        args = dict(q=x[:, :24], k=x[:, 24:32], v=x[:, 32:], k_cache=pools[0], v_cache=pools[1], q_out=pools[2])
        b.append(**args).h.sync()
        made.append((args, pools, [t.clone() for t in pools]))
    assert not any(torch.equal(x, y) for x, y in zip(made[0][2], made[1][2]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        torch.cuda.synchronize()
        for s, (args, pools, _) in zip(streams, made):
            with torch.cuda.stream(s):
                for t in pools:
                    t.fill_(7.0)
                b.append(**args)
        torch.cuda.synchronize()
        b.h.sync()
        for _, pools, want in made:
            assert all(torch.equal(x, y) for x, y in zip(pools, want))


@pytest.mark.parametrize("lens", [([1], [1]), ([90, 200], [90, 200]), ([1] * 40, [900] * 40)])
def test_plans_of_rows_and_of_pages_are_no_plans_of_each_other(lens):
    """Reported, and nothing is written.  (Each has room for what the other's calls read before its header:
    test_paged_apart.py.)"""
    b = Step(*lens, 4, 2, 1, seed=34)
    K, h, T = b.K, b.h, b.q.shape[0]
    cu_k = torch.tensor([0] + lens[1], dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    rows = h.packed_plan(b.cu_q, cu_k, T, sum(lens[1]), 2, 1)
    h.sync()

    def refused(call):
        with pytest.raises(K.K6Error) as e:
            call()  # at once where the room that the plan should have, and has not, holds another argument
            h.sync()
        assert e.value.status == K.ERR_INVALID_ARG
        assert bool((b.out == 7.0).all()) and bool((b.lse == 7.0).all())

    p = K.PagedPlan(b.plan.batch, rows.buffer, b.table)
    refused(lambda: h.paged_forward(p, b.q, b.k_cache, b.v_cache, b.out, b.lse, workspace=b.ws))
    pools = [torch.full_like(x, 7.0) for x in (b.k_cache, b.v_cache)]
    x = torch.zeros((T, 8, 128), dtype=torch.bfloat16, device="cuda")
    rotated = torch.full_like(b.q, 7.0)
    pos = torch.zeros((T, 3), dtype=torch.int32, device="cuda")
    refused(lambda: h.paged_append(p, x[:, :4], x[:, 4:6], x[:, 6:], pos, q_out=rotated, k_cache=pools[0], v_cache=pools[1]))
    assert all(bool((x == 7.0).all()) for x in (rotated, *pools))
    p = K.PackedPlan(rows.batch, b.plan.buffer)
    k, v = (torch.zeros((sum(lens[1]), 2, 128), dtype=t, device="cuda") for t in (b.q.dtype, torch.bfloat16))
    ws = torch.empty(h.packed_workspace_bytes(rows), dtype=torch.uint8, device="cuda")
    refused(lambda: h.packed_forward(p, b.q, k, v, b.out, b.lse, workspace=ws))
    b.forward().check()


@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("tokens", [2540, 6079, 6080])
def test_tokens_on_both_sides_of_the_strides(Hkv, tokens):
    """Stretches of passes below 40 tokens a SM, and with few key heads beyond; whole runs in strides from there on."""
    b = Append([tokens - 40, 40 - 4], [tokens - 40, 300], 24, Hkv, page=64, seed=35, pad=2).append()
    b.h.sync()
    a, n = b.pad, b.q_out.shape[0] - b.pad
    assert b.q_out.shape[0] == tokens
    b.near(b.q_out[a:n], b.q[a:n], b.qw, "q")
    at = torch.cat((torch.arange(tokens - 40, device="cuda"), torch.arange(264, 300, device="cuda")))
    row = torch.cat((b.table[0].expand(tokens - 40, -1), b.table[1].expand(36, -1)))
    pages = row.gather(1, (at // 64)[:, None])[:, 0].long()
    b.near(b.k_cache[pages, at % 64], b.k[a:n], b.kw, "k")
    assert torch.equal(b.v_cache[pages, at % 64], b.v[a:n])
    for cache in (b.k_cache, b.v_cache):  # nothing else
        cache[pages, at % 64] = 7.0
        assert bool((cache == 7.0).all())


def test_appends_past_four_gigabytes():
    """A pool of 5.4 GB of keys and as much of values, whose last pages are a stream's."""
    n_pages, page, Hkv = 82_000, 64, 4
    b = Append([70], [250], 8, Hkv, page=page, seed=36)
    k, v = (torch.zeros((n_pages, page, Hkv, 128), dtype=t, device="cuda") for t in (b.t, torch.bfloat16))
    assert k.numel() * 2 > 1 << 32
    table = torch.tensor([[n_pages - 1, 5, n_pages - 2, n_pages - 9]], dtype=torch.int32, device="cuda")
    plan = b.h.paged_plan(b.cu_q, b.k_now, table, b.q.shape[0], Hkv, page, n_pages, 1)
    b.append(plan=plan, k_cache=k, v_cache=v).h.sync()
    at = torch.arange(180, 250, device="cuda")
    pages, n = table[0].long()[at // page], slice(b.pad, b.pad + 70)
    b.near(k[pages, at % page], b.k[n], b.kw, "k")
    assert torch.equal(v[pages, at % page], b.v[n])
    for cache in (k, v):
        cache[pages, at % page] = 0.0
        assert not cache.any()


def part_of(t, width, at):
    """The rows of t as a part of wider ones: heads `at` and on of `width`, sevens beside them."""
    x = torch.full((t.shape[0], width, 128), 7.0, dtype=t.dtype, device="cuda")
    x[:, at:at + t.shape[1]] = t
    return x, x[:, at:at + t.shape[1]]


@pytest.mark.parametrize("qk", ["f16", "bf16"])
@pytest.mark.parametrize("lse", [True, False])
def test_rows_that_are_parts_of_wider_ones(qk, lse):
    """Queries out of a fused projection, results into part of a wider tensor, joins and shared prefixes among them; with
    and without lse."""
    lens = [1, 1, 1, 1, 90], [1300, 1301, 1302, 700, 5000]
    want = Step(*lens, 6, 2, 1, qk=qk, seed=37, groups=[(4, 690)]).forward().check()
    b = Step(*lens, 6, 2, 1, qk=qk, seed=37, groups=[(4, 690)])
    _, b.q = part_of(b.q, 11, 0)
    whole, b.out = part_of(b.out, 9, 2)
    b.h.paged_forward(b.plan, b.q, b.k_cache, b.v_cache, b.out, b.lse if lse else None, workspace=b.ws)
    b.h.sync()
    assert torch.equal(b.out, want.out) and (not lse or torch.equal(b.lse, want.lse))
    assert lse or bool((b.lse == 7.0).all())
    assert bool((whole[:, :2] == 7.0).all()) and bool((whole[:, 8:] == 7.0).all())


@pytest.mark.parametrize("page,columns,cut", [(65536, 8191, 0), (64, 8388607, 5), (1 << 20, 511, 1)])
def test_positions_up_to_the_limit(page, columns, cut):
    """Streams of nearly 2^29 keys, every column of whose table names the pool's one page: attention is that over the
    page, every key as often as it comes, and new tokens lie at the end of it."""
    from video_dit_long_gb300 import k6attn as K
    g = torch.Generator(device="cuda").manual_seed(38)
    Lk, H, T = page * columns - cut, 2, 3
    k, v = (torch.randn((1, page, 1, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    v[..., :64] = 1.0
    q = torch.randn((T, H, 128), generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros((1, columns), dtype=torch.int32, device="cuda")
    h = K.Handle.for_packed(H)
    plan = h.paged_plan(i32(0, T), i32(Lk), table, T, 1, page, 1, 0)
    out, lse = torch.empty_like(q), torch.empty((H, T), device="cuda")
    ws = torch.empty(h.paged_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    h.paged_forward(plan, q, k, v, out, lse, workspace=ws)
    h.sync()
    s = torch.einsum("thd,kd->htk", q.double(), k[0, :, 0].double()) / 128 ** 0.5
    a = torch.einsum("thd,kd->htk", q.double().abs(), k[0, :, 0].double().abs()).amax(-1) / 128 ** 0.5
    times = torch.full((page,), columns, dtype=torch.float64, device="cuda")
    times[page - cut:] -= 1
    want = torch.logsumexp(s + times.log(), -1)
    # as packed_ref.attention; the fp32 row sums add a term of 128 keys at a time, each off by 2^-24 of the sum
    tiles = Lk / 128 / torch.cuda.get_device_properties(0).multi_processor_count
    R.assert_within(lse, want, 2.0 ** -19 * (a + 1) + 2.0 ** -20 * want.abs() + tiles * 2.0 ** -24, "lse")
    p = torch.exp(s + times.log() - want[..., None])
    ref, mag = (torch.einsum("htk,kd->thd", p, x) for x in (v[0, :, 0].double(), v[0, :, 0].double().abs()))
    # a tile adds 8 products of 16 keys to O, each sum cut off below 2^-23 of it
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13 + tiles * 8 * 2.0 ** -23) * mag
    R.assert_within(out, ref, bound, "out")
    kc, vc = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    x = torch.randn((T, H + 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    zero = torch.zeros((T, 3), dtype=torch.int32, device="cuda")
    h.paged_append(plan, None, x[:, H:H + 1], x[:, H + 1:], zero, q_out=None, k_cache=kc, v_cache=vc)
    h.sync()
    at = (torch.arange(Lk - T, Lk, device="cuda") % page)
    for cache, rows in ((kc, x[:, H:H + 1]), (vc, x[:, H + 1:])):  # at position (0, 0, 0) nothing turns
        assert torch.equal(cache[0, at], rows)
        cache[0, at] = 7.0
        assert bool((cache == 7.0).all())


@pytest.mark.parametrize("page,order", [(16, (1, 0, 2)), (48, "tokens"), (64, "tokens"), (64, "heads"), (128, "tokens")])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "behind"])
def test_a_page_that_is_none_over_every_kind_of_copy(page, order, bad):
    """A group's first stream names it: the group has results of some kind, the streams beside it theirs; reported."""
    q, k = [1, 1, 1, 1, 2, 70], [700, 701, 702, 703, 300, 500]
    b = Step(q, k, 6, 2, 1, page=page, seed=39, groups=[(4, 690)], order="heads" if order == "heads" else "tokens")
    if isinstance(order, tuple):
        b.k_cache, b.v_cache = laid(b.k_cache, order), laid(b.v_cache, order)
    want = b.forward().check().out.clone()
    good = b.table.clone()
    b.table[0, 200 // page] = b.k_cache.shape[0] if bad == "behind" else bad
    b.out.fill_(7.0)
    b.forward()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_INVALID_ARG
    own = slice(b.pad + 4, None)
    assert torch.equal(b.out[own], want[own]) and bool((b.out[:b.pad] == 7.0).all())
    b.table.copy_(good)
    b.forward().check()
    assert torch.equal(b.out, want)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("bad", [-1, 1, 2 ** 31 - 1])
def test_a_page_that_a_pool_of_one_does_not_have(page, bad):
    b = Step([2, 1], [page, page - 3], 6, 2, 1, page=page, seed=40)
    b.k_cache, b.v_cache = (c[b.table[0, :1].long()] for c in (b.k_cache, b.v_cache))
    b.table.fill_(-1)
    b.table[0, 0], b.table[1, 0] = 0, bad
    b.plan = b.h.paged_plan(b.cu_q, b.k_now, b.table, b.q.shape[0], 2, page, 1, 1)
    with pytest.raises(b.K.K6Error):  # the new token has no place
        b.h.sync()
    b.forward()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_INVALID_ARG
    ref, _, bo, _ = R.attention(b.q[b.pad:b.pad + 2], b.k[0], b.v[0], [2], [page], 1)
    R.assert_within(b.out[b.pad:b.pad + 2], ref, bo, "out")


@pytest.mark.parametrize("cu,shared", [([2, 8], [690]), ([0, 0, 2, 2, 2, 8, 8, 8, 8, 8, 8, 8], [5, 0, 2 ** 31 - 1, 9, 698, 1, 1, 1, 1, 1, 1]),
                                       ([8, 8], [3]), ([3, 5, 8], [690, 650])])
def test_groups_anywhere_among_the_streams(cu, shared):
    """Streams before the first group, groups of no streams, more groups than streams."""
    q, k = [4, 1, 1, 1, 0, 1, 1, 2], [100, 40, 700, 701, 702, 703, 704, 705]
    b = Step(q, k, 6, 2, 1, page=32, seed=41, groups=[(1, 0), (1, 0), (6, 698)])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b.more = dict(cu_groups=i32(cu), shared=i32(shared))
    b.plan = b.h.paged_plan(b.cu_q, b.k_now, b.table, b.q.shape[0], 2, 32, b.k_cache.shape[0], 1, **b.more)
    b.ws = torch.full((b.h.paged_workspace_bytes(b.plan),), 255, dtype=torch.uint8, device="cuda")
    b.forward().check().again_the_same()


def test_a_group_whose_streams_have_nothing_new():
    b = Step([0, 0, 3, 0], [700, 701, 90, 700], 6, 2, 1, page=64, seed=42, groups=[(2, 690), (1, 0), (1, 700)])
    b.forward().check().again_the_same()

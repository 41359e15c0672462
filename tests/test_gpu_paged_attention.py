"""Attention over pages against the definition in 64 bits: page sizes and orders,
ragged and empty streams, masks, shared prefixes, garbage behind a stream's last
key, bad tables and plans, captured graphs."""
import pytest

from . import packed_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def pool(n_pages, page, Hkv, dtype, order="tokens"):
    """NaN pages [n_pages][page][Hkv][128]; `order`: what lies behind the page in memory, or both kinds' parts."""
    if order == "heads":
        return torch.full((n_pages, Hkv, page, 128), NAN, dtype=dtype, device="cuda").transpose(1, 2)
    return torch.full((n_pages, page, Hkv, 128), NAN, dtype=dtype, device="cuda")


class Step:
    """A step over pages between NaN rows and NaN pages, and its plan.  groups: [(streams, shared tokens)]."""

    def __init__(self, q_lens, k_lens, H, Hkv, block, page=16, qk="f16", seed=0, pad=3, order="tokens", groups=(),
                 std=1.0, extra_columns=2, copies=False):
        from video_dit_long_gb300 import k6attn as K
        self.K, self.q_lens, self.k_lens, self.H, self.Hkv, self.block, self.pad = K, q_lens, k_lens, H, Hkv, block, pad
        self.page = page
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = torch.float16 if qk == "f16" else torch.bfloat16
        n, nq = len(q_lens), sum(q_lens)
        first = list(range(n))  # of each stream's group, and what it shares
        shared = [0] * n
        at = 0
        for streams, tokens in groups:
            for s in range(at, at + streams):
                first[s], shared[s] = at, tokens
            at += streams
        wanted = [-(-k // page) for k in k_lens]
        n_pages = sum(wanted) + 2
        free = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        self.q = torch.full((nq + 2 * pad, H, 128), NAN, dtype=t, device="cuda")
        self.q[pad:pad + nq] = (torch.randn((nq, H, 128), generator=g, device="cuda") * std).to(t)
        self.k_cache, self.v_cache = pool(n_pages, page, Hkv, t, order), pool(n_pages, page, Hkv, torch.bfloat16, order)
        columns = max(wanted, default=0) + extra_columns
        table = torch.full((n, columns), -7, dtype=torch.int32)
        self.k, self.v = [], []
        for s, (w, lk) in enumerate(zip(wanted, k_lens)):
            k = (torch.randn((lk, Hkv, 128), generator=g, device="cuda") * std).to(t)
            v = torch.randn((lk, Hkv, 128), generator=g, device="cuda").to(torch.bfloat16)
            f = first[s]
            common = min(shared[s], lk, k_lens[f])
            k[:common], v[:common] = self.k[f][:common] if f != s else k[:common], self.v[f][:common] if f != s else v[:common]
            self.k.append(k)
            self.v.append(v)
            same = 0 if f == s or copies else common // page
            table[s, :same] = table[f, :same]
            for j in range(same, w):
                table[s, j] = free.pop()
            for cache, x in ((self.k_cache, k), (self.v_cache, v)):
                for j in range(same, w):
                    part = x[j * page:(j + 1) * page]
                    cache[int(table[s, j]), :part.shape[0]] = part
        self.table = table.cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cu_q = i32([0] + q_lens).cumsum(0).to(torch.int32) + pad
        self.k_now = i32(k_lens)
        self.more = {}
        if groups:
            self.more = dict(cu_groups=i32([0] + [x for x, _ in groups]).cumsum(0).to(torch.int32),
                             shared=i32([x for _, x in groups]))
        self.h = K.Handle.for_packed(H)
        self.plan = self.h.paged_plan(self.cu_q, self.k_now, self.table, nq + 2 * pad, Hkv, page, n_pages, block, **self.more)
        self.out = torch.full((nq + 2 * pad, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((H, nq + 2 * pad), 7.0, device="cuda")
        self.ws = torch.full((self.h.paged_workspace_bytes(self.plan),), 255, dtype=torch.uint8, device="cuda")

    def forward(self):
        self.h.paged_forward(self.plan, self.q, self.k_cache, self.v_cache, self.out, self.lse, workspace=self.ws)
        return self

    def check(self):
        self.h.sync()
        a, n = self.pad, self.out.shape[0] - self.pad
        zero = torch.zeros((0, self.Hkv, 128), device="cuda")
        ref, rl, bo, bl = R.attention(self.q[a:n], torch.cat([zero.to(self.q.dtype)] + self.k),
                                      torch.cat([zero.to(torch.bfloat16)] + self.v), self.q_lens, self.k_lens, self.block)
        R.assert_within(self.out[a:n], ref, bo, "out")
        R.assert_within(self.lse[:, a:n], rl, bl, "lse")
        for x in (self.out[:a], self.out[n:], self.lse[:, :a], self.lse[:, n:]):
            assert bool((x == 7.0).all())  # rows outside the streams
        return self

    def again_the_same(self):
        """Another plan and pass leave the same bits."""
        first = self.out.clone(), self.lse.clone()
        self.h.paged_replan(self.plan, self.cu_q, self.k_now, self.table, **self.more)
        self.ws.fill_(255)
        self.forward().h.sync()
        assert torch.equal(first[0], self.out) and torch.equal(first[1], self.lse)
        return self


@pytest.mark.parametrize("page", [16, 48, 64, 112, 128, 384])
@pytest.mark.parametrize("order", ["tokens", "heads"])
@pytest.mark.parametrize("qk", ["f16", "bf16"])
def test_page_sizes_and_orders(page, order, qk):
    Step([1, 3, 70, 5], [1, 129, 500, 65], 6, 2, 1, page=page, qk=qk, order=order, seed=1).forward().check()


@pytest.mark.parametrize("lens", [([1], [1]), ([1], [16]), ([1], [17]), ([1, 1, 1], [15, 127, 129]), ([128], [128]),
                                  ([0, 5, 0, 300], [0, 5, 9, 300]), ([300, 0, 2], [10, 40, 1]), ([2, 1], [0, 3])])
@pytest.mark.parametrize("H,Hkv", [(6, 1), (6, 2), (4, 4), (128, 1)])
@pytest.mark.parametrize("block", [0, 1, 50])
def test_lengths_and_masks(lens, H, Hkv, block):
    """Empty streams, no keys at all, more queries than keys (rows that see nothing, tokens that no page holds)."""
    Step(*lens, H, Hkv, block, seed=2).forward().check()


@pytest.mark.parametrize("q_lens,k_lens,Hkv", [([1], [9000], 1), ([1, 1, 1], [5000, 1, 1300], 2), ([3, 2], [4097, 8192], 4),
                                               ([200], [6000], 4)])
@pytest.mark.parametrize("block", [0, 1, 432])
def test_long_key_ranges_are_split_and_joined(q_lens, k_lens, Hkv, block):
    Step(q_lens, k_lens, 8, Hkv, block, seed=4).forward().check().again_the_same()


GROUPS = [
    # (q_lens, k_lens, groups): tokens over a common prompt; a prefix that ends inside a page and a tile; one group of
    # one stream; streams without a group behind the last; a stream with nothing new and one with nothing at all; one
    # shorter than the prefix; queries that begin inside it
    ([1] * 6, [700, 650, 641, 900, 1000, 641], [(6, 640)]),
    ([1] * 9, [2100] * 4 + [300, 301, 302, 303, 50], [(4, 2000), (4, 299)]),
    ([2, 1, 1, 3, 1], [600, 610, 620, 50, 40], [(3, 590), (1, 40)]),
    ([1, 0, 1, 0, 1, 1], [1000, 1000, 1001, 0, 1002, 1000], [(6, 999)]),
    ([1, 1, 1, 1, 1, 1], [1000, 1000, 130, 1000, 1000, 1000], [(6, 999)]),
    ([200, 1, 1, 1, 1, 1, 1], [700, 700, 700, 700, 700, 700, 700], [(7, 690)]),
    ([5] * 14, [4357, 4500, 5000, 4400, 4700, 4900, 6000, 4358, 1086, 1100, 1500, 1200, 1300, 2500],
     [(8, 4352), (5, 1081), (1, 0)]),
    ([1] * 5, [513] * 5, [(5, 513)]),
    ([1] * 70, [1300 + n for n in range(70)], [(70, 1280)]),
]


@pytest.mark.parametrize("case", GROUPS)
@pytest.mark.parametrize("H,Hkv", [(6, 2), (8, 8), (24, 1)])
@pytest.mark.parametrize("block", [0, 1, 64])
def test_shared_prefixes(case, H, Hkv, block):
    q, k, groups = case
    Step(q, k, H, Hkv, block, seed=5, groups=groups).forward().check().again_the_same()


def test_a_shared_prefix_in_copies():
    """The streams' first tokens are the same, in pages of their own."""
    Step([1] * 6, [700, 650, 641, 900, 1000, 641], 6, 2, 1, seed=6, groups=[(6, 640)], copies=True).forward().check()


def test_with_and_without_groups():
    """The same streams planned as a group and on their own: each within the bounds of the definition."""
    b = Step([1] * 12, [3000 + n for n in range(12)], 8, 2, 1, seed=7, groups=[(12, 2944)]).forward().check()
    b.more["shared"].fill_(0)
    b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table, **b.more)
    b.out.fill_(7.0)
    b.forward().check()


def test_more_streams_than_one_block_plans():
    """Past 1,024 streams the batch is dealt out from a sorted list; groups and long key ranges among them."""
    g = torch.Generator().manual_seed(1)
    q = torch.randint(0, 4, (1100,), generator=g).tolist()
    k = [x + (x % 3) for x in q]
    for s in range(40, 60):
        q[s], k[s] = 1, 700 + s
    q[700], k[700] = 2, 20_000
    q[3], k[3] = 300, 310
    Step(q, k, 4, 2, 1, seed=17, groups=[(40, 0), (20, 690)]).forward().check().again_the_same()


def test_a_batch_too_large_for_stretches():
    """30 prompts of 512 tokens and one of 9,000, 24 key heads: dealt out by load; checked against its own parts."""
    lens = [512] * 30 + [9000]
    b = Step(lens, lens, 24, 24, 1, seed=18, page=64)
    b.forward().h.sync()
    rows = slice(b.pad + 512 * 7, b.pad + 512 * 8)
    ref, rl, bo, bl = R.attention(b.q[rows], b.k[7], b.v[7], [512], [512], 1)
    R.assert_within(b.out[rows], ref, bo, "out")
    R.assert_within(b.lse[:, rows], rl, bl, "lse")
    last = slice(b.pad + 512 * 30, b.pad + 512 * 30 + 9000)
    h = 17
    ref, rl, bo, bl = R.attention(b.q[last, h:h + 1][-100:], b.k[30][:, h:h + 1], b.v[30][:, h:h + 1], [100], [9000], 1)
    R.assert_within(b.out[last, h:h + 1][-100:], ref, bo, "out")


def test_large_and_equal_logits():
    Step([300], [300], 4, 2, 1, seed=7, std=6.0).forward().check()
    b = Step([1] * 4, [1000] * 4, 4, 2, 0, seed=8, groups=[(4, 900)])
    b.q.fill_(0.0)  # every key alike: lse = log(1000)
    b.forward().check()


def test_infinite_and_nan_queries_stay_in_their_rows():
    b = Step([1] * 8, [700 + n for n in range(8)], 4, 2, 1, seed=9, groups=[(8, 690)])
    b.forward().h.sync()
    want = b.out.clone()
    b.q[b.pad + 2, 1] = NAN
    b.q[b.pad + 5, 2, 3] = float("inf")
    b.forward().h.sync()
    assert bool(b.out[b.pad + 2, 1].isnan().all()) and bool(b.out[b.pad + 5, 2].isnan().all())
    b.out[b.pad + 2, 1], b.out[b.pad + 5, 2] = want[b.pad + 2, 1], want[b.pad + 5, 2]
    assert torch.equal(b.out, want)


@pytest.mark.parametrize("interleaved", ["page", "token", "head"])
def test_keys_and_values_of_one_tensor(interleaved):
    """Pools that are parts of one tensor, by page, token or head."""
    want = Step([3, 70], [300, 200], 6, 2, 1, qk="bf16", seed=10).forward().check()
    b = Step([3, 70], [300, 200], 6, 2, 1, qk="bf16", seed=10)
    both = torch.stack((b.k_cache, b.v_cache), {"page": 1, "token": 2, "head": 3}[interleaved]).contiguous()
    b.k_cache, b.v_cache = both.unbind({"page": 1, "token": 2, "head": 3}[interleaved])
    b.forward().check()
    assert torch.equal(b.out, want.out)


def test_pages_past_four_gigabytes():
    """A pool of 5.4 GB whose last pages are a stream's."""
    from video_dit_long_gb300 import k6attn as K
    n_pages, page, Hkv = 82_000, 64, 4
    k, v = (torch.empty((n_pages, page, Hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    assert k.numel() * 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(11)
    pages = torch.tensor([n_pages - 1, 5, n_pages - 2, n_pages - 9], dtype=torch.int32, device="cuda")
    for x in (k, v):
        x[pages.long()] = torch.randn((4, page, Hkv, 128), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((7, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    h = K.Handle.for_packed(8)
    plan = h.paged_plan(i32(0, 7), i32(250), pages[None].contiguous(), 7, Hkv, page, n_pages, 1)
    out, lse = torch.empty_like(q), torch.empty((8, 7), device="cuda")
    ws = torch.empty(h.paged_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    h.paged_forward(plan, q, k, v, out, lse, workspace=ws)
    h.sync()
    kd, vd = (x[pages.long()].reshape(-1, Hkv, 128)[:250] for x in (k, v))
    ref, rl, bo, bl = R.attention(q, kd, vd, [7], [250], 1)
    R.assert_within(out, ref, bo, "out")
    R.assert_within(lse, rl, bl, "lse")


def test_captured_with_its_plan_and_on_another_stream():
    """A graph that plans and attends, replayed as the streams grow; and the same calls on a stream of their own."""
    b = Step([1, 1, 1, 1], [700, 701, 702, 703], 4, 2, 1, seed=12, groups=[(4, 690)])
    b.forward().check()
    k_lens = b.k_lens
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table, **b.more)
        b.forward()
    k, v = b.k, b.v
    for cut in (0, 3, 90):
        b.k_lens = [x - cut for x in k_lens]
        b.k, b.v = [x[:n] for x, n in zip(k, b.k_lens)], [x[:n] for x, n in zip(v, b.k_lens)]
        b.k_now.copy_(torch.tensor(b.k_lens, dtype=torch.int32))
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        graph.replay()
        b.check()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table, **b.more)
        b.forward()
        b.check()


def test_two_calls_at_once_on_two_streams():
    """One plan, two streams, a workspace each."""
    a, b = (Step([1] * 8, [2100 + n for n in range(8)], 8, 4, 1, seed=s, groups=[(8, 2000)]) for s in (19, 20))
    b.table.copy_(a.table)
    c = Step([1] * 8, [2100 + n for n in range(8)], 8, 4, 1, seed=19, groups=[(8, 2000)])
    a.forward().h.sync()
    want = a.out.clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, x in zip(streams, (a, c)):
            with torch.cuda.stream(s):
                x.out.fill_(7.0)
                x.h.paged_forward(a.plan, x.q, x.k_cache, x.v_cache, x.out, x.lse, workspace=x.ws)
    torch.cuda.synchronize()
    for x in (a, c):
        x.h.sync()
        assert torch.equal(x.out, want)


def test_bad_lengths_and_plans_are_reported_and_write_nothing():
    b = Step([90, 200], [90, 200], 4, 2, 1, seed=13, groups=[(2, 0)])
    K = b.K
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(cu_q=b.cu_q.clone(), k=b.k_now.clone(), g=b.more["cu_groups"].clone(), s=b.more["shared"].clone())
    for bad in (dict(cu_q=[3, 200, 100]), dict(cu_q=[-1, 50, 100]), dict(cu_q=[0, 50, 10_000]), dict(k=[-1, 200]),
                dict(k=[90, 100_000]), dict(g=[0, 3]), dict(g=[-1, 2]), dict(g=[2, 0]), dict(s=[-1])):
        x = {**good, **{n: i32(v) for n, v in bad.items()}}
        b.h.paged_replan(b.plan, x["cu_q"], x["k"], b.table, cu_groups=x["g"], shared=x["s"])
        b.forward()
        with pytest.raises(K.K6Error) as e:
            b.h.sync()
        assert e.value.status == K.ERR_INVALID_ARG, bad
        assert bool((b.out == 7.0).all()) and bool((b.lse == 7.0).all())
    b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table, **b.more)
    # a plan that was never made, one made for another mask, and one of packed sequences
    b.h.sync()
    for kind in ("zero", "mask"):
        p = b.h.paged_plan(b.cu_q, b.k_now, b.table, b.out.shape[0], 2, b.page, b.k_cache.shape[0], 5, **b.more)
        if kind == "zero":
            p.buffer.zero_()
        else:
            p.batch.mask_block = 1
        b.h.paged_forward(p, b.q, b.k_cache, b.v_cache, b.out, b.lse, workspace=b.ws)
        with pytest.raises(K.K6Error) as e:
            b.h.sync()
        assert e.value.status == K.ERR_INVALID_ARG
        assert bool((b.out == 7.0).all())
    b.forward().check()


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10_000_000, 2 ** 31 - 1])
def test_a_page_that_the_pool_does_not_have_is_reported(bad):
    """Other streams are as they were."""
    b = Step([1, 1, 2], [300, 200, 170], 4, 2, 1, seed=21)
    b.table[1, 3] = bad
    b.forward()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_INVALID_ARG
    ref, _, bo, _ = R.attention(b.q[3:-3], torch.cat(b.k), torch.cat(b.v), b.q_lens, b.k_lens, 1)
    for rows in (slice(0, 1), slice(2, 4)):
        R.assert_within(b.out[3:-3][rows], ref[rows], bo[rows], "out")
    assert bool((b.out[:3] == 7.0).all()) and bool((b.out[-3:] == 7.0).all())


def test_a_plan_of_a_smaller_batch_is_reported_and_nothing_is_written():
    small, big = Step([1], [1], 4, 4, 1, seed=62), Step([1] * 40, [900] * 40, 4, 4, 1, seed=63, groups=[(40, 890)])
    assert small.plan.buffer.numel() < big.plan.buffer.numel() and big.ws.numel() > 0
    room = torch.full_like(big.plan.buffer, 255)
    room[:small.plan.buffer.numel()] = small.plan.buffer
    p = big.K.PagedPlan(big.plan.batch, room, big.table)
    big.h.paged_forward(p, big.q, big.k_cache, big.v_cache, big.out, big.lse, workspace=big.ws)
    with pytest.raises(big.K.K6Error) as e:
        big.h.sync()
    assert e.value.status == big.K.ERR_INVALID_ARG
    assert bool((big.out == 7.0).all()) and bool((big.lse == 7.0).all())


def test_a_wait_limit_of_zero_gives_up():
    b = Step([90, 200], [90, 200], 4, 2, 1, seed=14)
    b.h.set_option(b.K.OPT_WAIT_LIMIT_NS, 0)
    b.forward()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_TIMEOUT
    b.h.set_option(b.K.OPT_WAIT_LIMIT_NS, 2_000_000_000)
    b.forward().check()


def test_no_queries_no_pages_and_no_lse():
    from video_dit_long_gb300 import k6attn as K
    h = K.Handle.for_packed(4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    e = lambda *s: torch.full((*s, 128), 3.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    table = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    p = h.paged_plan(i32(0, 0, 0), i32(0, 0), table, 0, 2, 16, 0)
    h.paged_forward(p, e(0, 4), e(0, 16, 2), e(0, 16, 2), e(0, 4))
    h.sync()
    p = h.paged_plan(i32(0, 2, 5), i32(0, 0), table, 5, 2, 16, 0)
    out, lse = e(5, 4), torch.zeros((4, 5), device="cuda")
    h.paged_forward(p, e(5, 4), e(0, 16, 2), e(0, 16, 2), out, lse)
    h.sync()
    assert not out.any() and bool((lse == -float("inf")).all())
    b = Step([90, 200], [90, 200], 4, 2, 1, seed=15).forward()
    want = b.out.clone()
    b.out.fill_(7.0)
    b.h.paged_forward(b.plan, b.q, b.k_cache, b.v_cache, b.out, workspace=b.ws)
    b.h.sync()
    assert torch.equal(b.out, want)


def test_keys_without_pages_make_a_bad_plan():
    """A pool of no pages has no tensor map: a plan with keys must not reach the copies."""
    from video_dit_long_gb300 import k6attn as K
    h = K.Handle.for_packed(4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    e = lambda *s: torch.full((*s, 128), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    p = h.paged_plan(i32(0, 5), i32(20), torch.zeros((1, 2), dtype=torch.int32, device="cuda"), 5, 2, 16, 0, 0)
    with pytest.raises(K.K6Error) as err:
        h.sync()
    assert err.value.status == K.ERR_INVALID_ARG
    out = e(5, 4)
    h.paged_forward(p, e(5, 4), e(0, 16, 2), e(0, 16, 2), out)
    with pytest.raises(K.K6Error) as err:
        h.sync()
    assert err.value.status == K.ERR_INVALID_ARG and bool((out == 7.0).all())


def test_refusals():
    b = Step([90], [90], 4, 2, 1, qk="bf16", seed=16)
    K, h = b.K, b.h
    args = dict(plan=b.plan, q=b.q, k_cache=b.k_cache, v_cache=b.v_cache, out=b.out, lse=b.lse, workspace=b.ws)
    wide = torch.zeros((*b.k_cache.shape[:3], 256), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=b.q[:, :3]), dict(k_cache=b.k_cache.half()), dict(q=b.q.cpu()), dict(v_cache=b.v_cache[:, :8]),
                dict(k_cache=wide[..., ::2]), dict(k_cache=b.k_cache[:1])):
        with pytest.raises(ValueError):
            h.paged_forward(**{**args, **bad})
    overlapping = b.k_cache.flatten()[:128 * 3].as_strided(b.k_cache.shape, (128, 128, 128, 1))
    odd = torch.zeros((*b.k_cache.shape[:3], 132), dtype=torch.bfloat16, device="cuda")[..., :128]
    for bad, status in ((dict(k_cache=overlapping), K.ERR_INVALID_ARG), (dict(k_cache=odd), K.ERR_INVALID_ARG),
                        (dict(out=b.q), K.ERR_INVALID_ARG)):
        with pytest.raises(K.K6Error) as e:
            h.paged_forward(**{**args, **bad})
        assert e.value.status == status, bad.keys()
    big = Step([1], [4000], 4, 2, 1, seed=16)
    with pytest.raises(K.K6Error) as e:
        h.paged_forward(big.plan, big.q, big.k_cache, big.v_cache, big.out, big.lse, workspace=big.ws[:16])
    assert e.value.status == K.ERR_WORKSPACE
    n = b.k_cache.shape[0]
    for kw, status in ((dict(kv_heads=3), K.ERR_INVALID_ARG), (dict(mask_block=-1), K.ERR_INVALID_ARG),
                       (dict(page_tokens=8), K.ERR_INVALID_ARG), (dict(page_tokens=24), K.ERR_INVALID_ARG),
                       (dict(n_pages=1 << 40), K.ERR_UNSUPPORTED), (dict(page_tokens=1 << 30), K.ERR_UNSUPPORTED)):
        with pytest.raises(K.K6Error) as e:
            h.paged_plan(b.cu_q, b.k_now, b.table, 96, **{"kv_heads": 2, "page_tokens": 16, "n_pages": n, **kw})
        assert e.value.status == status, kw
    for kw in (dict(shared=b.k_now), dict(cu_groups=b.cu_q)):
        with pytest.raises(ValueError):
            h.paged_plan(b.cu_q, b.k_now, b.table, 96, 2, 16, n, **kw)
    with pytest.raises(ValueError):
        h.paged_plan(b.cu_q, b.k_now, b.table[0], 96, 2, 16, n)
    f32 = K.Handle.for_packed(4, 64, "f32", (16, 24, 24))
    with pytest.raises(K.K6Error):
        f32.paged_plan(b.cu_q, b.k_now, b.table, 96, 2, 16, n)
    h.sync()


def off16(t):
    """A copy of t whose first element lies 16 bytes behind a 32-byte boundary."""
    n, skip = t.numel(), 16 // t.element_size()
    x = torch.empty(n + skip, dtype=t.dtype, device="cuda")[skip:].view(t.shape)
    assert n == 0 or x.data_ptr() % 32 == 16
    return x.copy_(t)


def test_everything_sixteen_byte_aligned_only():
    args = ([1, 1, 3, 130], [5000, 5001, 5002, 200], 4, 2, 1)
    want = Step(*args, seed=61, groups=[(3, 4900)]).forward()
    b = Step(*args, seed=61, groups=[(3, 4900)])
    b.q, b.k_cache, b.v_cache, b.out, b.lse, b.ws = (off16(x) for x in (b.q, b.k_cache, b.v_cache, b.out, b.lse, b.ws))
    b.plan.buffer = off16(b.plan.buffer)
    b.plan.ptr = b.plan.buffer.data_ptr()
    b.forward().check()
    assert torch.equal(b.out[3:-3], want.out[3:-3]) and torch.equal(b.lse[:, 3:-3], want.lse[:, 3:-3])


def laid(cache, order):
    """The pool's axes (pages, tokens, heads) from the outermost to the innermost in memory."""
    return cache.permute(*order, 3).contiguous().permute(*[order.index(i) for i in range(3)], 3)


@pytest.mark.parametrize("order", [(1, 0, 2), (2, 0, 1), (1, 2, 0), (2, 1, 0)])
@pytest.mark.parametrize("page", [16, 32, 64, 80])
def test_any_order_of_the_pool(order, page):
    """Tokens or heads outermost, pages innermost: a call takes what strides can say."""
    b = Step([1, 3, 70, 5], [1, 129, 500, 65], 6, 2, 1, page=page, seed=21)
    b.k_cache = laid(b.k_cache, order)
    b.forward().check()  # keys in one order, values in another
    b.out.fill_(7.0)
    b.v_cache = laid(b.v_cache, order)
    b.forward().check()


@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (2, 1, 0)])
@pytest.mark.parametrize("page,k", [(16, 16), (16, 9), (32, 31), (64, 60), (1024, 1000)])
def test_a_pool_of_one_page(order, page, k):
    b = Step([2], [k], 6, 2, 1, page=page, seed=22)
    b.k_cache, b.v_cache = (laid(c[b.table[0, :1].long()], order) for c in (b.k_cache, b.v_cache))
    b.table.fill_(-1)
    b.table[0, 0] = 0
    b.plan = b.h.paged_plan(b.cu_q, b.k_now, b.table, b.q.shape[0], 2, page, 1, 1)
    b.ws = torch.full((b.h.paged_workspace_bytes(b.plan),), 255, dtype=torch.uint8, device="cuda")
    b.forward().check()


def test_joins_of_few_and_of_many_rows():
    """A stream alone in a step, whose joins take two blocks an entry, and among streams enough for whole entries."""
    Step([5], [9000], 24, 8, 1, page=64, seed=23).forward().check().again_the_same()
    Step([5] + [60] * 12, [9000] + [2000 + 37 * n for n in range(12)], 24, 8, 1, page=64, seed=23).forward().check().again_the_same()

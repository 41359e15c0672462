"""Appending new tokens to pages against the definition in 64 bits: the norm and
rotation of packed_norm_rope, the places that the table gives, everything else left
as it was."""
import pytest

from . import packed_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

AXES, THETA, EPS = (32, 48, 48), 10000.0, 1e-6
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Step:
    """New tokens of streams between NaN rows, a pool of sevens, and the plan."""

    def __init__(self, q_lens, k_lens, H, Hkv, page=16, out="f16", seed=0, pad=2, order="tokens", norm=True, far=0):
        from video_dit_long_gb300 import k6attn as K
        self.K, self.q_lens, self.k_lens, self.pad, self.page, self.Hkv = K, q_lens, k_lens, pad, page, Hkv
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.t = t = torch.float16 if out == "f16" else torch.bfloat16
        n, T = sum(q_lens), sum(q_lens) + 2 * pad
        wanted = [-(-k // page) for k in k_lens]
        self.n_pages = n_pages = sum(wanted) + 2
        free = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        table = torch.full((len(q_lens), max(wanted) + 1), -3, dtype=torch.int32)
        for s, w in enumerate(wanted):
            for j in range(w):
                table[s, j] = free.pop()
        self.table = table.cuda()
        self.qkv = torch.full((T, H + 2 * Hkv, 128), NAN, dtype=torch.bfloat16, device="cuda")
        self.qkv[pad:pad + n] = torch.randn((n, H + 2 * Hkv, 128), generator=g, device="cuda").to(torch.bfloat16)
        self.q, self.k, self.v = self.qkv[:, :H], self.qkv[:, H:H + Hkv], self.qkv[:, H + Hkv:]
        self.positions = torch.randint(-3, 100, (T, 3), generator=g, device="cuda").to(torch.int32)
        self.positions[:, 0] += far
        w = lambda: torch.randn(128, generator=g, device="cuda") * 0.2 + 1.0  # noqa: E731
        self.qw, self.kw = (w(), w()) if norm else (None, None)

        def pool(dtype):
            if order == "heads":
                return torch.full((n_pages, Hkv, page, 128), 7.0, dtype=dtype, device="cuda").transpose(1, 2)
            if order == "wide":  # rows of a wider token
                return torch.full((n_pages, page, Hkv + 3, 128), 7.0, dtype=dtype, device="cuda")[:, :, 1:1 + Hkv]
            return torch.full((n_pages, page, Hkv, 128), 7.0, dtype=dtype, device="cuda")

        self.k_cache, self.v_cache = pool(t), pool(torch.bfloat16)
        self.q_out = torch.full((T, H, 128), 7.0, dtype=t, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cu_q = i32([0] + q_lens).cumsum(0).to(torch.int32) + pad
        self.k_now = i32(k_lens)
        self.h = K.Handle.for_packed(H)
        self.plan = self.h.paged_plan(self.cu_q, self.k_now, self.table, T, Hkv, page, n_pages, 1)

    def append(self, **kw):
        args = dict(plan=self.plan, q=self.q, k=self.k, v=self.v, positions=self.positions, q_weight=self.qw,
                    k_weight=self.kw, eps=EPS, q_out=self.q_out, k_cache=self.k_cache, v_cache=self.v_cache)
        self.h.paged_append(**{**args, **kw})
        return self

    def near(self, got, x, w, what):
        ref, mag = R.norm_rope(x, w, self.positions[self.pad:self.positions.shape[0] - self.pad], AXES, THETA, EPS)
        # half a step of the output's type, and of fp32 for the norm, the weight, the angle (2^-23.4) and the rotation
        R.assert_within(got, ref, R.HALF[self.t] * ref.abs() + 2.0 ** -20 * mag + 2.0 ** -25, what)

    def check(self, q=True):
        self.h.sync()
        a, n = self.pad, self.q_out.shape[0] - self.pad
        if q:
            self.near(self.q_out[a:n], self.q[a:n], self.qw, "q")
            assert bool((self.q_out[:a] == 7.0).all()) and bool((self.q_out[n:] == 7.0).all())
        else:
            assert bool((self.q_out == 7.0).all())
        k = torch.full((n - a, self.Hkv, 128), 0.0, dtype=self.t, device="cuda")
        keep = torch.zeros(n - a, dtype=torch.bool, device="cuda")
        left_k, left_v = self.k_cache.clone(), self.v_cache.clone()
        c = 0
        for s, (lq, lk) in enumerate(zip(self.q_lens, self.k_lens)):
            for i in range(lq):
                p = lk - lq + i
                if p >= 0:
                    page, tok = int(self.table[s, p // self.page]), p % self.page
                    k[c + i] = self.k_cache[page, tok]
                    keep[c + i] = True
                    assert torch.equal(self.v_cache[page, tok], self.v[a + c + i])
                    left_k[page, tok] = left_v[page, tok] = 7.0
            c += lq
        pos, self.positions = self.positions, torch.cat((self.positions[:a], self.positions[a:n][keep], self.positions[n:]))
        self.near(k[keep], self.k[a:n][keep], self.kw, "k")
        self.positions = pos
        assert bool((left_k == 7.0).all()) and bool((left_v == 7.0).all())  # every other place
        return self


@pytest.mark.parametrize("page", [16, 48, 64, 128])
@pytest.mark.parametrize("order", ["tokens", "heads", "wide"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_pages_and_orders(page, order, out):
    Step([1, 3, 70, 5], [1, 129, 500, 65], 6, 2, page=page, out=out, order=order, seed=1).append().check()


@pytest.mark.parametrize("lens", [([1], [1]), ([1], [17]), ([0, 5, 0, 40], [0, 5, 9, 40]), ([30, 0, 2], [10, 40, 1]),
                                  ([2, 1], [0, 3]), ([1] * 50, [100 + n for n in range(50)])])
@pytest.mark.parametrize("H,Hkv", [(6, 1), (24, 8), (4, 4), (128, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_lengths(lens, H, Hkv, norm):
    """Streams with nothing new, more queries than keys (tokens before position 0 are not stored)."""
    Step(*lens, H, Hkv, seed=2, norm=norm, far=100_000).append().check()


@pytest.mark.parametrize("Hkv", [1, 3, 24])
def test_enough_tokens_for_whole_token_runs(Hkv):
    """Past 16 tokens a SM a warp takes all heads of a token."""
    b = Step([2500, 40], [2500, 300], 24, Hkv, page=64, seed=3).append()
    b.h.sync()
    a, n = b.pad, b.q_out.shape[0] - b.pad
    b.near(b.q_out[a:n], b.q[a:n], b.qw, "q")
    at = torch.arange(2500, device="cuda")
    pages = b.table[0].long()[at // 64]
    b.positions = b.positions[:a + 2500 + b.pad]
    b.near(b.k_cache[pages, at % 64], b.k[a:a + 2500], b.kw, "k")
    assert torch.equal(b.v_cache[pages, at % 64], b.v[a:a + 2500])


@pytest.mark.parametrize("tokens", [3, 2600])
def test_keys_and_values_alone(tokens):
    b = Step([tokens], [tokens + 5], 24, 2, page=64, seed=4)
    b.append(q=None, q_out=None)
    if tokens == 3:
        b.check(q=False)
    else:
        k, v = b.k_cache.clone(), b.v_cache.clone()
        b.h.sync()
        b.k_cache.fill_(7.0)
        b.v_cache.fill_(7.0)
        b.append().h.sync()
        assert torch.equal(k, b.k_cache) and torch.equal(v, b.v_cache)


def test_the_same_as_packed_norm_rope():
    """The same bits as the call over rows."""
    b = Step([33, 7, 1], [33, 100, 900], 24, 8, seed=5).append()
    q, k = torch.full_like(b.q_out, 7.0), torch.zeros((b.q_out.shape[0], 8, 128), dtype=b.t, device="cuda")
    b.h.packed_norm_rope(b.q, b.k, b.positions, b.qw, b.kw, EPS, q_out=q, k_out=k, offsets=b.cu_q)
    b.h.sync()
    assert torch.equal(q, b.q_out)
    p = 99 // 16  # the last token of the second stream
    assert torch.equal(b.k_cache[int(b.table[1, p]), 99 % 16], k[b.pad + 39])


def test_in_place_and_interleaved():
    """q_out over q; keys and values in one pool, by page, token and head."""
    for dim in (1, 2, 3):
        b = Step([33, 7, 1], [33, 100, 900], 24, 8, out="bf16", seed=6)
        want = Step([33, 7, 1], [33, 100, 900], 24, 8, out="bf16", seed=6).append().check()
        both = torch.stack((b.k_cache, b.v_cache), dim).contiguous()
        k, v = both.unbind(dim)
        b.append(q_out=b.q, k_cache=k, v_cache=v).h.sync()
        n = slice(b.pad, b.q.shape[0] - b.pad)
        assert torch.equal(b.q[n], want.q_out[n]) and torch.equal(k, want.k_cache) and torch.equal(v, want.v_cache)


def test_a_page_that_the_pool_does_not_have_is_reported():
    b = Step([1, 20, 2], [17, 50, 3], 6, 2, seed=7)
    good = b.table.clone()
    b.table[1, 3] = 1_000_000
    b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table)
    b.append()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_INVALID_ARG
    page = int(good[1, 3])
    assert bool((b.k_cache[page] == 7.0).all()) and bool((b.v_cache[page] == 7.0).all())
    b.table.copy_(good)
    b.h.paged_replan(b.plan, b.cu_q, b.k_now, b.table)
    b.append().check()


def test_a_bad_plan_writes_nothing():
    b = Step([5, 9], [5, 9], 6, 2, seed=8)
    bad = torch.tensor([0, 9, 3], dtype=torch.int32, device="cuda")
    b.h.paged_replan(b.plan, bad, b.k_now, b.table)
    b.append()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_INVALID_ARG
    for x in (b.q_out, b.k_cache, b.v_cache):
        assert bool((x == 7.0).all())


def test_a_key_that_leaves_fp16_is_reported():
    b = Step([5], [5], 6, 2, seed=9, norm=False)
    b.qkv[b.pad + 1, 6, 0] = 1e5
    b.append()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_RANGE


def test_refusals():
    b = Step([5, 9], [5, 9], 6, 2, out="bf16", seed=10)
    K = b.K
    for bad in (dict(q_out=b.q_out.half()), dict(k=b.k.half()), dict(positions=b.positions[:-1]),
                dict(v_cache=b.v_cache.half()), dict(k_cache=b.k_cache[1:])):
        with pytest.raises(ValueError):
            b.append(**bad)
    one = torch.empty((2 * b.k_cache.numel(),), dtype=torch.bfloat16, device="cuda")
    n = b.k_cache.numel()
    for bad in (dict(q=None), dict(q_out=None), dict(q_weight=None), dict(eps=-1.0), dict(eps=NAN),
                dict(k_cache=b.v_cache), dict(q_out=b.q[:, :6].clone().new_empty(b.q_out.shape).copy_(b.q_out),
                                              k_cache=one[:n].view(b.k_cache.shape), v_cache=one[128:128 + n].view(b.k_cache.shape)),
                dict(k_cache=b.k_cache[:, :, :1].expand(b.k_cache.shape))):
        with pytest.raises(K.K6Error) as e:
            b.append(**bad)
        assert e.value.status == K.ERR_INVALID_ARG, bad.keys()
    b.h.sync()
    assert bool((b.q_out == 7.0).all()) and bool((b.k_cache == 7.0).all())


@pytest.mark.parametrize("Hkv,queries", [(8, True), (12, True), (24, False), (8, False)])
def test_enough_tokens_for_strides(Hkv, queries):
    """Past 40 tokens a SM, with key heads for whole passes, warps stride over the tokens; the last stream's rows too."""
    b = Step([6100, 0, 77], [6103, 5, 100], 24, Hkv, page=64, seed=6)
    b.append(**({} if queries else dict(q=None, q_out=None))).h.sync()
    a, n = b.pad, b.q_out.shape[0] - b.pad
    if queries:
        b.near(b.q_out[a:n], b.q[a:n], b.qw, "q")
        assert bool((b.q_out[:a] == 7.0).all()) and bool((b.q_out[n:] == 7.0).all())
    else:
        assert bool((b.q_out == 7.0).all())
    at = torch.cat((torch.arange(3, 6103, device="cuda"), torch.arange(23, 100, device="cuda")))
    row = torch.cat((b.table[0].expand(6100, -1), b.table[2].expand(77, -1)))
    pages = row.gather(1, (at // 64)[:, None])[:, 0].long()
    b.near(b.k_cache[pages, at % 64], b.k[a:n], b.kw, "k")
    assert torch.equal(b.v_cache[pages, at % 64], b.v[a:n])
    for cache in (b.k_cache, b.v_cache):  # nothing else
        cache[pages, at % 64] = 7.0
        assert bool((cache == 7.0).all())


@pytest.mark.parametrize("order", [(1, 0, 2), (2, 0, 1), (1, 2, 0), (2, 1, 0)])
def test_any_order_of_the_pool(order):
    b, c = (Step([1, 3, 70, 5], [1, 129, 500, 65], 6, 2, page=48, seed=7) for _ in range(2))
    b.append().check()
    back = [order.index(i) for i in range(3)]
    c.k_cache, c.v_cache = (x.permute(*order, 3).contiguous().permute(*back, 3) for x in (c.k_cache, c.v_cache))
    c.append().h.sync()
    assert torch.equal(b.k_cache, c.k_cache) and torch.equal(b.v_cache, c.v_cache) and torch.equal(b.q_out, c.q_out)


def test_two_appends_at_once_on_two_streams():
    """Two layers' calls from one plan, into pools of their own, on streams of their own, over and over."""
    b = Step([700, 1, 77], [900, 40, 77], 24, 8, page=16, seed=8)
    b.append().h.sync()
    pools = [(torch.full_like(b.k_cache, 7.0), torch.full_like(b.v_cache, 7.0), torch.full_like(b.q_out, 7.0)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (k, v, q) in zip(streams, pools):
            b.append(k_cache=k, v_cache=v, q_out=q, stream=s)
    torch.cuda.synchronize()
    b.h.sync()
    for k, v, q in pools:
        assert torch.equal(k, b.k_cache) and torch.equal(v, b.v_cache) and torch.equal(q, b.q_out)

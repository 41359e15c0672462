"""A layer over pages as it is used: streams read their prompts, grow step by step,
share a beginning, and are replayed from a captured graph; each step against the
definition in 64 bits over the tokens that the stream has had so far."""
import pytest

from . import packed_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

AXES, THETA, EPS = (32, 48, 48), 10000.0, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Streams:
    """Tokens of n streams, drawn ahead, and what each step of a layer must give."""

    def __init__(self, n, length, H, kv, seed, block):
        from video_dit_long_gb300 import k6attn as K
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.kv, self.block = H, kv, block
        self.qkv = torch.randn((n, length, H + 2 * kv, 128), generator=g, device="cuda").to(torch.bfloat16)
        i = torch.arange(length, device="cuda")
        self.positions = torch.stack((i // 60, i // 6 % 10, i % 6), 1).to(torch.int32)
        self.w = [torch.randn(128, generator=g, device="cuda") * 0.2 + 1.0 for _ in "qk"]
        self.h = K.Handle.for_packed(H)

    def step(self, lens, k_lens, tokens):
        """qkv and positions of a step's tokens, NaN and zero behind them."""
        qkv = torch.full((tokens, (self.H + 2 * self.kv) * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros((tokens, 3), dtype=torch.int32, device="cuda")
        c = 0
        for s, (a, b) in enumerate(zip(lens, k_lens)):
            qkv[c:c + a] = self.qkv[s, b - a:b].flatten(1)
            pos[c:c + a] = self.positions[b - a:b]
            c += a
        return qkv, pos

    def check(self, layer, lens, k_lens):
        """out of the step against attention of the rotated rows, as the layer has them in 16 bits, over the streams'
        own keys; those against the definition of norm and rotation."""
        n = sum(lens)
        table, page = layer.batch.table.long(), layer.k_cache.shape[1]
        keys, values = [], []
        for s, b in enumerate(k_lens):
            rows = [x[table[s, :-(-b // page)]].reshape(-1, self.kv, 128)[:b] for x in (layer.k_cache, layer.v_cache)]
            ref, mag = R.norm_rope(self.qkv[s, :b, self.H:self.H + self.kv], self.w[1], self.positions[:b], AXES, THETA, EPS)
            R.assert_within(rows[0], ref, R.HALF[rows[0].dtype] * ref.abs() + 2.0 ** -20 * mag + 2.0 ** -25, f"keys of {s}")
            assert torch.equal(rows[1], self.qkv[s, :b, self.H + self.kv:])
            keys.append(rows[0])
            values.append(rows[1])
        ref, rl, bo, bl = R.attention(layer.q[:n], torch.cat(keys), torch.cat(values), lens, k_lens, self.block)
        R.assert_within(layer.out[:n], ref, bo, "out")
        R.assert_within(layer.lse[:, :n], rl, bl, "lse")
        assert not layer.out[n:].any()


def pages_for(k_lens, page, seed):
    """A table that gives each stream pages of its own, scattered over a pool."""
    wanted = [-(-k // page) for k in k_lens]
    free = torch.randperm(sum(wanted) + 2, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(k_lens), max(wanted)), -1, dtype=torch.int32)
    at = 0
    for s, w in enumerate(wanted):
        table[s, :w] = free[at:at + w]
        at += w
    return table, sum(wanted) + 2


@pytest.mark.parametrize("page,by_head,qk", [(16, False, "f16"), (48, True, "bf16"), (128, False, "f16")])
def test_streams_grow(page, by_head, qk):
    """Prompts of different lengths, then a token, five tokens and nothing at all each, in one batch."""
    from video_dit_long_gb300.packed import PagedAttention, PagedBatch
    steps = [[70, 1, 200, 33], [1, 1, 1, 1], [5, 0, 1, 2], [1, 1, 0, 1], [60, 1, 1, 17]]
    last = [sum(x) for x in zip(*steps)]
    st = Streams(4, max(last), 6, 2, 1, 1)
    table, n_pages = pages_for(last, page, 1)
    k_lens, batch, layer = [0] * 4, None, None
    for lens in steps:
        k_lens = [a + b for a, b in zip(k_lens, lens)]
        if batch is None:
            batch = PagedBatch(st.h, lens, k_lens, table, 310, 2, page, n_pages, 1)
            layer = PagedAttention(batch, st.w[0], st.w[1], EPS, qk=qk, by_head=by_head)
            layer.k_cache.fill_(float("nan"))  # whatever pages held before
            layer.v_cache.fill_(float("nan"))
        else:
            batch.next(lens, k_lens)
        layer.out.zero_()
        layer.forward(*st.step(lens, k_lens, 310))
        st.h.sync()
        st.check(layer, lens, k_lens)


def test_a_prefix_read_once_and_shared():
    """One stream reads a prompt; seven more begin from its pages (a last one begun is copied) and all go their own way."""
    from video_dit_long_gb300.packed import PagedAttention, PagedBatch
    page, prompt, n = 32, 1000, 8
    st = Streams(n, prompt + 60, 8, 2, 2, 1)
    st.qkv[:, :prompt] = st.qkv[:1, :prompt]
    table, n_pages = pages_for([prompt + 60] * n, page, 2)
    whole = prompt // page
    table[1:, :whole] = table[0, :whole]
    first = PagedBatch(st.h, [prompt] + [0] * (n - 1), [prompt] + [0] * (n - 1), table, prompt, 2, page, n_pages, 1)
    layer = PagedAttention(first, st.w[0], st.w[1], EPS)
    layer.forward(*st.step([prompt], [prompt], prompt))
    for s in range(1, n):
        for c in (layer.k_cache, layer.v_cache):
            c[int(table[s, whole])] = c[int(table[0, whole])]
    batch = PagedBatch(st.h, [1] * n, [prompt + 1] * n, table, 8 * 20, 2, page, n_pages, 1, groups=[(n, prompt)])
    more = PagedAttention(batch, st.w[0], st.w[1], EPS)
    more.k_cache, more.v_cache = layer.k_cache, layer.v_cache
    k_lens = [prompt] * n
    for step in ([1] * n, [3, 1, 0, 20, 1, 1, 1, 1], [1] * n):
        k_lens = [a + b for a, b in zip(k_lens, step)]
        batch.next(step, k_lens)
        more.out.zero_()
        more.forward(*st.step(step, k_lens, 8 * 20))
        st.h.sync()
        st.check(more, step, k_lens)


def test_captured_steps():
    """Plan, append and attention of two layers in one graph, replayed as the streams grow past page and tile borders."""
    from video_dit_long_gb300.packed import PagedAttention, PagedBatch
    page, n = 16, 3
    st = Streams(n, 300, 4, 2, 3, 1)
    table, n_pages = pages_for([300] * n, page, 3)
    prompts = [120, 127, 250]
    batch = PagedBatch(st.h, prompts, prompts, table, sum(prompts), 2, page, n_pages, 1)
    layers = [PagedAttention(batch, st.w[0], st.w[1], EPS) for _ in range(2)]
    for x in layers:
        x.forward(*st.step(prompts, prompts, sum(prompts)))
    one = PagedBatch(st.h, [1] * n, [x + 1 for x in prompts], table, n, 2, page, n_pages, 1)
    steps = [PagedAttention(one, st.w[0], st.w[1], EPS) for _ in range(2)]
    for x, y in zip(steps, layers):
        x.k_cache, x.v_cache = y.k_cache, y.v_cache
    qkv, pos = st.step([1] * n, [x + 1 for x in prompts], n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one.k_lens.add_(1)
        st.h.paged_replan(one.plan, one.offsets, one.k_lens, one.table)
        for x in steps:
            x.forward(qkv, pos)
    one.k_lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    k_lens = prompts
    for _ in range(20):
        k_lens = [x + 1 for x in k_lens]
        a, b = st.step([1] * n, k_lens, n)
        qkv.copy_(a)
        pos.copy_(b)
        graph.replay()
        st.h.sync()
        st.check(steps[0], [1] * n, k_lens)
        assert torch.equal(steps[0].out, steps[1].out)


def test_frames_over_frames():
    """A stream that generates a frame at a time sees the frame whole, and gives what the packed call gives over rows."""
    from video_dit_long_gb300.packed import PagedAttention, PagedBatch
    frame, page = 60, 48
    st = Streams(1, 5 * frame, 6, 2, 4, frame)
    table, n_pages = pages_for([5 * frame], page, 4)
    batch = PagedBatch(st.h, [frame], [frame], table, frame, 2, page, n_pages, frame)
    layer = PagedAttention(batch, st.w[0], st.w[1], EPS)
    for i in range(5):
        k = (i + 1) * frame
        batch.next(k_lens=[k])
        out = layer.forward(*st.step([frame], [k], frame))
        st.h.sync()
        st.check(layer, [frame], [k])
    rows = st.qkv[0]
    q, kk = (torch.empty((5 * frame, n, 128), dtype=torch.float16, device="cuda") for n in (6, 2))
    st.h.packed_norm_rope(rows[:, :6], rows[:, 6:8], st.positions, *st.w, EPS, q_out=q, k_out=kk)
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = st.h.packed_plan(cu(0, frame), cu(0, 5 * frame), frame, 5 * frame, 2, frame)
    want = torch.empty_like(out)
    ws = torch.empty(st.h.packed_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    st.h.packed_forward(plan, q[4 * frame:], kk, rows[:, 8:], want, workspace=ws)
    st.h.sync()
    ref, _, bo, _ = R.attention(q[4 * frame:], kk, rows[:, 8:], [frame], [5 * frame], frame)
    R.assert_within(want, ref, bo, "over rows")
    R.assert_within(out, ref, bo, "over pages")

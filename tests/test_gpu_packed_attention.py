"""Attention over packed sequences against the definition in 64 bits: grouped
heads, masks, ragged and empty sequences, new tokens over long key ranges,
strides, garbage outside the sequences, captured graphs and bad plans."""
import pytest

from . import packed_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Batch:
    """Inputs of a packed batch between NaN rows, and its plan."""

    def __init__(self, q_lens, k_lens, H, Hkv, block, qk="f16", seed=0, pad=3, std=1.0, fused=False):
        from video_dit_long_gb300 import k6attn as K
        self.K, self.q_lens, self.k_lens, self.H, self.Hkv, self.block, self.pad = K, q_lens, k_lens, H, Hkv, block, pad
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = torch.float16 if qk == "f16" else torch.bfloat16

        def rows(n, heads, dtype, std=1.0):
            x = torch.full((n + 2 * pad, heads, 128), NAN, dtype=dtype, device="cuda")
            x[pad:pad + n] = (torch.randn((n, heads, 128), generator=g, device="cuda") * std).to(dtype)
            return x

        nq, nk = sum(q_lens), sum(k_lens)
        if fused:  # q, k, v as parts of one projection
            x = rows(nq, H + 2 * Hkv, torch.bfloat16, std)
            self.q, self.k, self.v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        else:
            self.q, self.k, self.v = rows(nq, H, t, std), rows(nk, Hkv, t, std), rows(nk, Hkv, torch.bfloat16)
        self.dout = rows(nq, H, torch.bfloat16)
        cu = lambda lens: (torch.tensor([0] + lens).cumsum(0) + pad).to(torch.int32).cuda()  # noqa: E731
        self.cu_q, self.cu_k = cu(q_lens), cu(k_lens)
        self.h = K.Handle.for_packed(H)
        self.plan = self.h.packed_plan(self.cu_q, self.cu_k, nq + 2 * pad, nk + 2 * pad, Hkv, block)
        self.out = torch.full((nq + 2 * pad, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((H, nq + 2 * pad), 7.0, device="cuda")
        self.ws = torch.full((self.h.packed_workspace_bytes(self.plan),), 255, dtype=torch.uint8, device="cuda")

    def forward(self):
        self.h.packed_forward(self.plan, self.q, self.k, self.v, self.out, self.lse, workspace=self.ws)
        return self

    def check(self):
        self.h.sync()
        a, n = self.pad, self.out.shape[0] - self.pad
        ref, rl, bo, bl = R.attention(self.q, self.k, self.v, self.q_lens, self.k_lens, self.block, a, a)
        R.assert_within(self.out[a:n], ref[a:n], bo[a:n], "out")
        R.assert_within(self.lse[:, a:n], rl[:, a:n], bl[:, a:n], "lse")
        for x in (self.out[:a], self.out[n:], self.lse[:, :a], self.lse[:, n:]):
            assert bool((x == 7.0).all())  # rows outside the sequences
        return self


SHAPES = [
    ([1], [1]), ([128], [128]), ([127, 129, 1], [127, 129, 1]), ([0, 5, 0, 300], [0, 5, 0, 300]),
    ([77, 1, 130, 43], [77, 1, 130, 43]),
]


@pytest.mark.parametrize("lens", SHAPES)
@pytest.mark.parametrize("H,Hkv", [(6, 1), (6, 2), (4, 4), (8, 2)])
@pytest.mark.parametrize("block", [0, 1, 50])
def test_same_lengths(lens, H, Hkv, block):
    Batch(*lens, H, Hkv, block, seed=1).forward().check()


@pytest.mark.parametrize("lens", [([1, 3, 200, 5, 64], [700, 3, 64, 0, 400]), ([300, 0, 2], [10, 40, 1])])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 6])
@pytest.mark.parametrize("block", [0, 1, 7, 256])
@pytest.mark.parametrize("qk", ["f16", "bf16"])
def test_other_lengths(lens, Hkv, block, qk):
    """New tokens over kept keys, more queries than keys (rows that see nothing), no keys at all."""
    Batch(*lens, 6, Hkv, block, qk=qk, seed=2).forward().check()


@pytest.mark.parametrize("H,Hkv", [(24, 1), (24, 4), (5, 1), (128, 1), (7, 7)])
def test_head_groups(H, Hkv):
    Batch([40, 9], [40, 300], H, Hkv, 1, seed=3).forward().check()


@pytest.mark.parametrize("q_lens,k_lens,Hkv", [([1], [9000], 1), ([1, 1, 1], [5000, 1, 1300], 2), ([3, 2], [4097, 8192], 4),
                                               ([200], [6000], 4)])
@pytest.mark.parametrize("block", [0, 1])
def test_long_key_ranges_are_split_and_joined(q_lens, k_lens, Hkv, block):
    b = Batch(q_lens, k_lens, 8, Hkv, block, seed=4).forward().check()
    assert b.ws.numel() > 0
    first = b.out.clone(), b.lse.clone()
    b.h.packed_replan(b.plan, b.cu_q, b.cu_k)
    b.forward().h.sync()
    assert torch.equal(first[0], b.out) and torch.equal(first[1], b.lse)


def test_many_short_sequences():
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    Batch(lens, lens, 3, 1, 1, seed=5).forward().check()


def test_more_sequences_than_one_block_plans():
    """Past 1,024 sequences the batch is not cut into stretches but dealt out from a sorted list; a long key range of a
    few queries among them is split all the same."""
    g = torch.Generator().manual_seed(1)
    q = torch.randint(0, 9, (1500,), generator=g).tolist()
    k = [x + (x % 3) for x in q]
    q[700], k[700] = 2, 20_000
    q[3], k[3] = 300, 310
    b = Batch(q, k, 4, 2, 1, seed=17).forward().check()
    first = b.out.clone(), b.lse.clone()
    b.h.packed_replan(b.plan, b.cu_q, b.cu_k)
    b.forward().h.sync()
    assert torch.equal(first[0], b.out) and torch.equal(first[1], b.lse)


def test_a_batch_too_large_for_stretches():
    """30 sequences of 512 tokens and one of 9,000, 24 heads: more than 256 key tiles a SM, dealt out by load; checked against its own parts."""
    lens = [512] * 30 + [9000]
    b = Batch(lens, lens, 24, 24, 1, seed=18)
    b.forward().h.sync()
    part = slice(b.pad + 512 * 7, b.pad + 512 * 8)
    ref, rl, bo, bl = R.attention(b.q[part], b.k[part], b.v[part], [512], [512], 1)
    R.assert_within(b.out[part], ref, bo, "out")
    R.assert_within(b.lse[:, part], rl, bl, "lse")
    last = slice(b.pad + 512 * 30, b.pad + 512 * 30 + 9000)
    h = 17  # one head of the long sequence, its last 100 queries
    ref, rl, bo, bl = R.attention(b.q[last, h:h + 1][-100:], b.k[last, h:h + 1], b.v[last, h:h + 1], [100], [9000], 1)
    R.assert_within(b.out[last, h:h + 1][-100:], ref, bo, "out")
    assert bool((b.out[:b.pad] == 7.0).all()) and bool(b.out[b.pad:-b.pad].isfinite().all())


def test_no_query_rows_or_no_key_rows():
    from video_dit_long_gb300 import k6attn as K
    h = K.Handle.for_packed(4)
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    e = lambda n, heads, t=torch.bfloat16: torch.full((n, heads, 128), 3.0, dtype=t, device="cuda")  # noqa: E731
    p = h.packed_plan(cu(0, 0), cu(0, 5), 0, 5, 2)
    h.packed_forward(p, e(0, 4), e(5, 2), e(5, 2), e(0, 4), torch.empty((4, 0), device="cuda"))
    ws = torch.empty(h.packed_backward_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    dk, dv = e(5, 2), e(5, 2)
    h.packed_backward(p, e(0, 4), e(5, 2), e(5, 2), e(0, 4), e(0, 4), torch.empty((4, 0), device="cuda"), e(0, 4), dk, dv,
                      workspace=ws)
    h.sync()
    assert not dk.any() and not dv.any()
    p = h.packed_plan(cu(0, 5), cu(0, 0), 5, 0, 2)
    out, lse = e(5, 4), torch.zeros((4, 5), device="cuda")
    h.packed_forward(p, e(5, 4), e(0, 2), e(0, 2), out, lse)
    ws = torch.empty(h.packed_backward_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    dq = e(5, 4)
    h.packed_backward(p, e(5, 4), e(0, 2), e(0, 2), out, e(5, 4), lse, dq, e(0, 2), e(0, 2), workspace=ws)
    h.sync()
    assert not out.any() and bool((lse == -float("inf")).all()) and not dq.any()
    p = h.packed_plan(cu(0, 0), None, 0, 0, 2)
    h.packed_forward(p, e(0, 4), e(0, 2), e(0, 2), e(0, 4))
    h.sync()


def test_two_calls_at_once_on_two_streams():
    """One plan, two streams, a workspace each."""
    a, b = Batch([3, 200], [6000, 200], 8, 4, 1, seed=19), Batch([3, 200], [6000, 200], 8, 4, 1, seed=20)
    a.forward().h.sync()
    b.forward().h.sync()
    want = a.out.clone(), b.out.clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                x.out.fill_(7.0)
                x.h.packed_forward(a.plan, x.q, x.k, x.v, x.out, x.lse, workspace=x.ws)
    torch.cuda.synchronize()
    a.h.sync()
    b.h.sync()
    for x, y in zip((a, b), want):
        n = slice(x.pad, x.out.shape[0] - x.pad)
        assert torch.equal(x.out[n], y[n])


def test_parts_of_a_fused_projection():
    Batch([150, 60], [150, 60], 6, 2, 1, qk="bf16", seed=6, fused=True).forward().check()


def test_large_and_equal_logits():
    # logits up to a few hundred: the running maximum moves, most weights vanish
    Batch([300], [300], 4, 2, 1, seed=7, std=6.0).forward().check()
    b = Batch([100], [1000], 4, 2, 0, seed=8)
    b.q.fill_(0.0)  # every key alike: lse = log(1000)
    b.forward().check()


def test_infinite_and_nan_queries_stay_in_their_rows():
    b = Batch([200, 100], [200, 100], 4, 2, 1, seed=9)
    b.forward().h.sync()
    want = b.out.clone()
    b.q[b.pad + 17, 1] = NAN
    b.q[b.pad + 90, 2, 3] = float("inf")
    b.forward().h.sync()
    assert bool(b.out[b.pad + 17, 1].isnan().all()) and bool(b.out[b.pad + 90, 2].isnan().all())
    b.out[b.pad + 17, 1], b.out[b.pad + 90, 2] = want[b.pad + 17, 1], want[b.pad + 90, 2]
    assert torch.equal(b.out, want)


def test_a_sequence_of_nan_leaves_the_others_alone():
    b = Batch([60, 70, 200], [60, 70, 200], 4, 2, 0, seed=10).forward()
    b.h.sync()
    want, lse = b.out.clone(), b.lse.clone()
    s = slice(b.pad + 60, b.pad + 130)
    for x in (b.q, b.k, b.v):
        x[s] = NAN
    b.forward().h.sync()
    assert bool(b.out[s].isnan().all())
    for x, y in ((b.out, want), (b.lse.T, lse.T)):
        assert torch.equal(x[:s.start], y[:s.start]) and torch.equal(x[s.stop:], y[s.stop:])


def test_rows_past_four_gigabytes():
    """Token strides and rows whose byte offsets pass 32 bits, at the end of 4.9 GB tensors."""
    from video_dit_long_gb300 import k6attn as K
    T, wide, n = 600_000, 32, 333
    x = torch.empty((T, wide, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)
    x[T - n:] = torch.randn((n, wide, 128), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:8]
    cu = torch.tensor([T - n, T - 100, T], dtype=torch.int32, device="cuda")
    h = K.Handle.for_packed(4)
    plan = h.packed_plan(cu, None, T, T, 2, 1)
    out = x[:, 8:12]
    lse = torch.zeros((4, T), device="cuda")
    ws = torch.empty(h.packed_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    h.packed_forward(plan, q, k, v, out, lse, workspace=ws)
    h.sync()
    s = slice(T - n, T)
    ref, rl, bo, bl = R.attention(q[s], k[s], v[s], [n - 100, 100], [n - 100, 100], 1)
    R.assert_within(out[s], ref, bo, "out")
    R.assert_within(lse[:, s], rl, bl, "lse")


def test_captured_with_its_plan_and_on_another_stream():
    """A graph that plans and attends, replayed with other offsets; and the same calls on a stream of their own."""
    b = Batch([90, 200], [90, 200], 4, 2, 1, seed=12)
    b.forward().check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.h.packed_replan(b.plan, b.cu_q, b.cu_k)
        b.forward()
    for lens in ([290, 0], [1, 289], [100, 190]):
        b.q_lens = b.k_lens = lens
        b.cu_q.copy_((torch.tensor([0] + lens).cumsum(0) + b.pad).to(torch.int32))
        b.cu_k.copy_(b.cu_q)
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        graph.replay()
        b.check()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        b.h.packed_replan(b.plan, b.cu_q, b.cu_k)
        b.forward()
        b.check()


def test_bad_offsets_and_plans_are_reported_and_write_nothing():
    b = Batch([90, 200], [90, 200], 4, 2, 1, seed=13)
    K = b.K
    for bad in ([3, 200, 100], [-1, 50, 100], [0, 50, 10_000]):
        b.cu_q.copy_(torch.tensor(bad, dtype=torch.int32))
        b.h.packed_replan(b.plan, b.cu_q, b.cu_k)
        b.forward()
        with pytest.raises(K.K6Error) as e:
            b.h.sync()
        assert e.value.status == K.ERR_INVALID_ARG
        assert bool((b.out == 7.0).all()) and bool((b.lse == 7.0).all())
    # a plan that was never made, and one made for another mask
    for other in (0, 5):
        p = b.h.packed_plan(b.cu_k, None, b.out.shape[0], b.out.shape[0], 2, other)
        if other == 0:
            p.buffer.zero_()
        else:
            p.batch.mask_block = 1
        b.h.packed_forward(p, b.q, b.k, b.v, b.out, b.lse, workspace=b.ws)
        with pytest.raises(K.K6Error) as e:
            b.h.sync()
        assert e.value.status == K.ERR_INVALID_ARG
        assert bool((b.out == 7.0).all())


def test_a_wait_limit_of_zero_gives_up():
    b = Batch([90, 200], [90, 200], 4, 2, 1, seed=14)
    b.h.set_option(b.K.OPT_WAIT_LIMIT_NS, 0)
    b.forward()
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_TIMEOUT
    b.h.set_option(b.K.OPT_WAIT_LIMIT_NS, 2_000_000_000)
    b.forward().check()


def test_lse_may_be_left_out():
    b = Batch([90, 200], [90, 200], 4, 2, 1, seed=15).forward()
    want = b.out.clone()
    b.out.fill_(7.0)
    b.h.packed_forward(b.plan, b.q, b.k, b.v, b.out, workspace=b.ws)
    b.h.sync()
    assert torch.equal(b.out, want)


def test_refusals():
    b = Batch([90], [90], 4, 2, 1, seed=16)
    K, h = b.K, b.h
    with pytest.raises(ValueError):
        h.packed_forward(b.plan, b.q[:, :3], b.k, b.v, b.out, b.lse, workspace=b.ws)
    with pytest.raises(ValueError):
        h.packed_forward(b.plan, b.q, b.k.to(torch.bfloat16), b.v, b.out, b.lse, workspace=b.ws)
    with pytest.raises(ValueError):
        h.packed_forward(b.plan, b.q.cpu(), b.k, b.v, b.out, b.lse, workspace=b.ws)
    with pytest.raises(ValueError):
        h.packed_forward(b.plan, b.q, b.k, b.v.transpose(0, 1).contiguous().transpose(0, 1), b.out, b.lse, workspace=b.ws)
    big = Batch([1], [4000], 4, 2, 1, seed=16)
    with pytest.raises(K.K6Error) as e:
        h.packed_forward(big.plan, big.q, big.k, big.v, big.out, big.lse, workspace=big.ws[:16])
    assert e.value.status == K.ERR_WORKSPACE
    for kw in (dict(kv_heads=3), dict(mask_block=-1)):
        with pytest.raises(K.K6Error) as e:
            h.packed_plan(b.cu_q, b.cu_k, 96, 96, **{"kv_heads": 2, **kw})
        assert e.value.status == K.ERR_INVALID_ARG
    f32 = K.Handle.for_packed(4, 64, "f32", (16, 24, 24))
    with pytest.raises(K.K6Error):
        f32.packed_plan(b.cu_q, b.cu_k, 96, 96, 2)
    with pytest.raises(K.K6Error) as e:  # the output over an input
        h.packed_forward(b.plan, b.out, b.k.to(torch.bfloat16), b.v, b.out, b.lse, workspace=b.ws)
    assert e.value.status == K.ERR_INVALID_ARG


@pytest.mark.parametrize("as_pointer", [False, True])
def test_a_plan_made_on_a_stream_of_its_own(as_pointer):
    """The plan's memory belongs to the stream that is given: work still running on the current one cannot reach it."""
    from video_dit_long_gb300 import k6attn as K
    H, kv, L = 2, 1, 200
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((L, n, 128), generator=g, device="cuda").to(torch.bfloat16) for n in (H, kv, kv))
    cu = torch.tensor([0, 80, L], dtype=torch.int32, device="cuda")
    h = K.Handle.for_packed(H)
    want, out = torch.empty_like(q), torch.empty_like(q)
    plan = h.packed_plan(cu, None, L, L, kv, 1)
    h.packed_forward(plan, q, k, v, want, workspace=torch.empty(h.packed_workspace_bytes(plan), dtype=torch.uint8,
                                                                device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    room = torch.empty(plan.buffer.numel(), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        room.random_(0, 255)  # on the current stream; freed while it runs
        del room
        s = side.cuda_stream if as_pointer else side
        mine = h.packed_plan(cu, None, L, L, kv, 1, stream=s)
        h.packed_forward(mine, q, k, v, out, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), stream=s)
        h.sync(s)
        assert torch.equal(out, want)
        room = torch.empty(plan.buffer.numel(), dtype=torch.uint8, device="cuda")


def off16(t):
    """A copy of t whose first element lies 16 bytes behind a 32-byte boundary."""
    n, skip = t.numel(), 16 // t.element_size()
    x = torch.empty(n + skip, dtype=t.dtype, device="cuda")[skip:].view(t.shape)
    assert n == 0 or x.data_ptr() % 32 == 16
    return x.copy_(t)


@pytest.mark.parametrize("q_lens,k_lens", [([1, 1, 3], [5000, 300, 4097]), ([130, 60], [130, 60])])
def test_everything_sixteen_byte_aligned_only(q_lens, k_lens):
    """The alignment that the library asks for, on every tensor and workspace, split key ranges included."""
    want = Batch(q_lens, k_lens, 4, 2, 1, seed=61).forward()
    b = Batch(q_lens, k_lens, 4, 2, 1, seed=61)
    b.q, b.k, b.v, b.out, b.lse, b.ws = (off16(x) for x in (b.q, b.k, b.v, b.out, b.lse, b.ws))
    b.plan.buffer = off16(b.plan.buffer)
    b.plan.ptr = b.plan.buffer.data_ptr()
    b.forward().check()
    assert torch.equal(b.out[3:-3], want.out[3:-3]) and torch.equal(b.lse[:, 3:-3], want.lse[:, 3:-3])
    grads = []
    for x in (want, b):
        o = [torch.zeros_like(x.q, dtype=torch.bfloat16), torch.zeros_like(x.v), torch.zeros_like(x.v)]
        room = torch.empty(x.h.packed_backward_workspace_bytes(x.plan), dtype=torch.uint8, device="cuda")
        dout = x.dout
        if x is b:
            o, room, dout = [off16(y) for y in o], off16(room), off16(dout)
        x.h.packed_backward(x.plan, x.q, x.k, x.v, x.out, dout, x.lse, *o, workspace=room)
        x.h.sync()
        grads.append([y[3:-3] for y in o])
    for x, y in zip(*grads):
        assert torch.equal(x, y)


@pytest.mark.parametrize("Hkv", [4, 1])
def test_a_plan_of_a_smaller_batch_is_reported_and_nothing_is_written(Hkv):
    """A call whose batch has more sequences, tokens and split tiles than the plan it is given was made for: its lists
    would lie behind the end of that plan, in memory that holds anything."""
    small, big = Batch([1], [1], 4, 4, 1, seed=62), Batch([1, 200], [9000, 5000], 4, Hkv, 1, seed=63)
    assert small.plan.buffer.numel() < big.plan.buffer.numel() and big.ws.numel() > 0
    room = torch.full_like(big.plan.buffer, 255)
    room[:small.plan.buffer.numel()] = small.plan.buffer
    p = big.K.PackedPlan(big.plan.batch, room)
    big.h.packed_forward(p, big.q, big.k, big.v, big.out, big.lse, workspace=big.ws)
    with pytest.raises(big.K.K6Error) as e:
        big.h.sync()
    assert e.value.status == big.K.ERR_INVALID_ARG
    assert bool((big.out == 7.0).all()) and bool((big.lse == 7.0).all())
    grads = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (big.q, big.k, big.v)]
    ws = torch.empty(big.h.packed_backward_workspace_bytes(big.plan), dtype=torch.uint8, device="cuda")
    big.h.packed_backward(p, big.q, big.k, big.v, big.out, big.dout, big.lse, *grads, workspace=ws)
    with pytest.raises(big.K.K6Error) as e:
        big.h.sync()
    assert e.value.status == big.K.ERR_INVALID_ARG
    assert all(bool((x == 7.0).all()) for x in grads)
    big.forward().check()  # its own plan still serves


def test_a_batch_that_is_refused_keeps_its_status():
    """Planning: a type the library does not take is 'unsupported', a bad count an invalid argument."""
    from video_dit_long_gb300 import k6attn as K
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for h, kw, status in ((K.Handle.for_packed(4, 64, "f32", (16, 24, 24)), {}, K.ERR_UNSUPPORTED),
                          (K.Handle.for_packed(300), {"kv_heads": 1}, K.ERR_UNSUPPORTED),
                          (K.Handle.for_packed(4), {"kv_heads": 3}, K.ERR_INVALID_ARG),
                          (K.Handle.for_packed(4), {"mask_block": 1 << 30}, K.ERR_INVALID_ARG)):
        with pytest.raises(K.K6Error) as e:
            h.packed_plan(cu, None, 4, 4, **{"kv_heads": 2, **kw})
        assert e.value.status == status and "packed_plan" in str(e.value)

"""The packed calls together, as a layer makes them: norm and rotation, attention,
and their gradients, against one 64-bit computation of the whole."""
import pytest

from . import packed_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

AXES = (32, 48, 48)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def whole(qkv, positions, wq, wk, H, kv, lens, block, dout):
    """out and the gradients of sum(out * dout), differentiated through everything in float64."""
    x = qkv.double().view(qkv.shape[0], H + 2 * kv, 128).requires_grad_(True)
    wq, wk = wq.double().requires_grad_(True), wk.double().requires_grad_(True)
    q, _ = R.norm_rope(x[:, :H], wq, positions, AXES, 10000.0, 1e-6)
    k, _ = R.norm_rope(x[:, H:H + kv], wk, positions, AXES, 10000.0, 1e-6)
    outs = []
    for r, _ in R.sequences(lens, lens):
        L = r.stop - r.start
        hide = torch.arange(L, device="cuda")[None] >= R.limits(L, L, block, "cuda")[:, None]
        s = torch.einsum("ihd,jhd->hij", q[r], k[r].repeat_interleave(H // kv, 1)) / 128 ** 0.5
        p = torch.softmax(s.masked_fill(hide, -float("inf")), -1)
        outs.append(torch.einsum("hij,jhd->ihd", p, x[r, H + kv:].repeat_interleave(H // kv, 1)))
    out = torch.cat(outs)
    n = out.shape[0]
    return (out.detach(),) + torch.autograd.grad((out * dout[:n].double()).sum(), (x, wq, wk))


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("qk", ["f16", "bf16"])
@pytest.mark.parametrize("lens,block,H,kv", [([150, 1, 61], 1, 6, 2), ([40, 200], 50, 4, 4), ([97, 33], 0, 4, 1)])
def test_layer_forward_and_backward(qk, lens, block, H, kv):
    from video_dit_long_gb300 import k6attn as K
    from video_dit_long_gb300.packed import PackedAttention, PackedBatch
    g = torch.Generator(device="cuda").manual_seed(41)
    T = sum(lens) + 2  # two rows behind the last sequence
    qkv = torch.randn((T, (H + 2 * kv) * 128), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((T, H, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 60, (T, 3), generator=g, device="cuda").to(torch.int32)
    wq, wk = (torch.randn(128, generator=g, device="cuda") * 0.2 + 1 for _ in range(2))
    h = K.Handle.for_packed(H)
    batch = PackedBatch(h, lens, T, kv, block)
    layer = PackedAttention(batch, wq, wk, qk=qk)
    dqkv = torch.zeros_like(qkv)
    out = layer.forward(qkv, pos)
    dwq, dwk = layer.backward(dout, qkv, pos, dqkv)
    h.sync()
    ref, gx, gwq, gwk = whole(qkv, pos, wq, wk, H, kv, lens, block, dout)
    n = sum(lens)
    # Errors of independent roundings add in squares; as shares of the 2-norm, each at most its type's half step:
    # rotated q and k (u: 2^-11 or 2^-8) move logits of order 1, P and out 2^-8 each; backward, dS and P 2^-8, the
    # gradients of the rotated q and k 2^-8 and of qkv 2^-8, out in D 2^-8.  Below 4 * 2^-8 in all.
    assert rel(out[:n], ref) <= 4 * 2.0 ** -8
    dx = dqkv.view(T, H + 2 * kv, 128)
    for s in (slice(0, H), slice(H, H + kv), slice(H + kv, H + 2 * kv)):
        assert rel(dx[:n, s], gx[:n, s]) <= 4 * 2.0 ** -8, s
    assert not out[n:].any() and not dx[n:].any()
    # the weights' gradients: sums of the same terms, whose errors do not all cancel
    assert rel(dwq, gwq) <= 4 * 2.0 ** -8 and rel(dwk, gwk) <= 4 * 2.0 ** -8


def test_a_captured_layer_follows_new_lengths():
    """Forward and backward in one graph; new inputs and lengths at replay, while the eager layer's results live."""
    from video_dit_long_gb300 import k6attn as K
    from video_dit_long_gb300.packed import PackedAttention, PackedBatch
    H, kv, T = 4, 2, 300
    g = torch.Generator(device="cuda").manual_seed(43)
    new = lambda: torch.randn((T, (H + 2 * kv) * 128), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    qkv, dout = new(), torch.randn((T, H, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 60, (T, 3), generator=g, device="cuda").to(torch.int32)
    wq, wk = torch.ones(128, device="cuda"), torch.ones(128, device="cuda")
    h = K.Handle.for_packed(H)

    def eager(x, lens):
        layer = PackedAttention(PackedBatch(h, lens, T, kv, 1), wq, wk)
        d = torch.zeros_like(x)
        layer.forward(x, pos)
        layer.backward(dout, x, pos, d)
        return layer, d

    keep = eager(qkv, [100, 200])
    batch = PackedBatch(h, [100, 200], T, kv, 1)
    layer, d = PackedAttention(batch, wq, wk), torch.zeros_like(qkv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.forward(qkv, pos)
        layer.backward(dout, qkv, pos, d)
    for lens in ([100, 200], [299, 1], [0, 300]):
        if lens != [100, 200]:
            qkv.copy_(new())
        batch.set_offsets(torch.tensor([0] + lens).cumsum(0).to(torch.int32))
        graph.replay()
        want, wd = eager(qkv.clone(), lens)
        h.sync()
        assert torch.equal(layer.out, want.out) and torch.equal(d, wd)
        assert torch.equal(layer.dq_weight, want.dq_weight) and torch.equal(layer.dk_weight, want.dk_weight)
    assert keep[0].out.isfinite().all() and keep[1].isfinite().all()


def test_rows_behind_a_padded_batch_enter_nothing():
    """A batch padded with NaN, then one of fewer tokens in the same buffers: padding rows are left as they were, and
    the weights' gradients are those of the batch alone, to the bit."""
    from video_dit_long_gb300 import k6attn as K
    from video_dit_long_gb300.packed import PackedAttention, PackedBatch
    H, kv, T = 4, 2, 300
    g = torch.Generator(device="cuda").manual_seed(47)
    qkv = torch.randn((T, (H + 2 * kv) * 128), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((T, H, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 60, (T, 3), generator=g, device="cuda").to(torch.int32)
    wq, wk = torch.ones(128, device="cuda"), torch.ones(128, device="cuda")
    h = K.Handle.for_packed(H)
    given = torch.tensor([0, 120, 280], dtype=torch.int32, device="cuda")
    batch = PackedBatch(h, given, T, kv, 1)
    layer = PackedAttention(batch, wq, wk)
    for offsets in ([0, 120, 280], [3, 50, 90], [7, 7, 7]):
        lo, hi = offsets[0], offsets[-1]
        x, dy, d = (t.clone() for t in (qkv, dout, torch.full_like(qkv, 7.0)))
        for t in (x, dy):
            t[:lo], t[hi:] = float("nan"), float("nan")
        batch.set_offsets(torch.tensor(offsets, dtype=torch.int32))
        layer.forward(x, pos)
        layer.backward(dy, x, pos, d)
        h.sync()
        assert (d[:lo] == 7).all() and (d[hi:] == 7).all()
        alone = PackedAttention(PackedBatch(h, [b - a for a, b in zip(offsets, offsets[1:])], T, kv, 1), wq, wk)
        # the same rows at the same places, other rows zero
        z, dz, want = torch.zeros_like(qkv), torch.zeros_like(dout), torch.zeros_like(qkv)
        z[:hi - lo], dz[:hi - lo] = qkv[lo:hi], dout[lo:hi]
        p = torch.zeros_like(pos)
        p[:hi - lo] = pos[lo:hi]
        alone.forward(z, p)
        alone.backward(dz, z, p, want)
        h.sync()
        assert torch.equal(d[lo:hi], want[:hi - lo]) and torch.equal(layer.out[lo:hi], alone.out[:hi - lo])
        # sums over the tokens in another order: fp32, n <= T H terms of the same sign structure
        for a, b in ((layer.dq_weight, alone.dq_weight), (layer.dk_weight, alone.dk_weight)):
            assert a.isfinite().all()
            assert (a - b).abs().max() <= 2.0 ** -12 * max(1.0, float(b.abs().max()))
    assert given.tolist() == [0, 120, 280]  # the caller's own
    assert not layer.dq_weight.any() and not layer.dk_weight.any()  # of no token

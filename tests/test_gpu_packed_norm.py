"""Per-head QK-norm with multi-axis rotary positions on packed token rows, and its
gradient, against the definition in 64 bits."""
import pytest

from . import packed_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

AXES = {128: (32, 48, 48), 64: (16, 24, 24)}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(T, H, Hkv, d, dtype, seed=0, far=False, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((T, H + 2 * Hkv, d), generator=g, device="cuda") * std).to(dtype)
    lo, hi = (-2 ** 31, 2 ** 31) if far else (0, 300)
    pos = torch.randint(lo, hi, (T, 3), generator=g, device="cuda").to(torch.int32)
    wq, wk = (torch.randn(d, generator=g, device="cuda") * 0.2 + 1 for _ in range(2))
    return x, pos, wq, wk, g


def bound(ref, mag, t):
    # r to 2^-21.4 (sum of d squares, rsqrt), three products 2^-24 each, cos and sin to 2^-22, the rotation's two
    # products and sum: below 2^-19 of the pair's norm; then the output's rounding, and fp16's last step 2^-25
    return (2.0 ** -19 * mag) * (1 + R.HALF[t]) + R.HALF[t] * ref.abs() + (2.0 ** -25 if t == torch.float16 else 0.0)


SHAPES = [(1, 2, 1, 128), (8, 24, 8, 128), (257, 6, 2, 128), (3001, 5, 3, 128), (97, 4, 4, 64), (5000, 3, 1, 64)]


@pytest.mark.parametrize("T,H,Hkv,d", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "f16"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(T, H, Hkv, d, dtype, out, norm):
    from video_dit_long_gb300 import k6attn as K
    if dtype == "bf16" and d != 128:
        pytest.skip("bf16 handles have d = 128")
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    to = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}[out]
    x, pos, wq, wk, _ = make(T, H, Hkv, d, t, far=T == 257)
    if not norm:
        wq = wk = None
    h = K.Handle.for_packed(H, d, dtype, AXES[d])
    q, k = x[:, :H], x[:, H:H + Hkv]  # parts of a fused projection
    buf = torch.full((T, H + Hkv + 1, d), 7.0, dtype=to, device="cuda")
    h.packed_norm_rope(q, k, pos, wq, wk, 1e-6, q_out=buf[:, :H], k_out=buf[:, H:H + Hkv])
    h.sync()
    for got, src, w in ((buf[:, :H], q, wq), (buf[:, H:H + Hkv], k, wk)):
        ref, mag = R.norm_rope(src, w, pos, AXES[d], 10000.0, 1e-6)
        R.assert_within(got, ref, bound(ref, mag, to))
    assert bool((buf[:, H + Hkv:] == 7.0).all())  # the rest of the rows is left alone


@pytest.mark.parametrize("T,H,Hkv,d", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope_backward(T, H, Hkv, d, dtype, norm):
    from video_dit_long_gb300 import k6attn as K
    if dtype == "bf16" and d != 128:
        pytest.skip("bf16 handles have d = 128")
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x, pos, wq, wk, g = make(T, H, Hkv, d, t, seed=3, far=T == 257)
    if not norm:
        wq = wk = None
    gz = torch.randn((T, H + Hkv, d), generator=g, device="cuda").to(t)
    h = K.Handle.for_packed(H, d, dtype, AXES[d])
    dx = torch.full((T, H + 2 * Hkv, d), 7.0, dtype=t, device="cuda")
    dwq, dwk = (torch.full((d,), 7.0, device="cuda") if norm else None for _ in range(2))
    ws = torch.empty(h.packed_norm_rope_backward_workspace_bytes(T, Hkv), dtype=torch.uint8, device="cuda")

    def run():
        h.packed_norm_rope_backward(gz[:, :H], gz[:, H:], x[:, :H] if norm else None, x[:, H:H + Hkv] if norm else None,
                                    pos, wq, wk, 1e-6, dq=dx[:, :H], dk=dx[:, H:H + Hkv], dq_weight=dwq,
                                    dk_weight=dwk, workspace=ws if norm else None)
        h.sync()

    run()
    for s, w, dw in ((slice(0, H), wq, dwq), (slice(H, H + Hkv), wk, dwk)):
        ref, rw, mag, magw = R.norm_rope_grads(x[:, s], w, pos, AXES[d], 10000.0, 1e-6, gz[:, s])
        # as the forward pass, with the mean of 128 products besides: 2^-18 of the magnitudes
        R.assert_within(dx[:, s], ref, 2.0 ** -18 * mag + R.HALF[t] * (ref.abs() + 2.0 ** -18 * mag), "dx")
        if norm:
            # each term to 2^-19; a lane adds at most 64 + its share of the terms in fp32 one after another, the
            # joins add 2^-24 each: below 2^-24 * (number of adds) of the sum of magnitudes, 2^-13 is far above
            R.assert_within(dw, rw, 2.0 ** -13 * magw * 2.0 ** -2, "dw")
    assert bool((dx[:, H + Hkv:] == 7.0).all())
    if norm:
        first = dwq.clone(), dwk.clone(), dx.clone()
        run()
        assert torch.equal(first[0], dwq) and torch.equal(first[1], dwk) and torch.equal(first[2], dx)


def test_gradient_against_differences():
    """The fp32 backward against central differences of the fp32 forward, along random directions."""
    from video_dit_long_gb300 import k6attn as K
    T, H, Hkv, d = 5, 2, 1, 64
    x, pos, wq, wk, g = make(T, H, Hkv, d, torch.float32, seed=5)
    gz = torch.randn((T, H + Hkv, d), generator=g, device="cuda")
    h = K.Handle.for_packed(H, d, "f32", AXES[d])

    def loss(q, k, wq, wk):
        z = torch.empty((T, H + Hkv, d), device="cuda")
        h.packed_norm_rope(q, k, pos, wq, wk, 1e-3, q_out=z[:, :H], k_out=z[:, H:])
        return (z.double() * gz.double()).sum()

    q, k = x[:, :H].contiguous(), x[:, H:H + Hkv].contiguous()
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dwq, dwk = torch.empty_like(wq), torch.empty_like(wk)
    ws = torch.empty(h.packed_norm_rope_backward_workspace_bytes(T, Hkv), dtype=torch.uint8, device="cuda")
    h.packed_norm_rope_backward(gz[:, :H], gz[:, H:], q, k, pos, wq, wk, 1e-3, dq=dq, dk=dk, dq_weight=dwq,
                                dk_weight=dwk, workspace=ws)
    args, grads, step = [q, k, wq, wk], [dq, dk, dwq, dwk], 2.0 ** -7
    for i in range(4):
        dirn = torch.randn(args[i].shape, generator=g, device="cuda")
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * dirn, args[i] - step * dirn
        num = float((loss(*up) - loss(*down)) / (2 * step))
        ana = float((grads[i].double() * dirn.double()).sum())
        # forward values of order 1 to 2^-19 each: about 1000 of them over 2 steps, sqrt(1000) * 2^-19 * 64 = 4e-3;
        # third derivatives times step^2 / 6: of order 1e-5 of the gradient's sum of magnitudes
        tol = 4e-3 + 1e-4 * float((grads[i].abs() * dirn.abs()).sum())
        assert abs(num - ana) <= tol, (i, num, ana, tol)


def test_in_place_and_zero_tokens():
    from video_dit_long_gb300 import k6attn as K
    x, pos, wq, wk, g = make(50, 4, 2, 128, torch.bfloat16, seed=8)
    h = K.Handle.for_packed(4)
    want = torch.empty((50, 6, 128), dtype=torch.bfloat16, device="cuda")
    h.packed_norm_rope(x[:, :4], x[:, 4:6], pos, wq, wk, q_out=want[:, :4], k_out=want[:, 4:])
    h.packed_norm_rope(x[:, :4], x[:, 4:6], pos, wq, wk, q_out=x[:, :4], k_out=x[:, 4:6])
    h.sync()
    assert torch.equal(x[:, :6], want)
    e = lambda n: torch.empty((0, n, 128), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    p0 = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    h.packed_norm_rope(e(4), e(2), p0, wq, wk, q_out=e(4), k_out=e(2))
    dwq, dwk = torch.ones(128, device="cuda"), torch.ones(128, device="cuda")
    h.packed_norm_rope_backward(e(4), e(2), e(4), e(2), p0, wq, wk, dq=e(4), dk=e(2), dq_weight=dwq, dk_weight=dwk)
    h.sync()
    assert not dwq.any() and not dwk.any()
    # gradients over their own gradients
    gz = torch.randn((50, 6, 128), generator=g, device="cuda").to(torch.bfloat16)
    ws = torch.empty(h.packed_norm_rope_backward_workspace_bytes(50, 2), dtype=torch.uint8, device="cuda")
    d = torch.empty_like(gz)
    for dst in (d, gz):
        h.packed_norm_rope_backward(gz[:, :4], gz[:, 4:], x[:, :4], x[:, 4:6], pos, wq, wk, dq=dst[:, :4],
                                    dk=dst[:, 4:], dq_weight=dwq, dk_weight=dwk, workspace=ws)
    h.sync()
    assert torch.equal(d, gz)


def test_out_of_range_and_nan():
    from video_dit_long_gb300 import k6attn as K
    x, pos, wq, wk, _ = make(4, 2, 2, 128, torch.bfloat16, seed=9)
    h = K.Handle.for_packed(2)
    qo = torch.empty((4, 2, 128), dtype=torch.float16, device="cuda")
    ko = torch.empty_like(qo)
    big = x[:, :2] * 1e5  # without the norm, beyond fp16
    h.packed_norm_rope(big, x[:, 2:4], pos, q_out=qo, k_out=ko)
    with pytest.raises(K.K6Error) as e:
        h.sync()
    assert e.value.status == K.ERR_RANGE
    h.packed_norm_rope(big, x[:, 2:4], pos, wq, wk, q_out=qo, k_out=ko)  # the norm brings it back
    h.sync()
    # a NaN stays in its head row
    x[1, 0, 5] = float("nan")
    o = torch.empty((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    o2 = torch.empty_like(o)
    h.packed_norm_rope(x[:, :2], x[:, 2:4], pos, wq, wk, q_out=o, k_out=o2)
    h.sync()
    assert bool(o[1, 0].isnan().all()) and int(o.isnan().sum()) == 128 and not o2.isnan().any()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("lo,hi", [(0, 5), (2, 40), (39, 40), (17, 17), (9, 3)])
def test_offsets_bound_the_tokens(dtype, d, lo, hi):
    """With offsets only the tokens between the first and the last are read and written: the others may hold NaN, and
    the results are those of the same tokens alone."""
    from video_dit_long_gb300 import k6attn as K
    T, H, kv, axes = 40, 3, 1, {128: (32, 48, 48), 64: (16, 24, 24)}[d]
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, gq, gk = (torch.randn((T, n, d), generator=g, device="cuda").to(t) for n in (H, kv, H, kv))
    pos = torch.randint(-9, 90, (T, 3), generator=g, device="cuda").to(torch.int32)
    wq, wk = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    h = K.Handle.for_packed(H, d, dtype, axes)
    cu = torch.tensor([lo, min(lo, hi), hi], dtype=torch.int32, device="cuda")
    room = lambda n: torch.empty(h.packed_norm_rope_backward_workspace_bytes(n, kv), dtype=torch.uint8,  # noqa: E731
                                 device="cuda")

    def both(sel, offsets):
        n = q[sel].shape[0]
        a = [x[sel].clone() for x in (q, k, gq, gk)]
        if offsets is not None:
            for x in a:
                x[:lo], x[max(lo, hi):] = float("nan"), float("nan")
        o = [torch.full_like(x, 7.0) for x in a]
        dw = [torch.full((d,), 9.0, device="cuda") for _ in range(2)]
        h.packed_norm_rope(a[0], a[1], pos[sel], wq, wk, q_out=o[0], k_out=o[1], offsets=offsets)
        h.packed_norm_rope_backward(a[2], a[3], a[0], a[1], pos[sel], wq, wk, dq=o[2], dk=o[3], dq_weight=dw[0],
                                    dk_weight=dw[1], workspace=room(n), offsets=offsets)
        h.sync()
        return o, dw

    got, dw = both(slice(0, T), cu)
    want, dw1 = both(slice(lo, max(lo, hi)), None)
    for a, b in zip(got, want):
        assert torch.equal(a[lo:max(lo, hi)], b)
        assert (a[:lo] == 7).all() and (a[max(lo, hi):] == 7).all()
    # at most 120 fp32 terms, in another order: n 2^-24 (sum of their sizes) for each of the two, terms below 30
    for a, b in zip(dw, dw1):
        assert (a - b).abs().max() <= 2 * 120 * 2.0 ** -24 * 120 * 30


def test_shapes_of_positions_and_offsets_are_checked():
    from video_dit_long_gb300 import k6attn as K
    T = 8
    h = K.Handle.for_packed(2)
    x = torch.zeros((T, 4, 128), dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(x)
    call = lambda pos, **kw: h.packed_norm_rope(x[:, :2], x[:, 2:], pos, q_out=o[:, :2], k_out=o[:, 2:], **kw)  # noqa: E731
    pos = torch.zeros((T, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        call(pos.view(3, T))
    with pytest.raises(ValueError):
        call(pos, offsets=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(K.K6Error):
        call(pos, offsets=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(K.K6Error):
        call(pos, offsets=o.view(torch.int32).view(-1)[:2])  # an output

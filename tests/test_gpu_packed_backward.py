"""Gradients of packed attention against the formula in 64 bits and against
differences, and a whole packed layer step (norm and rotation, attention, and
back)."""
import pytest

from . import packed_ref as R
from .test_gpu_packed_attention import NAN, SHAPES, Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def backward(b):
    b.dq = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    b.dk = torch.full(b.k.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    b.dv = torch.full(b.k.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((b.h.packed_backward_workspace_bytes(b.plan),), 255, dtype=torch.uint8, device="cuda")
    b.h.packed_backward(b.plan, b.q, b.k, b.v, b.out, b.dout, b.lse, b.dq, b.dk, b.dv, workspace=ws)
    return b


def check(b):
    b.h.sync()
    a = b.pad
    refs, bounds = R.attention_grads(b.q, b.k, b.v, b.out, b.lse, b.dout, b.q_lens, b.k_lens, b.block, a, a)
    for got, ref, bound, what in zip((b.dq, b.dk, b.dv), refs, bounds, ("dq", "dk", "dv")):
        n = got.shape[0] - a
        R.assert_within(got[a:n], ref[a:n], bound[a:n], what)
        assert bool((got[:a] == 7.0).all()) and bool((got[n:] == 7.0).all())
    return b


@pytest.mark.parametrize("lens", SHAPES)
@pytest.mark.parametrize("H,Hkv", [(6, 1), (6, 2), (4, 4), (8, 2)])
@pytest.mark.parametrize("block", [0, 1, 50])
def test_same_lengths(lens, H, Hkv, block):
    check(backward(Batch(*lens, H, Hkv, block, seed=21).forward()))


@pytest.mark.parametrize("lens", [([1, 3, 200, 5, 64], [700, 3, 64, 0, 400]), ([300, 0, 2], [10, 40, 1])])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 6])
@pytest.mark.parametrize("block", [0, 1, 7, 256])
@pytest.mark.parametrize("qk", ["f16", "bf16"])
def test_other_lengths(lens, Hkv, block, qk):
    check(backward(Batch(*lens, 6, Hkv, block, qk=qk, seed=22).forward()))


@pytest.mark.parametrize("H,Hkv", [(24, 1), (24, 4), (5, 1), (128, 1), (7, 7)])
def test_head_groups(H, Hkv):
    check(backward(Batch([40, 9], [40, 300], H, Hkv, 1, seed=23).forward()))


def test_longer_and_the_same_bits_every_run():
    b = check(backward(Batch([1000, 333], [1500, 333], 6, 2, 100, seed=24).forward()))
    first = b.dq.clone(), b.dk.clone(), b.dv.clone()
    b.h.packed_replan(b.plan, b.cu_q, b.cu_k)
    backward(b).h.sync()
    for x, y in zip(first, (b.dq, b.dk, b.dv)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("qk", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** 40])
def test_small_and_large_gradients_keep_their_precision(qk, size):
    """dS is held in 16 bits; its range must follow dout's (the bounds are relative to the gradients)."""
    b = Batch([300, 40], [300, 40], 6, 2, 1, qk=qk, seed=25).forward()
    b.dout = (b.dout.float() * size).to(torch.bfloat16)
    check(backward(b))


def test_gradients_into_a_fused_buffer():
    b = Batch([150, 60], [150, 60], 6, 2, 1, qk="bf16", seed=26, fused=True).forward()
    want = check(backward(b))
    d = torch.full((b.q.shape[0], 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(b.h.packed_backward_workspace_bytes(b.plan), dtype=torch.uint8, device="cuda")
    b.h.packed_backward(b.plan, b.q, b.k, b.v, b.out, b.dout, b.lse, d[:, :6], d[:, 6:8], d[:, 8:], workspace=ws)
    b.h.sync()
    assert torch.equal(d[:, :6], want.dq) and torch.equal(d[:, 6:8], want.dk) and torch.equal(d[:, 8:], want.dv)


def test_a_sequence_of_nan_leaves_the_others_alone():
    b = backward(Batch([60, 70, 200], [60, 70, 200], 4, 2, 1, seed=27).forward())
    b.h.sync()
    want = b.dq.clone(), b.dk.clone(), b.dv.clone()
    s = slice(b.pad + 60, b.pad + 130)
    for x in (b.q, b.k, b.v, b.dout):
        x[s] = NAN
    backward(b.forward()).h.sync()
    for x, y in zip((b.dq, b.dk, b.dv), want):
        assert bool(x[s].isnan().all())
        assert torch.equal(x[:s.start], y[:s.start]) and torch.equal(x[s.stop:], y[s.stop:])


def test_gradient_against_differences():
    """Along random directions, against central differences of the 64-bit definition, at inputs the types hold."""
    b = check(backward(Batch([40, 9], [60, 9], 4, 2, 5, seed=28, pad=0).forward()))
    g = torch.Generator(device="cuda").manual_seed(29)

    def loss(q, k, v):
        return (R.attention(q, k, v, b.q_lens, b.k_lens, b.block)[0] * b.dout.double()).sum()

    args = [b.q.double(), b.k.double(), b.v.double()]
    for i, grad in enumerate((b.dq, b.dk, b.dv)):
        dirn = torch.randn(args[i].shape, dtype=torch.float64, generator=g, device="cuda")
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * dirn, args[i] - 1e-5 * dirn
        num = float((loss(*up) - loss(*down)) / 2e-5)
        ana = float((grad.double() * dirn).sum())
        # roundings of P, dS, out (in D) and of the gradient itself, each at most 2^-8 of a term and of either sign
        # over thousands of terms: 4 * 2^-8 of the 2-norm of the products
        tol = 2.0 ** -6 * float((grad.double() * dirn).norm())
        assert abs(num - ana) <= tol, (i, num, ana, tol)


def test_a_captured_backward_with_an_eager_one_alive():
    b = backward(Batch([90, 200], [90, 200], 4, 2, 1, seed=30).forward())
    b.h.sync()
    want = b.dq.clone(), b.dk.clone(), b.dv.clone()
    ws = torch.empty(b.h.packed_backward_workspace_bytes(b.plan), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.h.packed_backward(b.plan, b.q, b.k, b.v, b.out, b.dout, b.lse, b.dq, b.dk, b.dv, workspace=ws)
    for _ in range(2):
        for x in (b.dq, b.dk, b.dv):
            x.fill_(7.0)
        graph.replay()
        b.h.sync()
        for x, y in zip(want, (b.dq, b.dk, b.dv)):
            assert torch.equal(x, y)


def test_many_sequences():
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 30, (1300,), generator=g).tolist()
    check(backward(Batch(lens, lens, 3, 1, 1, seed=32).forward()))


def test_a_wait_limit_of_zero_gives_up():
    b = Batch([90, 200], [90, 200], 4, 2, 1, seed=33).forward()
    b.h.sync()
    b.h.set_option(b.K.OPT_WAIT_LIMIT_NS, 0)
    backward(b)
    with pytest.raises(b.K.K6Error) as e:
        b.h.sync()
    assert e.value.status == b.K.ERR_TIMEOUT
    b.h.set_option(b.K.OPT_WAIT_LIMIT_NS, 2_000_000_000)
    check(backward(b))


def test_workspace_and_plan_refusals():
    b = backward(Batch([90], [90], 4, 2, 1, seed=31).forward())
    K = b.K
    with pytest.raises(K.K6Error) as e:
        b.h.packed_backward(b.plan, b.q, b.k, b.v, b.out, b.dout, b.lse, b.dq, b.dk, b.dv, workspace=b.lse[:0])
    assert e.value.status == K.ERR_WORKSPACE
    ws = torch.empty(b.h.packed_backward_workspace_bytes(b.plan), dtype=torch.uint8, device="cuda")
    with pytest.raises(K.K6Error) as e:
        b.h.packed_backward(b.plan, b.q, b.k, b.v, b.out, b.dout, b.lse, b.dq, b.dk, b.dk, workspace=ws)
    assert e.value.status == K.ERR_INVALID_ARG
    b.h.sync()
    b.plan.buffer.zero_()
    b.dq.fill_(7.0)
    b.h.packed_backward(b.plan, b.q, b.k, b.v, b.out, b.dout, b.lse, b.dq, b.dk, b.dv, workspace=ws)
    with pytest.raises(K.K6Error) as e:
        b.h.sync()
    assert e.value.status == K.ERR_INVALID_ARG and bool((b.dq == 7.0).all())


@pytest.mark.parametrize("qk", ["f16", "bf16"])
@pytest.mark.parametrize("block", [0, 1])
def test_few_queries_over_long_caches(qk, block):
    check(backward(Batch([3, 1, 8], [9000, 20000, 4097], 8, 4, block, qk=qk, seed=34).forward()))


@pytest.mark.parametrize("qk", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** 66, 2.0 ** 100])
@pytest.mark.parametrize("block", [0, 1])
def test_gradients_whose_squares_leave_fp32(qk, size, block):
    """bf16 holds dout whose squared norm is 0 or infinite in fp32."""
    b = Batch([300, 40], [300, 40], 6, 2, block, qk=qk, seed=35).forward()
    b.dout = (b.dout.float() * size).to(torch.bfloat16)
    check(backward(b))


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** 66])
def test_values_whose_squares_leave_fp32(size):
    b = Batch([200, 40], [200, 40], 4, 2, 1, seed=36)
    b.v = (b.v.float() * size).to(torch.bfloat16)
    check(backward(b.forward()))

"""Gradients of very different sizes in one packed batch: dS of fp16 q and k is
held in 16 bits, and every gradient row must keep its precision beside rows and
sequences whose dout or v are many powers of two larger."""
import pytest

from . import packed_ref as R
from .test_gpu_packed_attention import Batch
from .test_gpu_packed_backward import backward

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = R.HALF


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def one_sequence(q, k, v, out, lse, dout, block):
    """(dq, dk, dv) of one sequence in 64 bits, and error bounds relative to each row's own gradients.

    A term of dS is rounded to its type (u of the term).  In fp16 it is at least 2^-24 after scaling, half of that
    lost at most, where 2^15 stands for twice the row's bound (2^14 for the rounding up of the exponent): 2^-25 / 2^14
    times twice max(|dO_i| |v_j|, |D_i|), i.e. 2^-38 of that maximum; over the keys of the sequence for a row of dq,
    over the queries that see the key, of all heads of its group, for a row of dk.  The rest as in
    packed_ref.attention_grads."""
    H, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    G, sc, Lq, Lk = H // Hkv, d ** -0.5, q.shape[0], k.shape[0]
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=q.device)  # noqa: E731
    dq, dk, dv, bq, bk, bv = z(q), z(k), z(k), z(q), z(k), z(k)
    fp16 = q.dtype == torch.float16
    u = HALF[torch.float16] if fp16 else HALF[torch.bfloat16]
    sees = torch.arange(Lk, device=q.device)[None] < R.limits(Lq, Lk, block, q.device)[:, None]
    for j in range(Hkv):
        kd, vd = k[:, j].double(), v[:, j].double()
        parts, top_k = [], torch.zeros(Lk, dtype=torch.float64, device=q.device)
        for h in range(j * G, (j + 1) * G):
            qd, od, gd = q[:, h].double(), out[:, h].double(), dout[:, h].double()
            D = (gd * od).sum(-1, keepdim=True)
            p = torch.exp(qd @ kd.T * sc - lse[h].double()[:, None].clamp(min=-1e300)).masked_fill(~sees, 0.0)
            ds = p * (gd @ vd.T - D)
            top = torch.maximum(gd.norm(dim=-1)[:, None] * vd.norm(dim=-1)[None], D.abs()).masked_fill(~sees, 0.0)
            top_k = torch.maximum(top_k, top.amax(0))
            e = (u + 2.0 ** -13) * ds.abs() + p * 2.0 ** -19 * (gd.abs() @ vd.abs().T + (gd * od).abs().sum(-1, keepdim=True))
            dq[:, h] = ds @ kd * sc
            # |v_j| is taken over all keys of the row's key tiles, hidden ones too
            most = torch.maximum(gd.norm(dim=-1) * vd.norm(dim=-1).max(), D.abs()[:, 0])
            bq[:, h] = (e + 2.0 ** -38 * most[:, None] * sees * fp16) @ kd.abs() * sc
            parts.append((qd, gd, p, ds, e))
        for qd, gd, p, ds, e in parts:
            dv[:, j] += p.T @ gd
            dk[:, j] += ds.T @ qd * sc
            bk[:, j] += (e + 2.0 ** -38 * top_k[None] * sees * fp16).T @ qd.abs() * sc
            bv[:, j] += (2.0 ** -8 + 2.0 ** -13) * (p.T @ gd.abs())
    half = HALF[torch.bfloat16]
    return (dq, dk, dv), tuple(b * (1 + 2.0 ** -7) + half * r.abs() for b, r in ((bq, dq), (bk, dk), (bv, dv)))


def check(b):
    b.h.sync()
    for n, (rq, rk) in enumerate(R.sequences(b.q_lens, b.k_lens, b.pad, b.pad)):
        if rq.start == rq.stop or rk.start == rk.stop:
            continue
        refs, bounds = one_sequence(b.q[rq], b.k[rk], b.v[rk], b.out[rq], b.lse[:, rq], b.dout[rq], b.block)
        for got, ref, bound, what in zip((b.dq[rq], b.dk[rk], b.dv[rk]), refs, bounds, ("dq", "dk", "dv")):
            R.assert_within(got, ref, bound, f"{what} of sequence {n}")


def scale_rows(x, start, by):
    """Rows of x from start on times the factors `by` (one per row), held in x's type."""
    rows = slice(start, start + len(by))
    f = torch.tensor(by, dtype=torch.float64, device="cuda")[:, None, None]
    x[rows] = (x[rows].double() * f).to(x.dtype)


@pytest.mark.parametrize("qk", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv", [(6, 2), (4, 4)])
@pytest.mark.parametrize("block", [0, 1, 50])
@pytest.mark.parametrize("down", [12, 30, 60])
def test_a_sequence_of_small_gradients_beside_a_large_one(qk, H, Hkv, block, down):
    b = Batch([150, 200, 60], [150, 200, 60], H, Hkv, block, qk=qk, seed=71).forward()
    scale_rows(b.dout, b.pad + 150, [2.0 ** -down] * 200)
    check(backward(b))


@pytest.mark.parametrize("block", [0, 1])
def test_a_sequence_of_small_values_beside_a_large_one(block):
    b = Batch([150, 200], [150, 200], 6, 2, block, seed=72)
    scale_rows(b.v, b.pad + 150, [2.0 ** -30] * 200)
    check(backward(b.forward()))


@pytest.mark.parametrize("lens", [([300], [300]), ([260, 9], [700, 400])])
@pytest.mark.parametrize("H,Hkv", [(6, 2), (4, 4), (24, 1)])
@pytest.mark.parametrize("block", [1, 7, 50, 200, 600])
def test_tokens_of_small_gradients_behind_large_ones(lens, H, Hkv, block):
    """dout falls with the token: the last keys of a causal sequence are seen by small ones alone."""
    b = Batch(*lens, H, Hkv, block, seed=73).forward()
    scale_rows(b.dout, b.pad, [2.0 ** -(40 * i // lens[0][0]) for i in range(lens[0][0])])
    check(backward(b))


@pytest.mark.parametrize("block", [0, 1])
def test_heads_of_small_gradients_beside_large_ones(block):
    b = Batch([200], [200], 6, 2, block, seed=74).forward()
    b.dout[:, 3:] = (b.dout[:, 3:].double() * 2.0 ** -30).to(torch.bfloat16)  # the second key head's queries
    check(backward(b))


def test_one_huge_row_keeps_to_itself():
    b = Batch([200, 90], [200, 90], 4, 2, 1, seed=75).forward()
    scale_rows(b.dout, b.pad + 20, [2.0 ** 70])
    check(backward(b))


@pytest.mark.parametrize("block", [0, 1])
def test_the_gradients_of_a_sequence_are_those_of_it_alone(block):
    """To the bit, whatever the sizes of the other sequences' dout and v."""
    b = Batch([150, 200, 60], [150, 200, 60], 6, 2, block, seed=76)
    scale_rows(b.v, b.pad, [2.0 ** 9] * 150)
    b.forward()
    scale_rows(b.dout, b.pad, [2.0 ** 21] * 150)
    backward(b).h.sync()
    one = Batch([200], [200], 6, 2, block, seed=77)
    s, t = slice(b.pad + 150, b.pad + 350), slice(one.pad, one.pad + 200)
    for x in ("q", "k", "v", "dout"):
        getattr(one, x)[t] = getattr(b, x)[s]
    backward(one.forward()).h.sync()
    assert torch.equal(one.out[t], b.out[s])
    for x in ("dq", "dk", "dv"):
        assert torch.equal(getattr(one, x)[t], getattr(b, x)[s]), x


@pytest.mark.parametrize("H,Hkv", [(3, 3), (6, 2), (24, 1)])
@pytest.mark.parametrize("n,most", [(80, 5), (50, 20), (20, 60)])
def test_many_short_sequences_of_all_sizes(H, Hkv, n, most):
    """Tiles of a few rows, taken by one to sixteen warps each; sequences 2^-60 to 1 of the largest in turn."""
    g = torch.Generator().manual_seed(78)
    lens = torch.randint(0, most + 1, (n,), generator=g).tolist()
    b = Batch(lens, lens, H, Hkv, 1, seed=79).forward()
    scale_rows(b.dout, b.pad, [2.0 ** -(20 * (s % 4)) for s, L in enumerate(lens) for _ in range(L)])
    check(backward(b))

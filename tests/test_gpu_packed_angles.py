"""The rotation's angles: the kernel's own cos and sin against exact ones."""
import math
from fractions import Fraction

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

POSITIONS = [0, 1, -1, 2, 54, 12345, -12345, 999_983, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("d,axes", [(64, (16, 24, 24)), (128, (32, 48, 48))])
def test_unit_pairs_turn_by_their_angle(d, axes):
    """Each pair (1, 0) becomes (cos, sin).  The angle is off by the 64-bit fraction of the frequency (|position| 2^-55 of
    a turn), its cut to 32 bits (2^-32) and its rounding to a 24-bit float (half a step below half a turn, 2^-26); cos
    and sin themselves by two steps of a float below 1 (2 * 2^-24)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from video_dit_long_gb300 import k6attn as K
    h = K.Handle.for_packed(1, d, "f32", axes)
    rows = [(a, b, c) for a in POSITIONS for b, c in ((3, 5), (a, -7), (-a - 1, a))]
    pos = torch.tensor(rows, dtype=torch.int32, device="cuda")
    x = torch.zeros((len(rows), 1, d), device="cuda")
    x[..., 0::2] = 1.0
    q, k = torch.empty_like(x), torch.empty_like(x)
    h.packed_norm_rope(x, x, pos, q_out=q, k_out=k)
    h.sync()
    assert torch.equal(q, k)
    got = q.double().cpu()
    freq = [(n, Fraction(10000.0 ** (-2.0 * i / a) / 6.283185307179586476925)) for n, a in enumerate(axes)
            for i in range(a // 2)]
    worst = 0.0
    for r, p in enumerate(rows):
        for i, (n, f) in enumerate(freq):
            turn = f * p[n]
            turn = 2 * math.pi * float(turn - math.floor(turn))
            tol = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32 + abs(p[n]) * 2.0 ** -55) + 2 * 2.0 ** -24
            err = max(abs(float(got[r, 0, 2 * i]) - math.cos(turn)), abs(float(got[r, 0, 2 * i + 1]) - math.sin(turn)))
            worst = max(worst, err / tol)
            assert err <= tol, (p, i, err, tol)
    # the rounding to a float is there: no bound of 2^-32 of a turn holds for the kernel's angles
    assert worst > 0.1

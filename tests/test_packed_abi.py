"""Host-side refusals of the packed calls that need no GPU, and their host-side arithmetic."""
import ctypes

import pytest

from video_dit_long_gb300 import build as B
from video_dit_long_gb300 import k6attn as K

P = ctypes.c_void_p(0x10000000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.load()


def test_a_null_handle_is_refused_by_every_call(lib):
    b = ctypes.byref(K.PackedBatch(2, 2, 1, 100, 100))
    assert lib.k6attn_packed_norm_rope(None, 4, 2, None, 0, P, P, 512, P, 256, P, P, 1e-6, P, 512, P, 256,
                                       K.F16, None) == K.ERR_INVALID_ARG
    assert lib.k6attn_packed_norm_rope_backward(None, 4, 2, P, 2, P, P, 512, P, 256, P, 512, P, 256, P, P, 1e-6,
                                                P, 512, P, 256, P, P, P, 1 << 20, None) == K.ERR_INVALID_ARG
    assert lib.k6attn_packed_plan(None, b, P, P, P, 1 << 20, None) == K.ERR_INVALID_ARG
    assert lib.k6attn_packed_forward(None, b, P, P, 512, P, 256, P, 256, K.F16, P, 512, P, P, 1 << 20,
                                     None) == K.ERR_INVALID_ARG
    assert lib.k6attn_packed_backward(None, b, P, P, 512, P, 256, P, 256, K.F16, P, 512, P, 512, P, P, 512, P, 256, P,
                                      256, P, 1 << 20, None) == K.ERR_INVALID_ARG
    assert b"null handle" in lib.k6attn_last_error()
    for name in ("plan_bytes", "workspace_bytes", "backward_workspace_bytes"):
        assert getattr(lib, "k6attn_packed_" + name)(None, b) == 0
    assert lib.k6attn_packed_norm_rope_backward_workspace_bytes(None, 4, 2) == 0


def test_row_division_by_reciprocal():
    """The backward kernel's (row * ceil(2^16 / G)) >> 16 is row / G for every row of a tile and group size."""
    for G in range(1, 129):
        inv = (65536 + G - 1) // G
        assert all((r * inv) >> 16 == r // G for r in range(128)), G


def test_rotary_turns_in_fixed_point():
    """Angles as the kernel forms them (position * 64-bit fraction of a turn, top 32 bits) against exact arithmetic:
    within 2^-32 of a turn plus |position| 2^-55, at every 32-bit position."""
    from fractions import Fraction
    import math
    for a, i in ((32, 0), (32, 15), (48, 7), (48, 23)):
        turns = 10000.0 ** (-2.0 * i / a) / 6.283185307179586476925
        w = int(math.floor(math.ldexp(turns - math.floor(turns), 64) + 0.5))
        for pos in (0, 1, -1, 54, 12345, 2 ** 31 - 1, -2 ** 31):
            top = ((pos * w) % 2 ** 64) >> 32
            top -= 2 ** 32 if top >= 2 ** 31 else 0
            exact = Fraction(turns) * pos
            off = Fraction(top, 2 ** 32) - exact
            off -= round(off)
            assert abs(off) <= Fraction(1, 2 ** 32) + abs(pos) * Fraction(1, 2 ** 55), (a, i, pos)


def test_rotary_angles_as_floats():
    """The angle as the kernel takes sin and cos of it, rounded to a 24-bit float: within 2^-26 of a turn (half a step
    near half a turn) more, and not within 2^-32."""
    from fractions import Fraction
    import math
    np = pytest.importorskip("numpy")
    worst = Fraction(0)
    for a, i in ((32, 0), (32, 15), (48, 7), (48, 23)):
        turns = 10000.0 ** (-2.0 * i / a) / 6.283185307179586476925
        w = int(math.floor(math.ldexp(turns - math.floor(turns), 64) + 0.5))
        for pos in (0, 1, -1, 54, 12345, 999983, 2 ** 31 - 1, -2 ** 31):
            top = ((pos * w) % 2 ** 64) >> 32
            top -= 2 ** 32 if top >= 2 ** 31 else 0
            off = Fraction(float(np.float32(top))) / 2 ** 32 - Fraction(turns) * pos
            off = abs(off - round(off))
            assert off <= Fraction(1, 2 ** 26) + Fraction(1, 2 ** 32) + abs(pos) * Fraction(1, 2 ** 55), (a, i, pos)
            worst = max(worst, off)
    assert worst > Fraction(1, 2 ** 32)

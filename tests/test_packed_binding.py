"""Refusals and statuses of the packed binding that need no GPU: a handle on CPU
tensors whose library records the calls."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from video_dit_long_gb300 import k6attn as K  # noqa: E402


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def handle():
    K._torch_types()
    h = object.__new__(K.Handle)
    h.h, h._lib, h._H, h._d, h._elem = ctypes.c_void_p(), Library(), 4, 128, torch.bfloat16
    h._dev, h._raw_stream = -1, lambda dev: 0  # the device index of CPU tensors
    return h


def tensors(T=6):
    x = torch.zeros((T, 8, 128), dtype=torch.bfloat16)
    return x[:, :4], x[:, 4:6], torch.zeros((T, 3), dtype=torch.int32)


def forward(h, offsets):
    q, k, pos = tensors()
    h.packed_norm_rope(q, k, pos, q_out=torch.empty_like(q), k_out=torch.empty_like(k), offsets=offsets)


def backward(h, offsets):
    q, k, pos = tensors()
    h.packed_norm_rope_backward(q, k, None, None, pos, dq=torch.empty_like(q), dk=torch.empty_like(k), offsets=offsets)


@pytest.mark.parametrize("call", [forward, backward])
def test_empty_offsets_are_refused(handle, call):
    """An empty tensor has no address: it would reach the library as 'no offsets', and padding rows be taken."""
    with pytest.raises(ValueError):
        call(handle, torch.zeros(0, dtype=torch.int32))
    assert not handle._lib.calls
    call(handle, None)
    call(handle, torch.tensor([0, 4], dtype=torch.int32))
    (_, without), (_, given) = handle._lib.calls
    assert without[3] is None and given[3] and given[4] == 1

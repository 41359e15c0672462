"""Host-side refusals of the paged calls that need no GPU: the library's of a null handle, the binding's on CPU tensors."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from video_dit_long_gb300 import build as B  # noqa: E402
from video_dit_long_gb300 import k6attn as K  # noqa: E402

P = ctypes.c_void_p(0x10000000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.load()


def test_a_null_handle_is_refused_by_every_call(lib):
    b = ctypes.byref(K.PagedBatch(2, 2, 1, 16, 8, 0, 100, 100))
    c = K.Pages(0x10000000, 16 * 256, 256, 128)
    assert lib.k6attn_paged_plan(None, b, P, P, P, None, None, P, 1 << 20, None) == K.ERR_INVALID_ARG
    assert lib.k6attn_paged_append(None, b, P, P, 512, P, 256, P, 256, P, P, P, 1e-6, P, 512, c, c, K.F16,
                                   None) == K.ERR_INVALID_ARG
    assert lib.k6attn_paged_forward(None, b, P, P, P, 512, c, c, K.F16, P, 512, P, P, 1 << 20, None) == K.ERR_INVALID_ARG
    assert b"null handle" in lib.k6attn_last_error()
    for name in ("plan_bytes", "workspace_bytes"):
        assert getattr(lib, "k6attn_paged_" + name)(None, b) == 0


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


def step(T=6, n_pages=5, page=16, kv=2):
    K._torch_types()
    h = object.__new__(K.Handle)
    h.h, h._lib, h._H, h._d, h._elem = ctypes.c_void_p(), Library(), 4, 128, torch.bfloat16
    h._dev, h._raw_stream = -1, lambda dev: 0  # the device index of CPU tensors
    plan = K.PagedPlan(K.PagedBatch(2, kv, 1, page, 3, 0, n_pages, T), torch.zeros(256, dtype=torch.uint8),
                       torch.zeros((2, 3), dtype=torch.int32))
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    x = z(T, 8, 128)
    append = dict(plan=plan, q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], positions=z(T, 3, t=torch.int32),
                  q_weight=z(128, t=torch.float32), k_weight=z(128, t=torch.float32), q_out=z(T, 4, 128, t=torch.float16),
                  k_cache=z(n_pages, page, kv, 128, t=torch.float16), v_cache=z(n_pages, page, kv, 128))
    forward = dict(plan=plan, q=append["q_out"], k_cache=append["k_cache"], v_cache=append["v_cache"], out=z(T, 4, 128),
                   lse=z(4, T, t=torch.float32))
    return h, append, forward


def test_what_reaches_the_library():
    h, append, forward = step()
    h.paged_append(**append)
    h.paged_forward(**forward)
    by_head = append["v_cache"].transpose(1, 2).contiguous().transpose(1, 2)
    h.paged_append(**{**append, "q": None, "q_out": None, "v_cache": by_head})
    (n0, a), (n1, f), (_, alone) = h._lib.calls
    assert (n0, n1) == ("k6attn_paged_append", "k6attn_paged_forward")
    assert a[4] == a[6] == a[8] == 8 * 128 and a[17] == K.F16 and f[8] == K.F16
    assert (a[15].page_stride, a[15].token_stride, a[15].head_stride) == (16 * 256, 256, 128)
    assert alone[3] is None and alone[13] is None
    assert (alone[16].page_stride, alone[16].token_stride, alone[16].head_stride) == (16 * 256, 128, 16 * 128)


@pytest.mark.parametrize("name,change", [
    ("q", lambda t: t[:, :3]), ("q", lambda t: t.half()), ("k", lambda t: t[:5]), ("v", lambda t: t.float()),
    ("positions", lambda t: t.long()), ("q_weight", lambda t: t[:64]), ("k_weight", lambda t: t.half()),
    ("q_out", lambda t: t.bfloat16()), ("k_cache", lambda t: t[:4]), ("k_cache", lambda t: t.float()),
    ("v_cache", lambda t: t.half()), ("v_cache", lambda t: t.transpose(1, 2)), ("v_cache", lambda t: t.transpose(2, 3)),
])
def test_tensors_that_do_not_fit_the_plan_are_refused(name, change):
    h, append, _ = step()
    with pytest.raises(ValueError):
        h.paged_append(**{**append, name: change(append[name])})
    assert not h._lib.calls


def test_groups_need_both_of_their_tensors():
    h, *_ = step()
    cu, k, table = torch.tensor([0, 1, 2], dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    for more in (dict(cu_groups=cu), dict(shared=k)):
        with pytest.raises(ValueError):
            h.paged_plan(cu, k, table, 6, 2, 16, 5, **more)
    with pytest.raises(ValueError):
        h.paged_plan(cu, k, table[0], 6, 2, 16, 5)

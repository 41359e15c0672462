"""The pools of a layer over pages, its own or given ones, on a stand-in for the handle (no GPU)."""
import types

import pytest

torch = pytest.importorskip("torch")


class Cpu(str):
    """The device of CPU tensors, by name and by the index that they give."""
    __hash__ = str.__hash__

    def __eq__(self, other):
        return other == -1 or str.__eq__(self, other)

    def __ne__(self, other):
        return not self == other


PAGES = (5, 16, 2, 128)


def layer(**kw):
    from video_dit_long_gb300.packed import PagedAttention
    h = types.SimpleNamespace(_dev=Cpu("cpu"), _H=4, _d=128, paged_workspace_bytes=lambda plan: 64)
    batch = types.SimpleNamespace(handle=h, tokens=6, kv_heads=2, plan=types.SimpleNamespace(pages=PAGES))
    w = torch.ones(128)
    return PagedAttention(batch, w, w, **kw)


def pools(t=torch.float16):
    return dict(k_cache=torch.zeros(PAGES, dtype=t), v_cache=torch.zeros(PAGES, dtype=torch.bfloat16))


@pytest.mark.parametrize("qk,t", [("f16", torch.float16), ("bf16", torch.bfloat16)])
def test_its_own(qk, t):
    for by_head, strides in ((False, (4096, 256, 128, 1)), (True, (4096, 128, 2048, 1))):
        x = layer(qk=qk, by_head=by_head)
        assert (x.k_cache.dtype, x.v_cache.dtype) == (t, torch.bfloat16)
        for c in (x.k_cache, x.v_cache):
            assert c.shape == PAGES and c.stride() == strides


def test_given_ones_are_taken_as_they_are(monkeypatch):
    """And none are made beside them: pools may fill the GPU."""
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda s, **kw: made.append(tuple(s)) or empty(s, **kw))
    have = pools()
    x = layer(**have)
    assert x.k_cache is have["k_cache"] and x.v_cache is have["v_cache"]
    assert made and not any(len(s) == 4 for s in made)
    have = {n: c.transpose(1, 2).contiguous().transpose(1, 2) for n, c in pools(torch.bfloat16).items()}
    x = layer(qk="bf16", **have)
    assert x.k_cache is have["k_cache"] and x.v_cache is have["v_cache"]


@pytest.mark.parametrize("change", [
    dict(k_cache=None), dict(v_cache=None), dict(k_cache=torch.zeros(PAGES)), dict(k_cache=torch.zeros(PAGES, dtype=torch.bfloat16)),
    dict(v_cache=torch.zeros(PAGES, dtype=torch.float16)), dict(v_cache=torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)),
    dict(v_cache=torch.zeros((5, 2, 16, 128), dtype=torch.bfloat16)),
    dict(k_cache=torch.zeros((5, 16, 2, 256), dtype=torch.float16)[..., ::2]),
])
def test_pools_that_do_not_fit_are_refused(change):
    with pytest.raises(ValueError):
        layer(**{**pools(), **change})

"""The attention of one layer over a packed batch of clips, forward and backward,
and of the new tokens of growing streams over a cache of pages.

A batch of clips (or images, prompts, new tokens of running streams) of different
lengths lies one behind another in [tokens] rows.  The layer's fused projection
gives qkv [tokens][(H + 2 kv_heads) * d]; this module holds the buffers and makes
the library's calls in the layer's order ("Context Parallelism in vLLM Omni
Neuron", "Self-Attention with Context Parallelism": QK-norm, rotary embedding,
attention):

  forward:  k6attn_packed_norm_rope   q, k out of qkv into rotated copies (fp16 or bf16)
            k6attn_packed_forward     attention of the rotated q, k and of v in qkv
  backward: k6attn_packed_backward    gradients of the rotated q, k, and of v into dqkv
            k6attn_packed_norm_rope_backward   those of q, k into dqkv, and of the norm's weights

Streams that grow keep their keys and values in pages (PagedBatch, PagedAttention);
a step of new tokens is

            k6attn_paged_append       rotated q out of qkv, rotated k and v into the pages
            k6attn_paged_forward      attention of q over the streams' pages

All arithmetic runs in the library's kernels.  A layer stack makes one
PackedBatch per batch of lengths and one PackedAttention per layer whose
activations it keeps.
"""
from __future__ import annotations

from . import k6attn as K


def _int32(x):
    """x as a tensor of integers that int32 holds: anything else would be cut off without a word.  (Numbers on the device
    are taken as they are; the plan checks what it makes of them.)"""
    import torch
    x = torch.as_tensor(x)
    if x.is_floating_point() or (not x.is_cuda and x.numel() and not -2 ** 31 <= int(x.min()) <= int(x.max()) < 2 ** 31):
        raise ValueError(f"want integers of 32 bits, got {x.dtype} {tuple(x.shape)}"
                         + ("" if x.is_floating_point() else f" from {int(x.min())} to {int(x.max())}"))
    return x


class PackedBatch:
    """The offsets, mask and work list of a batch, shared by the layers that attend over it.

    lens: tokens of each sequence (a list, or int32 offsets [n + 1] on the device).  mask_block 0: full attention,
    1: causal, F: causal by frames of F tokens."""

    def __init__(self, handle, lens, tokens, kv_heads, mask_block=0):
        import torch
        self.handle, self.tokens, self.kv_heads = handle, int(tokens), int(kv_heads)
        lens = self._offsets(lens)
        self.offsets = torch.empty_like(lens, device=handle._dev).copy_(lens)  # its own: set_offsets writes to it
        self.plan = handle.packed_plan(self.offsets, None, self.tokens, self.tokens, self.kv_heads, mask_block)

    @staticmethod
    def _offsets(lens):
        import torch
        return lens if isinstance(lens, torch.Tensor) else _int32(torch.tensor([0] + list(lens)).cumsum(0)).to(torch.int32)

    def set_offsets(self, offsets):
        """Other lengths of as many sequences, in place (a captured layer sees them at its next replay): offsets [n + 1],
        or a list of lengths.  Offsets on the device are copied in stream order; the host waits for a copy of its own."""
        offsets = self._offsets(offsets)
        if offsets.shape != self.offsets.shape or offsets.is_floating_point():
            raise ValueError(f"offsets: want {self.offsets.numel()} integers for {self.offsets.numel() - 1} sequences, got "
                             f"{offsets.dtype} {tuple(offsets.shape)}")
        self.offsets.copy_(offsets)
        self.handle.packed_replan(self.plan, self.offsets, None)


class PackedAttention:
    """One layer's attention over a PackedBatch; keeps what its backward pass needs until the next forward."""

    def __init__(self, batch, q_weight, k_weight, eps=1e-6, qk="f16"):
        import torch
        if qk not in ("f16", "bf16"):
            raise ValueError(qk)
        self.batch, self.h = batch, batch.handle
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        T, H, kv, d = batch.tokens, self.h._H, batch.kv_heads, self.h._d
        self.H, self.kv, self.d = H, kv, d
        t = torch.float16 if qk == "f16" else torch.bfloat16
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=self.h._dev)  # noqa: E731
        self.q, self.k = new(T, H, d, dtype=t), new(T, kv, d, dtype=t)
        self.out, self.lse = new(T, H, d).zero_(), new(H, T, dtype=torch.float32)
        self.dq, self.dk = new(T, H, d), new(T, kv, d)
        self.dq_weight, self.dk_weight = torch.empty_like(q_weight), torch.empty_like(k_weight)
        room = max(self.h.packed_workspace_bytes(batch.plan), self.h.packed_backward_workspace_bytes(batch.plan),
                   self.h.packed_norm_rope_backward_workspace_bytes(T, kv))
        self.workspace = new(room, dtype=torch.uint8)

    def parts(self, qkv):
        """q, k, v of a fused projection [tokens][(H + 2 kv_heads) * d], as views."""
        x = qkv.view(qkv.shape[0], self.H + 2 * self.kv, self.d)
        return x[:, :self.H], x[:, self.H:self.H + self.kv], x[:, self.H + self.kv:]

    def forward(self, qkv, positions):
        """qkv bf16, positions int32 [tokens][3]; returns out [tokens][H][d] (bf16; rows outside the sequences stay)."""
        q, k, v = self.parts(qkv)
        self.h.packed_norm_rope(q, k, positions, self.q_weight, self.k_weight, self.eps, q_out=self.q, k_out=self.k,
                                offsets=self.batch.offsets)
        self.h.packed_forward(self.batch.plan, self.q, self.k, v, self.out, self.lse, workspace=self.workspace)
        return self.out

    def backward(self, dout, qkv, positions, dqkv):
        """The gradients of qkv into dqkv (as qkv; rows outside the sequences stay, and enter nothing) and of the
        norm's weights; returns (dq_weight, dk_weight)."""
        q, k, v = self.parts(qkv)
        dq, dk, dv = self.parts(dqkv)
        self.h.packed_backward(self.batch.plan, self.q, self.k, v, self.out, dout, self.lse, self.dq, self.dk, dv,
                               workspace=self.workspace)
        self.h.packed_norm_rope_backward(self.dq, self.dk, q, k, positions, self.q_weight, self.k_weight, self.eps,
                                         dq=dq, dk=dk, dq_weight=self.dq_weight, dk_weight=self.dk_weight,
                                         workspace=self.workspace, offsets=self.batch.offsets)
        return self.dq_weight, self.dk_weight


class PagedBatch:
    """A step of streams whose keys lie in pages: its offsets, lengths, table of pages and work list, shared by the layers
    of the step and made anew for the next one.

    lens: new tokens of each stream (a list, or int32 offsets [n + 1]); k_lens: keys of each with the new ones; table
    [n][max_pages]: its pages in order.  tokens: rows of qkv.  groups: [(streams, shared tokens)] of the streams in
    order that have a prefix in common, or None (a stream that sees much less of it than the others cuts what is read once
    for all of them: better a group of its own); mask_block as for PackedBatch."""

    def __init__(self, handle, lens, k_lens, table, tokens, kv_heads, page_tokens, n_pages, mask_block=1, groups=None):
        import torch
        self.handle, self.tokens, self.kv_heads = handle, int(tokens), int(kv_heads)
        own = lambda x: _int32(x).to(device=handle._dev, dtype=torch.int32, copy=True)  # noqa: E731
        self.offsets, self.k_lens, self.table = own(PackedBatch._offsets(lens)), own(k_lens), own(table)
        self.groups = {}
        if groups:
            self.groups = dict(cu_groups=own(PackedBatch._offsets([n for n, _ in groups])), shared=own([n for _, n in groups]))
        self.plan = handle.paged_plan(self.offsets, self.k_lens, self.table, self.tokens, self.kv_heads, page_tokens, n_pages,
                                      mask_block, **self.groups)

    def next(self, lens=None, k_lens=None, table=None, shared=None):
        """The next step of as many streams, in place (captured layers see it at their next replay); what is not given
        stays as it is.  Tensors on the device are copied in stream order; the host waits for copies of its own."""
        given = [(self.offsets, None if lens is None else PackedBatch._offsets(lens)), (self.k_lens, k_lens),
                 (self.table, table), (self.groups.get("shared"), shared)]
        given = [(to, _int32(x)) for to, x in given if x is not None]
        for to, x in given:
            if to is None:
                raise ValueError("shared: the batch has no groups")
            if x.shape != to.shape:
                raise ValueError(f"want integers of shape {tuple(to.shape)}, got {tuple(x.shape)}")
        for to, x in given:
            to.copy_(x)
        self.handle.paged_replan(self.plan, self.offsets, self.k_lens, self.table, **self.groups)


class PagedAttention:
    """One layer's attention over a PagedBatch, with the layer's pools of keys and values.

    qk: the type of rotated queries and keys.  k_cache, v_cache [n_pages][page_tokens][kv_heads][d] (qk's type, and bf16):
    pools that the layer already has, as when it goes on from the batch that read the prompts to the one that takes the
    steps; without them it makes its own, with one head's tokens after another's in a page where by_head says so (else
    one token's heads)."""

    def __init__(self, batch, q_weight, k_weight, eps=1e-6, qk="f16", by_head=False, *, k_cache=None, v_cache=None):
        import torch
        if qk not in ("f16", "bf16"):
            raise ValueError(qk)
        self.batch, self.h = batch, batch.handle
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        T, self.H, self.kv, self.d = batch.tokens, self.h._H, batch.kv_heads, self.h._d
        n, page, kv, d = batch.plan.pages
        t = torch.float16 if qk == "f16" else torch.bfloat16
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=self.h._dev)  # noqa: E731
        pool = lambda t: new(n, kv, page, d, dtype=t).transpose(1, 2) if by_head else new(n, page, kv, d, dtype=t)  # noqa: E731
        if (k_cache is None) != (v_cache is None):
            raise ValueError("k_cache, v_cache: give both, or neither")
        if k_cache is None:
            k_cache, v_cache = pool(t), pool(torch.bfloat16)
        K._pages(k_cache, batch.plan.pages, t, self.h._dev, "k_cache")
        K._pages(v_cache, batch.plan.pages, torch.bfloat16, self.h._dev, "v_cache")
        self.k_cache, self.v_cache = k_cache, v_cache
        self.q, self.out, self.lse = new(T, self.H, d, dtype=t), new(T, self.H, d).zero_(), new(self.H, T, dtype=torch.float32)
        self.workspace = new(self.h.paged_workspace_bytes(batch.plan), dtype=torch.uint8)

    parts = PackedAttention.parts

    def forward(self, qkv, positions):
        """qkv bf16 [tokens][(H + 2 kv_heads) * d], positions int32 [tokens][3] of the step's new tokens: their keys and
        values join the pages; returns out [tokens][H][d] (bf16; rows outside the streams stay)."""
        q, k, v = self.parts(qkv)
        plan = self.batch.plan
        self.h.paged_append(plan, q, k, v, positions, self.q_weight, self.k_weight, self.eps, q_out=self.q,
                            k_cache=self.k_cache, v_cache=self.v_cache)
        self.h.paged_forward(plan, self.q, self.k_cache, self.v_cache, self.out, self.lse, workspace=self.workspace)
        return self.out

"""The attention of one layer over a packed batch of clips, forward and backward.

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

All arithmetic runs in the library's kernels.  A layer stack makes one
PackedBatch per batch of lengths and one PackedAttention per layer whose
activations it keeps.
"""
from __future__ import annotations

from . import k6attn as K


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
        return lens if isinstance(lens, torch.Tensor) else torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)

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

"""Self-attention over the cells of a domain-sharded volume, held on the GPU.

One transformer branch of a sharded model, every step a call into the library:

    layer norm -> 1x1 conv to q, k, v -> rotary positions -> attention over all
    cells of the volume -> 1x1 conv back to the volume's channels

and its gradients.  Cells of all shards are the tokens of one sequence (or, of
one unsharded batch, of one sequence per sample).  The shard buffers are views
of one packed buffer, shard after shard, so the convs write the tokens where the
attention reads them; the order of the cells within a sequence does not matter,
each carries its place in the whole volume through the rotary positions.  On
one GPU every shard sees every key in place; across GPUs the keys and values of
the other shards would arrive by the ring that the ShardTensor summary names
(section 4, "Results and benchmarks": ring attention over sharded sequences).

torch is used for allocation and views only.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from . import (_TYPES, ST_BF16, ST_F32, ShardConvError, _cells, _stream, st_attention_packed,
               st_attention_packed_backward, st_attention_workspace_bytes, st_conv_dgrad_weights, st_conv_sharded,
               st_conv_wgrad, st_conv_wgrad_workspace_bytes, st_conv_workspace_bytes, st_layernorm_backward,
               st_layernorm_backward_workspace_bytes, st_layernorm_sharded, st_plan_positions, st_plan_sequences,
               st_plan_shards, st_rope_axes)


def _torch():
    import torch
    return torch


class ShardedAttention:
    """Buffers, plans and steps of one attention branch.

    spatial, shards: the volume and its per-axis shard sizes; channels: of the
    volume; heads, kv_heads, head_dim: of the attention (heads * head_dim need
    not be channels); axis_dims: rotary channels per spatial axis (default: an
    even split of head_dim).  The volume is fp32 (a conv's output); products
    run on bf16 operands.
    """

    def __init__(self, spatial: Sequence[int], shards, channels: int, heads: int, kv_heads: int, head_dim: int,
                 axis_dims: Optional[Sequence[int]] = None, batch: int = 1, eps: float = 1e-5, base: float = 10000.0,
                 device: str = "cuda"):
        torch = _torch()
        if not torch.cuda.is_available():
            raise ShardConvError(6, "no GPU: the layer runs only on the HIP library")
        nd = len(spatial)
        if batch > 1 and math.prod(len(s) for s in shards) > 1:
            raise ShardConvError(4, "a sharded volume is one sample (batch 1)")
        self.nd, self.eps, self.base = nd, eps, base
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.joint = heads + 2 * kv_heads
        if axis_dims is None:
            part = head_dim // nd // 2 * 2
            axis_dims = [part] * nd
        self.axis_dims = list(axis_dims)
        width, joint = heads * head_dim, self.joint * head_dim
        self.channels, self.width, self.joint_width = channels, width, joint
        plan = lambda c, t: st_plan_shards(nd, batch, c, spatial, shards, [0] * nd, t)  # noqa: E731
        self.x_plan, self.norm_plan = plan(channels, ST_F32), plan(channels, ST_BF16)
        self.joint_plan, self.width_plan = plan(joint, ST_BF16), plan(width, ST_BF16)
        cells = _cells(self.x_plan)
        self.starts = [sum(cells[:i]) for i in range(len(cells) + 1)]
        self.tokens = t = self.starts[-1]
        # every other packed buffer is cut into shard buffers; the narrowest rows
        # are the bf16 ones of the volume (normed, dy)
        if any(s * channels * 2 % 16 for s in self.starts[:-1]):
            raise ShardConvError(7, f"the packed shards of {channels} channels do not start on 16 bytes: "
                                    "use a multiple of 8 channels")
        self.device = torch.device(device)
        lens = [t // batch] * batch
        self.seqs = st_plan_sequences(lens, None, heads, kv_heads, head_dim, ST_BF16, causal=False)
        self.scale = 1.0 / math.sqrt(head_dim)

        new = lambda n, dt: torch.zeros(t, n, dtype=dt, device=self.device)  # noqa: E731
        f32, bf16 = torch.float32, torch.bfloat16
        self.normed, self.qkv, self.turned = new(channels, bf16), new(joint, f32), new(joint, bf16)
        self.attended, self.y = new(width, bf16), new(channels, f32)
        self.stats = torch.zeros(t, 2, device=self.device)
        self.lse = torch.zeros(t, heads, device=self.device)
        # (written shard by shard, then packed: a shard of the packed rows starts
        # wherever the cells before it end, a buffer of its own on 16 bytes)
        own = [torch.empty(n, nd, dtype=torch.int32, device=self.device) for n in cells]
        st_plan_positions(self.x_plan, own)
        self.positions = torch.cat(own)
        self.gamma = self.beta = None
        self._gamma, self._beta = (torch.ones(channels, device=self.device) for _ in range(2))
        self.w_qkv = torch.zeros(joint * channels, dtype=bf16, device=self.device)
        self.w_out = torch.zeros(channels * width, dtype=bf16, device=self.device)
        ws = [st_conv_workspace_bytes(self.norm_plan, joint, 1), st_conv_workspace_bytes(self.width_plan, channels, 1)]
        if 0 in ws:
            raise ShardConvError(4, "unsupported channel counts")
        self.conv_ws = torch.zeros(max(ws), dtype=torch.uint8, device=self.device)
        self.attn_ws = torch.zeros(max(16, st_attention_workspace_bytes(self.seqs, True)), dtype=torch.uint8,
                                   device=self.device)
        self.grads = None
        torch.cuda.synchronize()             # the steps may run on any stream: nothing is left to fill

    def parts(self, packed) -> list:
        """The shards' views of a packed [tokens, ...] buffer."""
        return [packed[a:b] for a, b in zip(self.starts, self.starts[1:])]

    def split(self, packed):
        """q, k, v views of a joint [tokens, (heads + 2 kv_heads) * head_dim] buffer."""
        v = packed.view(self.tokens, self.joint, self.head_dim)
        h, k = self.heads, self.kv_heads
        return v[:, :h], v[:, h:h + k], v[:, h + k:]

    def set_weights(self, w_qkv: np.ndarray, w_out: np.ndarray, gamma=None, beta=None) -> None:
        """w_qkv [(heads + 2 kv_heads) * head_dim, channels], w_out [channels,
        heads * head_dim] as float32 (rounded to bf16); gamma, beta [channels].
        Waits for the device before and after: steps on any stream see one set
        of weights."""
        torch = _torch()

        def put(name, a, to, *shape):
            if a is None:
                return None
            a = np.ascontiguousarray(a, np.float32)
            if a.size != to.numel() or (a.ndim > 1 and a.shape[:len(shape)] != shape):
                raise ShardConvError(2, f"{name}: expected {shape}, got {a.shape}")
            return to.copy_(torch.from_numpy(a.reshape(-1)))

        torch.cuda.synchronize()
        put("w_qkv", w_qkv, self.w_qkv, self.joint_width, self.channels)
        put("w_out", w_out, self.w_out, self.channels, self.width)
        self.gamma = put("gamma", gamma, self._gamma, self.channels)
        self.beta = put("beta", beta, self._beta, self.channels)
        torch.cuda.synchronize()

    # ------------------------------------------------------------- steps
    def forward(self, x, stream=None):
        """x: packed fp32 [tokens, channels] (the shards' cells one after the
        other; self.parts(x) are the shard buffers).  Returns the branch's
        output in the same layout (self.y)."""
        parts = self.parts
        st_layernorm_sharded(self.x_plan, parts(x), self.gamma, self.beta, self.eps, self.norm_plan,
                             parts(self.normed), self.stats, stream)
        st_conv_sharded(self.norm_plan, parts(self.normed), self.w_qkv, None, self.joint_width, 1, parts(self.qkv),
                        workspace=self.conv_ws, stream=stream)
        rows = (self.tokens, self.joint, self.head_dim)
        st_rope_axes(self.qkv.view(rows), self.positions, self.axis_dims, self.turned.view(rows),
                     rotated_heads=self.heads + self.kv_heads, base=self.base, stream=stream)
        q, k, v = self.split(self.turned)
        out = self.attended.view(self.tokens, self.heads, self.head_dim)
        st_attention_packed(self.seqs, q, k, v, self.scale, out, self.lse, self.attn_ws, stream)
        st_conv_sharded(self.width_plan, parts(self.attended), self.w_out, None, self.channels, 1, parts(self.y),
                        workspace=self.conv_ws, stream=stream)
        return self.y

    def alloc_backward(self) -> None:
        """The buffers of the backward steps.  The first backward() calls it; call
        it before a graph capture whose steps run on another stream than the
        current one."""
        if self.grads is not None:
            return
        torch = _torch()
        t, dev = self.tokens, self.device
        f32, bf16 = torch.float32, torch.bfloat16
        need = max(st_conv_wgrad_workspace_bytes(self.norm_plan, self.joint_width, 1),
                   st_conv_wgrad_workspace_bytes(self.width_plan, self.channels, 1),
                   st_layernorm_backward_workspace_bytes(self.x_plan), 16)
        conv = [st_conv_workspace_bytes(self.norm_plan, self.width, 1),
                st_conv_workspace_bytes(self.joint_plan, self.channels, 1)]
        if 0 in conv:
            raise ShardConvError(4, "unsupported channel counts")
        new = lambda *shape, dt=f32: torch.empty(*shape, dtype=dt, device=dev)  # noqa: E731
        g = {"wide": new(t, self.width), "dout": new(t, self.width, dt=bf16), "dqkv": new(t, self.joint_width, dt=bf16),
             "dnorm": new(t, self.channels), "dx": new(t, self.channels),
             "dw_qkv": new(self.joint_width, self.channels), "dw_out": new(self.channels, self.width),
             "dgamma": new(self.channels), "dbeta": new(self.channels),
             "wt": new(max(self.w_qkv.numel(), self.w_out.numel()), dt=bf16),
             "ws": new(need, dt=torch.uint8), "conv_ws": new(max(conv), dt=torch.uint8)}
        # Nothing is filled, but the memory may have had another owner, whose work
        # the current stream alone has in order: the steps may run on another.
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.synchronize()
        self.grads = g

    def backward(self, x, dy, stream=None) -> dict:
        """Gradients of the last forward(x) for dy (packed bf16 [tokens,
        channels]): dx (fp32, packed), dw_qkv, dw_out, dgamma, dbeta."""
        if self.grads is None:
            if _stream(stream).value != _stream(None).value and _torch().cuda.is_current_stream_capturing():
                raise ShardConvError(4, "the backward buffers are not there yet: call alloc_backward() before capturing")
            self.alloc_backward()
        if dy.dtype not in _TYPES[ST_BF16]:
            raise ShardConvError(1, f"dy: expected bfloat16, got {dy.dtype}")
        g, parts, nd = self.grads, self.parts, self.nd
        # the output projection: weight gradient, then the gradient at the
        # attention's output, rounded to bf16
        st_conv_wgrad(self.width_plan, parts(self.attended), self.norm_plan, parts(dy), 1, g["dw_out"], g["ws"], stream)
        st_conv_dgrad_weights(nd, self.width, self.channels, 1, ST_BF16, self.w_out, g["wt"], stream)
        st_conv_sharded(self.norm_plan, parts(dy), g["wt"], None, self.width, 1, parts(g["wide"]),
                        workspace=g["conv_ws"], stream=stream)
        heads = (self.tokens, self.heads, self.head_dim)
        st_rope_axes(g["wide"].view(heads), self.positions, self.axis_dims, g["dout"].view(heads), rotated_heads=0,
                     stream=stream)
        # attention, and the rotation turned back in place
        q, k, v = self.split(self.turned)
        dq, dk, dv = self.split(g["dqkv"])
        st_attention_packed_backward(self.seqs, q, k, v, self.attended.view(heads), self.lse, g["dout"].view(heads),
                                     self.scale, dq, dk, dv, self.attn_ws, stream)
        rows = g["dqkv"].view(self.tokens, self.joint, self.head_dim)
        st_rope_axes(rows, self.positions, self.axis_dims, rows, rotated_heads=self.heads + self.kv_heads,
                     base=self.base, inverse=True, stream=stream)
        # the joint projection and the norm
        st_conv_wgrad(self.norm_plan, parts(self.normed), self.joint_plan, parts(g["dqkv"]), 1, g["dw_qkv"], g["ws"], stream)
        st_conv_dgrad_weights(nd, self.channels, self.joint_width, 1, ST_BF16, self.w_qkv, g["wt"], stream)
        st_conv_sharded(self.joint_plan, parts(g["dqkv"]), g["wt"], None, self.channels, 1, parts(g["dnorm"]),
                        workspace=g["conv_ws"], stream=stream)
        st_layernorm_backward(self.x_plan, parts(x), self.x_plan, parts(g["dnorm"]), self.gamma, self.stats,
                              self.x_plan, parts(g["dx"]), g["dgamma"], g["dbeta"], g["ws"], stream)
        return {n: g[n] for n in ("dx", "dw_qkv", "dw_out", "dgamma", "dbeta")}

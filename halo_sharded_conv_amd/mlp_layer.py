"""The MLP branch of a transformer block over the cells of a domain-sharded
volume, held on the GPU.

Every step a call into the library:

    x + branch, RMS norm -> product to the hidden width, activation ->
    product back, plus the stream

and its gradients.  A cell's channels meet no other cell's, so the shards of a
volume need no exchange: the cells of all shards lie packed, one shard after
the other, as ShardedAttention has them, whose output is this branch's `branch`.

kept="mx8" holds what the backward pass reads (the sum, the normed cells, the
pre-activation) in 8 bits with a power of two per 32 channels: 2 + hidden /
channels bytes a channel and cell in place of 6 + 4 hidden / channels.  The 16-
and 32-bit buffers of the forward steps are scratch then, which the layers of
one model may share (`scratch`).

products="mx8" (forward only: nothing is kept, so that every buffer of the steps is
scratch, whatever `kept` says) multiplies in 8 bits: weights rounded once, the norm's
output where it is written, the hidden values in a pass of their own from
bf16 (128^2 cells of 2048 to 8192 channels 844 us; an 8-bit output of the product itself
would widen its operands, 1608).  So the hidden values are rounded twice, to bf16 from
sums that the 8-bit instructions cut and then to 8 bits: 3.4% of the codes differ from
those of one rounding, 0.017 of the norm, but the values are as near to the unrounded
ones (2.66% of the norm off, once rounded 2.65%).  The output is bf16, so that the stream
of several such layers is rounded to it in each.

torch is used for allocation and views only.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from . import (Mx8, ShardConvError, _ACTS, _stream, mx8_empty, st_linear, st_linear_backward, st_linear_workspace_bytes,
               st_mx8_load, st_mx8_store, st_rmsnorm, st_rmsnorm_backward, st_rmsnorm_backward_workspace_bytes)


def _torch():
    import torch
    return torch


class ShardedMLP:
    """Buffers and steps of one MLP branch.

    spatial, shards, batch: the volume and its per-axis shard sizes, as
    ShardedAttention takes them; channels: of the volume; hidden: of the wide
    product.  The stream is fp32 (with products="mx8" the output is bf16).
    """

    def __init__(self, spatial: Sequence[int], shards, channels: int, hidden: int, act: str = "gelu", kept: str = "bf16",
                 products: str = "bf16", batch: int = 1, eps: float = 1e-6, scratch: Optional["ShardedMLP"] = None,
                 device: str = "cuda"):
        torch = _torch()
        if not torch.cuda.is_available():
            raise ShardConvError(6, "no GPU: the layer runs only on the HIP library")
        if act not in _ACTS or kept not in ("bf16", "mx8") or products not in ("bf16", "mx8"):
            raise ShardConvError(1, f"ShardedMLP: unknown act, kept or products ({act!r}, {kept!r}, {products!r})")
        if len(shards) != len(spatial) or any(sum(s) != n or min(s) < 1 for s, n in zip(shards, spatial)):
            raise ShardConvError(2, "ShardedMLP: the shard sizes do not add up to the volume")
        if batch < 1 or channels < 1 or hidden < 1:
            raise ShardConvError(1, "ShardedMLP: batch, channels and hidden are at least 1")
        if batch > 1 and math.prod(len(s) for s in shards) > 1:
            raise ShardConvError(4, "a sharded volume is one sample (batch 1)")
        self.channels, self.hidden, self.act, self.kept, self.products, self.eps = channels, hidden, act, kept, products, eps
        cells = [batch]
        for s in shards:                         # shards row-major over their grid, axis 0 outermost
            cells = [a * b for a in cells for b in s]
        self.starts = [sum(cells[:i]) for i in range(len(cells) + 1)]
        self.tokens = t = self.starts[-1]
        # (8-bit products keep nothing: all their buffers are scratch)
        held = lambda k, p: None if p == "mx8" else k  # noqa: E731
        if scratch is not None and (scratch.tokens, scratch.channels, scratch.hidden, scratch.products, held(scratch.kept, scratch.products)) != \
                (t, channels, hidden, products, held(kept, products)):
            raise ShardConvError(2, "ShardedMLP: scratch of a layer of other sizes")
        if scratch is not None and held(kept, products) == "bf16":
            raise ShardConvError(4, "ShardedMLP: with kept=\"bf16\" the buffers are what the backward pass reads: not shared")
        self.device = torch.device(device)
        f32, bf16, dev = torch.float32, torch.bfloat16, self.device
        new = lambda *shape, dt=f32: torch.zeros(*shape, dtype=dt, device=dev)  # noqa: E731
        self.rstd = new(t)
        self._gamma = torch.ones(channels, device=dev)
        self._b_up, self._b_down = new(hidden), new(channels)
        self.gamma = self.b_up = self.b_down = None
        self.normed8 = self.total8 = self.pre8 = self.h8 = self.pre = self.normed = self.h = None
        if products == "mx8":
            self.w_up, self.w_down = mx8_empty(hidden, channels, device), mx8_empty(channels, hidden, device)
            if scratch is None:
                self.total, self.normed8, self.h8 = new(t, channels), mx8_empty(t, channels, device), mx8_empty(t, hidden, device)
                self.y, self.h = new(t, channels, dt=bf16), new(t, hidden, dt=bf16)
            else:
                self.total, self.normed8, self.h8, self.y = scratch.total, scratch.normed8, scratch.h8, scratch.y
                self.h = scratch.h
        else:
            self.w_up, self.w_down = new(hidden, channels, dt=bf16), new(channels, hidden, dt=bf16)
            if scratch is None:
                self.total, self.normed, self.h = new(t, channels), new(t, channels, dt=bf16), new(t, hidden, dt=bf16)
                self.y = new(t, channels)
            else:
                self.total, self.normed, self.h, self.y = scratch.total, scratch.normed, scratch.h, scratch.y
            if kept == "mx8":
                self.normed8, self.total8 = mx8_empty(t, channels, device), mx8_empty(t, channels, device)
                self.pre8 = mx8_empty(t, hidden, device)
            elif act != "none":
                self.pre = new(t, hidden, dt=bf16)
        need = max(st_linear_workspace_bytes(t, channels, hidden, products), st_linear_workspace_bytes(t, hidden, channels, products))
        self.ws = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
        self.grads = None if scratch is None else scratch.grads
        self._scratch = scratch
        torch.cuda.synchronize()             # the steps may run on any stream: nothing is left to fill

    def parts(self, packed) -> list:
        """The shards' views of a packed [tokens, ...] buffer."""
        return [packed[a:b] for a, b in zip(self.starts, self.starts[1:])]

    def set_weights(self, w_up: np.ndarray, w_down: np.ndarray, b_up=None, b_down=None, gamma=None) -> None:
        """w_up [hidden, channels], w_down [channels, hidden] as float32 (rounded to
        the products' type); b_up [hidden], b_down, gamma [channels] or None.  Waits
        for the device before and after: steps on any stream see one set of weights."""
        torch = _torch()

        def put(name, a, to, *shape):
            if a is None:
                return None
            a = np.ascontiguousarray(a, np.float32)
            if a.shape != shape:
                raise ShardConvError(2, f"{name}: expected {shape}, got {a.shape}")
            if isinstance(to, Mx8):
                st_mx8_store(torch.from_numpy(a).to(self.device), to)
                return to
            return to.copy_(torch.from_numpy(a))

        torch.cuda.synchronize()
        put("w_up", w_up, self.w_up, self.hidden, self.channels)
        put("w_down", w_down, self.w_down, self.channels, self.hidden)
        self.b_up = put("b_up", b_up, self._b_up, self.hidden)
        self.b_down = put("b_down", b_down, self._b_down, self.channels)
        self.gamma = put("gamma", gamma, self._gamma, self.channels)
        torch.cuda.synchronize()

    # ------------------------------------------------------------- steps
    def forward(self, x, branch=None, stream=None):
        """x: packed fp32 [tokens, channels], the stream; branch: fp32 or bf16 in the
        same layout, added to it (or None).  Returns (x + branch) + MLP(norm(x +
        branch)) (self.y, written by the next call again)."""
        if self.products == "mx8":
            st_rmsnorm(x, branch, self.gamma, self.eps, total=self.total, y8=self.normed8, stream=stream)
            st_linear(self.normed8, self.w_up, self.b_up, self.h, act=self.act, workspace=self.ws, stream=stream)
            st_mx8_store(self.h, self.h8, stream)
            st_linear(self.h8, self.w_down, self.b_down, self.y, residual=self.total, workspace=self.ws, stream=stream)
            return self.y
        eight = self.kept == "mx8"
        st_rmsnorm(x, branch, self.gamma, self.eps, total=self.total, y=self.normed, y8=self.normed8 if eight else None,
                   rstd=self.rstd, stream=stream)
        if eight:
            st_mx8_store(self.total, self.total8, stream)
        st_linear(self.normed, self.w_up, self.b_up, self.h, act=self.act, pre=self.pre8 if eight else self.pre,
                  workspace=self.ws, stream=stream)
        st_linear(self.h, self.w_down, self.b_down, self.y, residual=self.total, workspace=self.ws, stream=stream)
        return self.y

    def alloc_backward(self) -> None:
        """The buffers of the backward steps.  The first backward() calls it; call
        it before a graph capture whose steps run on another stream than the
        current one."""
        if self.grads is not None:
            return
        if self._scratch is not None:
            self._scratch.alloc_backward()
            self.grads = self._scratch.grads
            return
        torch = _torch()
        t, c, h, dev = self.tokens, self.channels, self.hidden, self.device
        f32, bf16 = torch.float32, torch.bfloat16
        new = lambda *shape, dt=f32: torch.empty(*shape, dtype=dt, device=dev)  # noqa: E731
        need = max(st_linear_workspace_bytes(t, c, h, "bf16", True), st_linear_workspace_bytes(t, h, c, "bf16", True),
                   st_rmsnorm_backward_workspace_bytes(t, c), 16)
        g = {"dh": new(t, h, dt=bf16), "dnorm": new(t, c, dt=bf16), "dx": new(t, c), "dw_up": new(h, c), "db_up": new(h),
             "dw_down": new(c, h), "db_down": new(c), "dgamma": new(c), "ws": new(need, dt=torch.uint8)}
        # Nothing is filled, but the memory may have had another owner, whose work
        # the current stream alone has in order: the steps may run on another.
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.synchronize()
        self.grads = g

    def backward(self, dy, stream=None) -> dict:
        """Gradients of the last forward() for dy (packed fp32 or bf16 [tokens,
        channels]): dx (fp32, packed; at x and at branch), dw_up, db_up, dw_down,
        db_down, dgamma.  Layers that share scratch return the same buffers."""
        if self.products == "mx8":
            raise ShardConvError(4, "ShardedMLP: 8-bit products are forward only")
        if self.grads is None:
            if _stream(stream).value != _stream(None).value and _torch().cuda.is_current_stream_capturing():
                raise ShardConvError(4, "the backward buffers are not there yet: call alloc_backward() before capturing")
            self.alloc_backward()
        g, eight = self.grads, self.kept == "mx8"
        if eight:
            # the hidden values are the activation of the kept pre-activation
            st_mx8_load(self.pre8, self.h, act=self.act, stream=stream)
        st_linear_backward(self.h, self.w_down, dy, g["dh"], g["dw_down"], g["db_down"], workspace=g["ws"], stream=stream)
        st_linear_backward(self.normed8 if eight else self.normed, self.w_up, g["dh"], g["dnorm"], g["dw_up"], g["db_up"],
                           act=self.act, pre=self.pre8 if eight else self.pre, workspace=g["ws"], stream=stream)
        st_rmsnorm_backward(self.total8 if eight else self.total, g["dnorm"], dy, self.gamma, self.rstd, g["dx"], g["dgamma"],
                            g["ws"], stream)
        return {n: g[n] for n in ("dx", "dw_up", "db_up", "dw_down", "db_down", "dgamma")}

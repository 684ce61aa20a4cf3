"""Shared by the tests of the MLP branch's operators: operands of every type with
guards around them, and their 64-bit values.

Roundings, relative to the value: bf16 2^-8, e4m3 2^-4 (its subnormals: half of
2^-9 times the block's scale, which is at most twice the largest magnitude / 224,
or the smallest scale there is, 2^-126: half a step of 2^-136).
"""
import math

import numpy as np
import torch

from oracle import mlp

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
GUARD = 0x5A


def npy(t):
    return t.detach().cpu().double().numpy()


class Operand:
    """[rows, channels] in 'f32', 'bf16' or 'mx8' inside a larger allocation: `extra`
    more elements between rows (a strided view) and two guard rows behind."""

    def __init__(self, lib, rows, channels, dtype, values=None, extra=0):
        self.rows, self.channels, self.dtype = rows, channels, dtype
        if dtype == "mx8":
            wide, sw = -(-(channels + extra) // 16) * 16, -(-channels // 128) * 4 + (4 if extra else 0)
            self.store = torch.full((rows + 2, wide), GUARD, dtype=torch.uint8, device="cuda")
            self.sstore = torch.full((rows + 2, sw), GUARD, dtype=torch.uint8, device="cuda")
            self.t = lib.Mx8(self.store[:rows], self.sstore[:rows], channels)
            if values is not None:
                codes, scales = mlp.mx8_store(npy(values))
                self.store[:rows, :channels] = torch.from_numpy(codes).cuda()
                self.sstore[:rows, :scales.shape[1]] = torch.from_numpy(scales).cuda()
            return
        es = 4 if dtype == "f32" else 2
        wide = channels if not extra else -(-(channels + extra) * es // 16) * 16 // es
        self.store = torch.empty(rows + 2, wide, dtype=TORCH[dtype], device="cuda")
        self.store.view(torch.uint8).fill_(GUARD)
        self.t = self.store[:rows, :channels]
        if values is not None:
            self.t.copy_(values)

    def values(self):
        """What the rows stand for, in 64 bits."""
        if self.dtype == "mx8":
            return mlp.mx8_values(self.t.codes.cpu().numpy(), self.t.scales.cpu().numpy(), self.channels)
        return npy(self.t)

    def check_guards(self):
        r, c = self.rows, self.channels
        if self.dtype == "mx8":
            blocks = -(-c // 32)
            assert bool((self.store[r:] == GUARD).all()) and bool((self.store[:, c:] == GUARD).all())
            assert bool((self.sstore[r:] == GUARD).all()) and bool((self.sstore[:, blocks:] == GUARD).all())
            return
        raw = self.store.view(torch.uint8)
        es = self.store.element_size()
        assert bool((raw[r:] == GUARD).all()) and bool((raw[:, c * es:] == GUARD).all())


def rounding(values, dtype):
    """Half a step of the type at these values (mx8: with the block's subnormals)."""
    if dtype == "f32":
        return 0.0
    a = np.abs(values)
    if dtype == "bf16":
        return 2.0 ** -8 * a * 1.001
    c = a.shape[1]
    pad = np.pad(a, ((0, 0), (0, -c % 32)))
    top = pad.reshape(a.shape[0], -1, 32).max(-1)
    return 2.0 ** -4 * a * 1.001 + (2.0 ** -136 + 2.0 ** -10 * 2 / 224 * 1.001 * top)[:, np.arange(c) // 32]


def within(name, got, want, tol):
    off = np.abs(got - want)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    assert np.all(off <= tol), f"{name}: off by {off.max():.3g}, over the tolerance by {np.max(off - tol):.3g}"


def sums(n):
    """Error of a sum of n products in fp32, relative to the sum of magnitudes."""
    return 2.0 ** -24 * (8 + 2 * math.sqrt(n))

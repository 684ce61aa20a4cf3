"""The 8-bit form of activations: codes and scales bit for bit against the
definition, and read back exactly."""
import math

import numpy as np
import pytest
import torch

from helpers import say
from mlp_helpers import Operand, TORCH, npy, rounding, within
from oracle import mlp

pytestmark = pytest.mark.gpu


def special(rows, c, dtype, seed):
    """Rows of every size a block may have: tiny and huge, zeros, values on the
    rounding ties and on the scale's border, subnormals of the input."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, c)) * 10.0 ** rng.integers(-6, 6, size=(rows, 1))
    x[rng.random((rows, c)) < 0.05] = 0
    if rows > 4:
        x[1] = 0
        x[2] = rng.choice([1.75, -1.75, 1.875, 1.0, 0.0625 + 1, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10], size=c)
        x[3] = rng.normal(size=c) * 1e-38
        x[4] = rng.normal(size=c) * 1e38
    return torch.from_numpy(x).to(TORCH[dtype])


@pytest.mark.parametrize("rows,c", [(1, 1), (1, 8), (7, 31), (5, 32), (9, 33), (3, 129), (130, 64), (17, 1000), (33, 1001), (6, 4104)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("extra", [0, 40])
def test_codes_bit_for_bit(gpu_lib, rows, c, dtype, extra):
    say(f"mx8 store {rows}x{c} {dtype} extra {extra}")
    x = Operand(gpu_lib, rows, c, dtype, special(rows, c, dtype, rows + c), extra)
    out = Operand(gpu_lib, rows, c, "mx8", extra=extra)
    gpu_lib.st_mx8_store(x.t, out.t)
    torch.cuda.synchronize()
    out.check_guards()
    codes, scales = mlp.mx8_store(x.values())
    assert np.array_equal(out.t.scales.cpu().numpy()[:, :scales.shape[1]], scales)
    got = out.t.codes.cpu().numpy()[:, :c]
    assert np.array_equal(np.where(got == 255, 127, got), codes)      # (NaN has two codes)
    want = out.values()
    finite = np.isfinite(x.values())
    within("stored", np.where(finite, want, 0), np.where(finite, x.values(), 0), rounding(np.where(finite, x.values(), 0), "mx8"))
    for back in ("f32", "bf16"):
        y = Operand(gpu_lib, rows, c, back, extra=extra)
        gpu_lib.st_mx8_load(out.t, y.t)
        torch.cuda.synchronize()
        y.check_guards()
        # below bf16's and fp32's smallest normal number the values keep fewer bits
        whole = finite & (np.abs(want) > 2.0 ** -120)
        told = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)   # rounded up past fp32's largest
        assert np.array_equal(np.isnan(y.values()), ~finite) and np.array_equal(y.values()[whole], told[whole])


def test_special_values(gpu_lib):
    """NaN and infinities take no part in the scale and come back as NaN."""
    v = torch.zeros(2, 64)
    v[0, 3], v[0, 5], v[0, 9], v[0, 40] = math.nan, math.inf, -math.inf, 3.0
    v[0, :3] = 1.5
    x, out = Operand(gpu_lib, 2, 64, "f32", v), Operand(gpu_lib, 2, 64, "mx8")
    gpu_lib.st_mx8_store(x.t, out.t)
    y = Operand(gpu_lib, 2, 64, "f32")
    gpu_lib.st_mx8_load(out.t, y.t)
    got = y.values()
    assert np.isnan(got[0, [3, 5, 9]]).all() and not np.isnan(got[1]).any()
    assert got[0, 40] == 3.0 and (got[0, :3] == 1.5).all() and got[0, 4] == 0


def test_foreign_scales(gpu_lib):
    """Scale bytes that the library does not write: 0 is 2^-127, 255 is NaN."""
    out = Operand(gpu_lib, 3, 64, "mx8", torch.ones(3, 64))
    out.sstore[0, 0], out.sstore[1, 1], out.sstore[2, 0] = 0, 255, 254
    y = Operand(gpu_lib, 3, 64, "f32")
    gpu_lib.st_mx8_load(out.t, y.t)
    got, want = y.values(), out.values()
    assert np.isnan(got[1, 32:]).all() and np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want.astype(np.float32)[ok])       # (256 * 2^127 is infinity there)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_load_through_activation(gpu_lib, act, out):
    rows, c = 40, 100
    x = Operand(gpu_lib, rows, c, "mx8", torch.from_numpy(np.random.default_rng(3).normal(size=(rows, c)) * 4))
    y = Operand(gpu_lib, rows, c, out)
    gpu_lib.st_mx8_load(x.t, y.t, act=act)
    torch.cuda.synchronize()
    y.check_guards()
    want = mlp.activate(x.values(), act)
    # the activation in fp32: a few steps of 2^-24 on values and exponents of up to z^2
    z = np.abs(x.values())
    tol = 2.0 ** -24 * (16 + 2 * z * z) * np.minimum(z, np.abs(want) + 0.2) + rounding(want, out)
    within(act, y.values(), want, tol)


def test_many_rows_past_32_bits(gpu_lib):
    """More than 2^32 bytes of input: the last rows."""
    rows, c = (1 << 21) + 5, 1032
    x = torch.empty(rows, c, dtype=torch.bfloat16, device="cuda")
    tail = torch.from_numpy(np.random.default_rng(4).normal(size=(7, c))).to(torch.bfloat16)
    x.fill_(1.0)
    x[-7:].copy_(tail)
    out = gpu_lib.mx8_empty(rows, c)
    gpu_lib.st_mx8_store(x, out)
    back = torch.empty_like(x)
    gpu_lib.st_mx8_load(out, back)
    codes, scales = mlp.mx8_store(npy(tail))
    assert np.array_equal(out.codes[-7:, :c].cpu().numpy(), codes) and np.array_equal(out.scales[-7:, :scales.shape[1]].cpu().numpy(), scales)
    assert np.array_equal(npy(back[-7:]), mlp.mx8_values(codes, scales, c))
    assert bool((back[:-7] == 1).all())

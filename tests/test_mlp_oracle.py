"""The fp64 definitions of the MLP branch's operators: gradients against central
differences, the 8-bit form against torch's own e4m3, and a planted mistake that
the differences must show."""
import numpy as np
import pytest
import torch

from oracle import mlp

TOL = 1e-7        # central differences at h = 1e-5 in 64 bits


def difference(f, x, t, h=1e-5):
    return (f(x + h * t) - f(x - h * t)) / (2 * h)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_linear_gradient(act):
    rng = np.random.default_rng(1)
    at = [rng.normal(size=(5, 6)), rng.normal(size=(4, 6)), rng.normal(size=4)]
    dy = rng.normal(size=(5, 4))
    pre = mlp.linear(*at)[1]
    assert np.abs(pre).min() > 1e-3                      # (relu: away from its corner)
    grads = mlp.linear_backward(at[0], at[1], dy, act, pre)
    for i, grad in enumerate(grads):
        t = rng.normal(size=grad.shape)

        def f(v):
            return float((mlp.linear(*[v if j == i else a for j, a in enumerate(at)], act=act)[0] * dy).sum())

        d = difference(f, at[i], t)
        assert abs(d - float((grad * t).sum())) < TOL * (1 + abs(d))
        assert abs(d - float((1.01 * grad * t).sum())) > TOL * (1 + abs(d))   # a planted mistake shows


def test_rms_norm_gradient():
    rng = np.random.default_rng(2)
    s, gamma, dy, dt = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dx, dg = mlp.rms_norm_backward(s, dy, dt, gamma)
    for grad, i in ((dx, 0), (dg, 1)):
        t = rng.normal(size=grad.shape)

        def f(v):
            a = [v if j == i else u for j, u in enumerate((s, gamma))]
            return float((mlp.rms_norm(*a)[0] * dy).sum() + (a[0] * dt).sum())

        d = difference(f, (s, gamma)[i], t)
        assert abs(d - float((grad * t).sum())) < TOL * (1 + abs(d))


def test_codes_against_torch():
    table = mlp.e4m3_table()
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(table), np.isnan(want)) and np.array_equal(table[~np.isnan(want)], want[~np.isnan(want)])


def test_store_rounds_to_nearest_even_and_never_saturates():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(40, 70)) * 10.0 ** rng.integers(-20, 20, size=(40, 1))
    codes, scales = mlp.mx8_store(x)
    assert codes.shape == (40, 70) and scales.shape == (40, 3)
    v = mlp.mx8_values(codes, scales, 70)
    block = np.arange(70) // 32
    k = scales[:, block].astype(int) - 127
    u = torch.from_numpy(np.ldexp(x, -k)).float().to(torch.float8_e4m3fn)   # (float32 holds enough: no double rounding at ties)
    assert np.mean(u.view(torch.uint8).numpy() == codes) > 0.999
    top = np.abs(x).reshape(40, -1).max()
    assert top > 0 and np.all(np.abs(v) <= 448 * 2.0 ** k) and np.all(np.abs(v - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** (k - 10.0))
    # the scale is the smallest that holds the block
    for b in range(3):
        m = np.abs(x[:, 32 * b:32 * b + 32]).max(1)
        assert np.all(m <= 448 * 2.0 ** k[:, 32 * b]) and np.all(m > 448 * 2.0 ** (k[:, 32 * b] - 1.0))

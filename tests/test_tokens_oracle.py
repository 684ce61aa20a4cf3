"""The fp64 definitions of the token operators: their gradients against central
differences, and a planted mistake that the differences must show."""
import numpy as np
import pytest

from oracle import tokens


def difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


# central differences at h = 1e-5 in 64 bits: truncation ~ h^2 = 1e-10 and
# rounding ~ 1e-16 / h = 1e-11 times the function's size
TOL = 1e-7


@pytest.mark.parametrize("shape", [(3, 2), (5, 8), (2, 3, 33)])
def test_layer_norm_gradient(shape):
    rng = np.random.default_rng(1)
    x, dy, gamma, beta = rng.normal(size=shape), rng.normal(size=shape), rng.normal(size=shape[-1]), rng.normal(size=shape[-1])
    dx, dg, db = tokens.layer_norm_backward(x, dy, gamma)
    for grad, arg in ((dx, 0), (dg, 1), (db, 2)):
        at = [x, gamma, beta]
        t = rng.normal(size=grad.shape)

        def f(v):
            return float((tokens.layer_norm(*[v if i == arg else a for i, a in enumerate(at)])[0] * dy).sum())

        assert abs(difference(f, at[arg], t) - float((grad * t).sum())) < TOL * (1 + abs(float((grad * t).sum())))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens", [([3, 0, 5], [3, 0, 5]), ([4, 1, 2], [7, 0, 1])])
def test_attention_gradient(causal, q_lens, k_lens):
    rng = np.random.default_rng(2)
    q = rng.normal(size=(sum(q_lens), 4, 8))
    k, v = rng.normal(size=(2, sum(k_lens), 2, 8))
    dout = rng.normal(size=q.shape)
    r = tokens.attention(q, k, v, q_lens, k_lens, 0.4, causal, dout)
    for name, arg in (("dq", 0), ("dk", 1), ("dv", 2)):
        at = [q, k, v]
        t = rng.normal(size=at[arg].shape)

        def f(x):
            args = [x if i == arg else a for i, a in enumerate(at)]
            return float((tokens.attention(*args, q_lens, k_lens, 0.4, causal)["out"] * dout).sum())

        want = float((r[name] * t).sum())
        assert abs(difference(f, at[arg], t) - want) < TOL * (1 + abs(want))


def test_a_wrong_gradient_shows():
    """The check above sees dk without its scale."""
    rng = np.random.default_rng(3)
    q, k, v, dout = rng.normal(size=(4, 6, 1, 8))
    r = tokens.attention(q, k, v, [6], [6], 0.4, False, dout)
    t = rng.normal(size=k.shape)

    def f(x):
        return float((tokens.attention(q, x, v, [6], [6], 0.4, False)["out"] * dout).sum())

    assert abs(difference(f, k, t) - float((r["dk"] / 0.4 * t).sum())) > 1e-3


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_rope_is_a_rotation(pairs):
    rng = np.random.default_rng(4)
    x = rng.normal(size=(7, 3, 14))
    pos = rng.integers(0, 100, size=(7, 2))
    y = tokens.rope(x, pos, [4, 6], pairs=pairs, rotated_heads=2)
    back = tokens.rope(y, pos, [4, 6], pairs=pairs, rotated_heads=2, inverse=True)
    assert np.abs(back - x).max() < 1e-13
    assert np.array_equal(y[:, 2], x[:, 2]) and np.array_equal(y[..., 10:], x[..., 10:])
    # relative positions alone: the product of two rotated rows depends on the
    # difference of their positions
    a, b = rng.normal(size=(2, 1, 1, 14))
    dots = [float((tokens.rope(a, [[p + 5, p + 1]], [4, 6], pairs=pairs) * tokens.rope(b, [[p, p]], [4, 6], pairs=pairs)).sum())
            for p in (0, 3, 50)]
    assert max(dots) - min(dots) < 1e-12


def test_rows_without_keys_are_zero():
    rng = np.random.default_rng(5)
    q, dout = rng.normal(size=(2, 5, 1, 8))
    k, v = rng.normal(size=(2, 2, 1, 8))
    r = tokens.attention(q, k, v, [5], [2], 0.3, True, dout)
    assert np.all(r["out"][:3] == 0) and np.all(np.isneginf(r["lse"][:3])) and np.all(r["dq"][:3] == 0)
    assert np.all(np.isfinite(r["lse"][3:]))

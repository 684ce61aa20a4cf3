"""Vectors beside the rows (bias, gamma, rstd, dgamma, dbias) that share bytes with an
output, or are outputs in an input's or each other's place: refused before any launch."""
import pytest

import halo_sharded_conv_amd as hsc
from test_mlp_host import AT, BAD_SHAPE, F32, MX8, WORKSPACE, lib, rows

V = lambda i, at=0: AT + (i << 36) + at  # noqa: E731
N, C = 8, 64


# operand 2 is total (fp32), 3 y (bf16), 4 y8 (codes, scales half way to 5)
@pytest.mark.parametrize("gamma,rstd", [
    (V(2), V(10)), (V(2, 4 * 63 * 4), V(10)), (V(3), V(10)), (V(3, N * C * 2 - 16), V(10)), (V(4), V(10)), (V(4, 1 << 35), V(10)),
    (V(9), V(0)), (V(9), V(1)), (V(9), V(2)), (V(9), V(3, 64)), (V(9), V(4, 16)), (V(9), V(9)), (V(9), V(9, 4 * C - 16)),
])
def test_rms_norm(gamma, rstd):
    assert lib.st_rmsnorm(N, C, rows(0, C), rows(1, C), gamma, 1e-6, rows(2, C, F32), rows(3, C), rows(4, C, MX8), rstd, None) == BAD_SHAPE


@pytest.mark.parametrize("gamma,rstd,dgamma", [
    (V(3), V(10), V(11)), (V(9), V(3), V(11)), (V(9), V(10), V(0)), (V(9), V(10), V(1)), (V(9), V(10), V(2)), (V(9), V(10), V(3)),
    (V(9), V(10), V(9)), (V(9), V(10), V(10)), (V(9), V(10, 4 * C), V(10, 16)),
])
def test_rms_norm_backward(gamma, rstd, dgamma):
    need = hsc.st_rmsnorm_backward_workspace_bytes(N, C)
    assert lib.st_rmsnorm_backward(N, C, rows(0, C), rows(1, C), rows(2, C), gamma, rstd, rows(3, C), dgamma, V(12), need, None) == BAD_SHAPE


@pytest.mark.parametrize("bias", [V(3), V(3, N * C * 4 - 16), V(4), V(4, 1 << 35)])
def test_linear(bias):
    need = hsc.st_linear_workspace_bytes(N, C, C, "bf16")
    assert lib.st_linear(N, C, C, rows(0, C), rows(1, C), bias, 0, rows(2, C), rows(3, C, F32), rows(4, C, MX8), V(12), need, None) == BAD_SHAPE


END = C * C * 4 - 16


# without rows dw and dbias are cleared all the same
@pytest.mark.parametrize("n,dbias", [*((N, V(i)) for i in range(6)), (N, V(5, END)), (0, V(1)), (0, V(5)), (0, V(5, END))])
def test_linear_backward(n, dbias):
    need = hsc.st_linear_workspace_bytes(N, C, C, "bf16", backward=True)
    assert lib.st_linear_backward(n, C, C, rows(0, C), rows(1, C), 1, rows(2, C), rows(3, C), rows(4, C, F32), rows(5, C, F32), dbias, V(12),
                                  need, None) == BAD_SHAPE


def test_vectors_apart_are_taken():
    """Side by side is not together, nor is a vector between the rows of a wider buffer:
    the next refusal comes, of a workspace that is missing."""
    need = hsc.st_linear_workspace_bytes(N, 60, C, "bf16")
    assert need > 0

    def linear(y, bias):
        return lib.st_linear(N, 60, C, rows(0, 60), rows(1, 60), bias, 0, None, y, None, None, 0, None)

    assert linear(rows(3, C, F32), V(3, N * C * 4)) == WORKSPACE and linear(rows(3, C, F32), V(3, -C * 4)) == WORKSPACE
    assert linear(rows(3, 3 * C, F32), V(3, C * 4)) == WORKSPACE and linear(rows(3, 3 * C, F32), V(3, 8 * C * 4)) == WORKSPACE
    for at in (C * 4 - 16, 2 * C * 4 + 16, 3 * C * 4, (N - 1) * 3 * C * 4 + 16):
        assert linear(rows(3, 3 * C, F32), V(3, at)) == BAD_SHAPE

"""Host side of the MLP branch's operators: argument checks of the C entry points
and workspace sizes (no call here reaches a launch)."""
import ctypes

import pytest
import torch

import halo_sharded_conv_amd as hsc

OK, INVALID, BAD_SHAPE, TOO_SMALL, UNSUPPORTED, WORKSPACE, HIP, ALIGN = range(8)
lib = hsc.lib
F32, BF16, MX8 = 0, 1, 2
AT = 1 << 40                                              # operands far apart, never touched


def rows(i, stride, dtype=BF16, data=None, scales=None, ss=None):
    p = AT + (i << 36)
    return hsc._PACK(p if data is None else data, (p + (1 << 35) if scales is None else scales) if dtype == MX8 else 0, stride,
                     (-(-stride // 128) * 4 if ss is None else ss) if dtype == MX8 else 0, dtype)


def test_mx8_refusals():
    def store(n=4, c=64, x=rows(0, 64, F32), out=rows(1, 64, MX8)):
        return lib.st_mx8_store(n, c, x, out, None)

    assert store(n=-1) == INVALID and store(c=0) == INVALID and store(n=1 << 31) == UNSUPPORTED and store(c=1 << 31) == UNSUPPORTED
    assert store(x=None) == INVALID and store(out=None) == INVALID
    assert store(x=rows(0, 64, MX8)) == INVALID and store(out=rows(1, 64, F32)) == INVALID and store(x=rows(0, 64, 7)) == INVALID
    assert store(x=rows(0, 63, F32)) == BAD_SHAPE and store(x=rows(0, 65, F32)) == ALIGN and store(x=rows(0, 64, F32, data=AT + 4)) == ALIGN
    assert store(x=rows(0, 64, F32, data=0)) == INVALID and store(out=rows(1, 64, MX8, scales=0)) == INVALID
    assert store(out=rows(1, 72, MX8)) == ALIGN and store(out=rows(1, 64, MX8, ss=1)) == BAD_SHAPE and store(out=rows(1, 64, MX8, ss=6)) == ALIGN
    assert store(out=rows(1, 64, MX8, scales=AT + 8)) == ALIGN
    assert store(out=rows(1, 64, MX8, data=AT + 512)) == BAD_SHAPE and store(out=rows(1, 64, MX8, scales=AT + 16)) == BAD_SHAPE
    assert store(n=0, x=rows(0, 64, F32, data=0), out=rows(1, 64, MX8, data=0, scales=0)) == OK
    # off the 8-bit form's grid rows cannot lie back to back; fp32 and bf16 rows can
    assert store(c=65, x=rows(0, 65, F32), out=rows(1, 65, MX8)) == ALIGN
    load = lib.st_mx8_load
    assert load(4, 64, rows(0, 64, MX8), 4, rows(1, 64), None) == INVALID and load(4, 64, rows(0, 64, MX8), -1, rows(1, 64), None) == INVALID
    assert load(4, 64, rows(0, 64, F32), 0, rows(1, 64), None) == INVALID and load(4, 64, rows(0, 64, MX8), 0, rows(0, 64), None) == BAD_SHAPE


def test_views_of_one_buffer():
    """Columns 0..63 and 60..123 of one buffer of 128 channels share bytes."""
    y = rows(0, 128, F32, data=AT + 60 * 4)
    assert lib.st_rmsnorm(1 << 20, 64, rows(0, 128, F32), None, None, 1e-6, y, None, None, None, None) == BAD_SHAPE


def test_rms_norm_refusals():
    def norm(n=4, c=64, x=rows(0, 64), r=rows(1, 64), g=AT + (9 << 36), eps=1e-6, t=rows(2, 64), y=rows(3, 64), y8=rows(4, 64, MX8), rstd=None):
        return lib.st_rmsnorm(n, c, x, r, g, eps, t, y, y8, rstd, None)

    assert norm(n=-1) == INVALID and norm(c=0) == INVALID and norm(c=16385) == UNSUPPORTED and norm(n=1 << 31) == UNSUPPORTED
    assert norm(eps=-1.0) == INVALID and norm(eps=float("nan")) == INVALID and norm(eps=float("inf")) == INVALID
    assert norm(g=AT + 4) == ALIGN and norm(rstd=AT + 4) == ALIGN and norm(x=None) == INVALID
    assert norm(t=None, y=None, y8=None) == INVALID
    assert norm(x=rows(0, 64, MX8)) == INVALID and norm(y=rows(3, 64, MX8)) == INVALID and norm(y8=rows(4, 64)) == INVALID
    assert norm(y=rows(0, 64)) == BAD_SHAPE and norm(y=rows(2, 64)) == BAD_SHAPE and norm(t=rows(0, 64, F32)) == BAD_SHAPE
    assert norm(t=rows(0, 72)) == BAD_SHAPE
    assert norm(n=0, x=rows(0, 64, data=0), r=None, t=None, y=rows(3, 64, data=0), y8=None) == OK
    need = hsc.st_rmsnorm_backward_workspace_bytes(4, 64)
    assert need > 0 and hsc.st_rmsnorm_backward_workspace_bytes(4, 16385) == 0 and hsc.st_rmsnorm_backward_workspace_bytes(-1, 4) == 0

    def back(s=rows(0, 64), dy=rows(1, 64), dt=rows(2, 64), rstd=AT + (9 << 36), dx=rows(3, 64), dg=AT + (10 << 36), ws=AT + (11 << 36), nb=need, c=64):
        return lib.st_rmsnorm_backward(4, c, s, dy, dt, None, rstd, dx, dg, ws, nb, None)

    assert back(rstd=None) == INVALID and back(ws=None) == WORKSPACE and back(nb=need - 1) == WORKSPACE and back(dg=AT + 8) == ALIGN
    assert back(dx=rows(0, 64)) == BAD_SHAPE and back(dx=rows(1, 64, F32)) == BAD_SHAPE and back(dy=rows(1, 64, MX8)) == INVALID
    assert back(dx=None) == INVALID and back(c=16385) == UNSUPPORTED


def test_linear_refusals():
    need = hsc.st_linear_workspace_bytes(4, 60, 64, "bf16")   # rows of 120 bytes: padded copies
    assert need >= 68 * 128

    def linear(n=4, k=60, m=64, x=rows(0, 60), w=rows(1, 60), b=None, act=0, r=rows(2, 64), y=rows(3, 64), pre=rows(4, 64), ws=AT + (9 << 36), nb=need):
        return lib.st_linear(n, k, m, x, w, b, act, r, y, pre, ws, nb, None)

    assert linear(n=-1) == INVALID and linear(k=0) == INVALID and linear(m=0) == INVALID
    assert linear(n=1 << 30) == UNSUPPORTED and linear(k=1 << 24) == UNSUPPORTED and linear(m=1 << 24) == UNSUPPORTED
    assert linear(act=4) == INVALID and linear(b=AT + 4) == ALIGN and linear(ws=AT + 4) == ALIGN
    assert linear(ws=None) == WORKSPACE and linear(nb=need - 1) == WORKSPACE
    assert linear(x=None) == INVALID and linear(w=None) == INVALID and linear(y=None) == INVALID
    assert linear(x=rows(0, 60, F32)) == INVALID and linear(r=rows(2, 64, MX8)) == INVALID
    assert linear(y=rows(0, 64)) == BAD_SHAPE and linear(y=rows(4, 64)) == BAD_SHAPE and linear(y=rows(2, 64, F32)) == BAD_SHAPE
    assert linear(pre=rows(1, 64)) == BAD_SHAPE and linear(pre=rows(2, 64)) == BAD_SHAPE
    assert linear(x=rows(0, 1 << 21)) == UNSUPPORTED and linear(w=rows(1, 1 << 21)) == UNSUPPORTED
    assert linear(n=0) == OK
    back_need = hsc.st_linear_workspace_bytes(4, 64, 64, "bf16", backward=True)

    def back(x=rows(0, 64), w=rows(1, 64), act=0, pre=rows(2, 64), dy=rows(3, 64), dx=rows(4, 64), dw=rows(5, 64), db=None, ws=AT + (9 << 36), nb=back_need, n=4):
        return lib.st_linear_backward(n, 64, 64, x, w, act, pre, dy, dx, dw, db, ws, nb, None)

    assert back(act=2, pre=None) == INVALID and back(act=9) == INVALID and back(w=rows(1, 64, MX8)) == INVALID
    assert back(x=rows(0, 64, F32)) == INVALID and back(dy=rows(3, 64, MX8)) == INVALID and back(dx=rows(4, 64, MX8)) == INVALID
    assert back(nb=back_need - 1) == WORKSPACE and back(ws=None) == WORKSPACE and back(db=AT + 4) == ALIGN
    assert back(dx=rows(3, 64)) == BAD_SHAPE and back(dw=rows(1, 64)) == BAD_SHAPE and back(dx=rows(5, 64)) == BAD_SHAPE
    assert back(dy=rows(3, 1 << 21)) == UNSUPPORTED


def test_workspace_queries():
    q = hsc.st_linear_workspace_bytes
    assert q(-1, 4, 4, "bf16") == 0 and q(4, 0, 4, "bf16") == 0 and q(4, 4, 4, 5) == 0 and q(4, 64, 64, "mx8", backward=True) == 0
    assert q(0, 64, 64, "bf16") == 0
    for t in ("f32", "bf16", "mx8"):
        assert q(1, 64, 64, t) <= q(4096, 64, 64, t) + (1 << 20)
    assert q(16384, 2048, 8192, "bf16") < 64 << 20        # many tiles: no partial sums
    assert q(8, 16384, 64, "bf16") < 64 << 20


def test_binding_checks():
    t = torch.zeros(4, 64)
    with pytest.raises(hsc.ShardConvError):
        hsc._rows(t, "call", "x", 4, 64, 0)                          # not on a GPU
    with pytest.raises(hsc.ShardConvError):
        hsc.Mx8(torch.zeros(4, 63, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(hsc.ShardConvError):
        hsc.Mx8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8), 64)
    with pytest.raises(hsc.ShardConvError):
        hsc.Mx8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.uint8), 64)
    with pytest.raises(hsc.ShardConvError):
        hsc._act("tanh", "x")
    e = hsc.mx8_empty(3, 33, device="cpu")
    assert e.codes.shape == (3, 48) and e.scales.shape == (3, 4) and e.rows == 3
    assert hsc._rows(None, "call", "x", 4, 4, 0) is None


def test_vectors_of_another_device():
    """Vectors and workspaces beside a call's rows are of the current device too."""
    class Elsewhere:
        is_cuda = True

        def get_device(self):
            return 1

    for check in (lambda: hsc._floats(Elsewhere(), "bias", 4, 0), lambda: hsc._ws_here(Elsewhere(), 0),
                  lambda: hsc._floats(torch.zeros(4), "bias", 16, 0), lambda: hsc._ws_here(torch.zeros(4), 0)):
        with pytest.raises(hsc.ShardConvError):
            check()
    assert not hsc._floats(None, "bias", 4, 0) and hsc._ws_here(None, 0)[1] == 0

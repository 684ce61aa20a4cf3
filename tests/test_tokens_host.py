"""Host side of the token operators: argument checks of the C entry points and
the sequence plan (no call here reaches a launch)."""
import ctypes

import pytest

import halo_sharded_conv_amd as hsc

OK, INVALID, BAD_SHAPE, TOO_SMALL, UNSUPPORTED, WORKSPACE, HIP, ALIGN = range(8)
lib = hsc.lib


def seqs(q, k=None, heads=4, kv=2, dim=64, dtype="bf16", causal=False):
    return hsc.st_plan_sequences(q, k, heads, kv, dim, dtype, causal)


@pytest.mark.parametrize("args,kw,status", [
    (([],), {}, INVALID), (([-1],), {}, INVALID), (([3], [3, 4]), {}, BAD_SHAPE), (([4],), dict(heads=4, kv=3), BAD_SHAPE),
    (([4],), dict(heads=0), INVALID), (([4],), dict(dim=60), UNSUPPORTED), (([4],), dict(dim=136), UNSUPPORTED),
    (([4],), dict(dim=0), UNSUPPORTED), (([4],), dict(dtype=7), INVALID), (([1 << 30],), {}, UNSUPPORTED),
    (([1 << 29] * 5,), dict(heads=1, kv=1), UNSUPPORTED),
])
def test_sequence_plan_refusals(args, kw, status):
    with pytest.raises(hsc.ShardConvError) as e:
        seqs(*args, **kw)
    assert e.value.status == status


def test_sequence_plan_nulls():
    out = ctypes.c_void_p()
    one = (ctypes.c_int32 * 1)(4)
    assert lib.st_plan_sequences(1, one, None, 4, 2, 64, 1, 0, None) == INVALID
    assert lib.st_plan_sequences(1, None, None, 4, 2, 64, 1, 0, ctypes.byref(out)) == INVALID
    assert lib.st_seqs_destroy(None) == INVALID and lib.st_seqs_upload(None, None) == INVALID
    assert lib.st_attention_workspace_bytes(None, 1) == 0
    s = seqs([3])
    s.destroy()
    with pytest.raises(hsc.ShardConvError):
        s.handle


def test_workspace_grows_only_with_splits():
    """Many tiles need no partial results; one token over a long list does, and
    the backward call's need covers both calls."""
    assert hsc.st_attention_workspace_bytes(seqs([4096] * 16)) == 0
    one = seqs([1], [65536])
    f, b = hsc.st_attention_workspace_bytes(one), hsc.st_attention_workspace_bytes(one, backward=True)
    assert 0 < f <= b < 64 << 20
    assert hsc.st_attention_workspace_bytes(seqs([0], [0])) == 0


def view(ptr, t=256, h=64):
    return hsc._Tokens(ptr, t, h)


def call(s, q=None, k=None, v=None, out=None, scale=0.1, lse=None, ws=None, nb=0):
    good = view(1 << 20)
    return lib.st_attention_packed(s, q or good, k or view(1 << 20, 128), v or view(1 << 20, 128), scale, out or good, lse, ws, nb, None)


def test_attention_refusals():
    s = seqs([8])
    h = s.handle
    assert lib.st_attention_packed(None, view(16), view(16), view(16), 0.1, view(16), None, None, 0, None) == INVALID
    assert call(h, scale=0.0) == INVALID and call(h, scale=-1.0) == INVALID and call(h, scale=float("inf")) == INVALID
    assert call(h, q=view(0)) == INVALID
    assert call(h, q=view((1 << 20) + 8)) == ALIGN
    assert call(h, k=view(1 << 20, 132)) == ALIGN
    assert call(h, v=view(1 << 20, 64)) == BAD_SHAPE
    assert call(h, out=view(1 << 20, -256)) == INVALID
    assert call(h, k=view(1 << 20, 1 << 40)) == UNSUPPORTED
    assert call(h, lse=(1 << 20) + 4) == ALIGN
    long = seqs([1], [65536])
    assert call(long.handle) == WORKSPACE
    assert call(long.handle, ws=1 << 20, nb=16) == WORKSPACE
    assert "workspace" in lib.st_last_error().decode()


def test_backward_refusals():
    s = seqs([8])
    q, k = view(1 << 20), view(1 << 20, 128)
    args = dict(q=q, k=k, v=k, out=q, lse=1 << 20, dout=q, scale=0.1, dq=q, dk=k, dv=k, ws=1 << 20, nb=1 << 20)

    def back(**kw):
        a = {**args, **kw}
        return lib.st_attention_packed_backward(s.handle, a["q"], a["k"], a["v"], a["out"], a["lse"], a["dout"], a["scale"],
                                                a["dq"], a["dk"], a["dv"], a["ws"], a["nb"], None)

    assert back(scale=float("nan")) == INVALID
    assert back(lse=None) == INVALID
    assert back(ws=None) == WORKSPACE and back(nb=8) == WORKSPACE
    assert back(dk=view(0, 128)) == INVALID
    assert back(dout=view(1 << 20, 100)) == ALIGN
    assert back(q=None) == INVALID
    assert back(q=view(1 << 20, 64, 1 << 29)) == UNSUPPORTED


def test_empty_batches_do_nothing():
    """No token at all: nothing to read, write or launch."""
    s = seqs([0, 0])
    null = view(0)
    assert lib.st_attention_packed(s.handle, null, null, null, 0.1, null, None, None, 0, None) == OK
    assert lib.st_attention_packed_backward(s.handle, null, null, null, null, None, null, 0.1, null, null, null, None, 0, None) == OK
    dims = (ctypes.c_int32 * 1)(8)
    assert lib.st_rope_axes(None, 0, 0, 0, 0, 1, 1, 8, None, 1, dims, 1e4, 0, 0, None, 0, 0, 0, None) == OK


def test_rope_refusals():
    dims = (ctypes.c_int32 * 2)(8, 8)

    def rope(x=1 << 20, xd=0, xt=64, xh=32, tokens=4, heads=2, rot=2, dim=32, pos=1 << 20, n=2, d=dims, base=1e4, pairs=0,
             out=1 << 21, od=0, ot=64, oh=32):
        return lib.st_rope_axes(x, xd, xt, xh, tokens, heads, rot, dim, pos, n, d, base, pairs, 0, out, od, ot, oh, None)

    assert rope(x=None) == INVALID and rope(pos=None) == INVALID and rope(d=None) == INVALID
    assert rope(xd=5) == INVALID and rope(rot=3) == INVALID and rope(heads=0) == INVALID and rope(tokens=-1) == INVALID
    assert rope(dim=33) == UNSUPPORTED and rope(dim=258) == UNSUPPORTED and rope(n=4) == UNSUPPORTED
    assert rope(dim=14) == BAD_SHAPE and rope(base=0.5) == INVALID and rope(pairs=2) == INVALID
    assert rope(x=(1 << 20) + 4) == ALIGN and rope(oh=16) == BAD_SHAPE and rope(xt=-1) == INVALID
    assert rope(out=1 << 20, od=1) == INVALID
    assert rope(pairs=1, xt=65) == ALIGN


def test_layer_norm_refusals():
    a = hsc.st_plan_shards(2, 1, 8, (4, 4), ((4,), (4,)), (0, 0), "f32")
    b = hsc.st_plan_shards(2, 1, 8, (4, 4), ((2, 2), (4,)), (0, 0), "f32")
    p1, p2 = (ctypes.c_void_p * 1)(1 << 20), (ctypes.c_void_p * 2)(1 << 20, 1 << 21)
    ln = lib.st_layernorm_sharded
    assert ln(None, p1, None, None, 1e-5, a.handle, p1, None, None) == INVALID
    assert ln(a.handle, p1, None, None, 1e-5, b.handle, p2, None, None) == BAD_SHAPE
    assert ln(a.handle, p1, None, None, -1.0, a.handle, p1, None, None) == INVALID
    assert ln(a.handle, (ctypes.c_void_p * 1)(0), None, None, 1e-5, a.handle, p1, None, None) == INVALID
    assert ln(a.handle, (ctypes.c_void_p * 1)(20), None, None, 1e-5, a.handle, p1, None, None) == ALIGN
    assert ln(a.handle, p1, 20, None, 1e-5, a.handle, p1, None, None) == ALIGN
    wide = hsc.st_plan_shards(2, 1, 16385, (1, 1), ((1,), (1,)), (0, 0), "f32")
    assert ln(wide.handle, p1, None, None, 1e-5, wide.handle, p1, None, None) == UNSUPPORTED
    assert lib.st_layernorm_backward_workspace_bytes(None) == 0 and hsc.st_layernorm_backward_workspace_bytes(wide) == 0
    back = lib.st_layernorm_backward
    need = hsc.st_layernorm_backward_workspace_bytes(a)
    assert need > 0
    assert back(a.handle, p1, a.handle, p1, None, None, a.handle, p1, None, None, 1 << 20, need, None) == INVALID
    assert back(a.handle, p1, a.handle, p1, None, 1 << 20, a.handle, p1, None, None, 1 << 20, need - 1, None) == WORKSPACE
    assert back(a.handle, p1, b.handle, p2, None, 1 << 20, a.handle, p1, None, None, 1 << 20, need, None) == BAD_SHAPE


def test_positions_refusals():
    a = hsc.st_plan_shards(2, 1, 8, (4, 4), ((4,), (4,)), (0, 0), "f32")
    assert lib.st_plan_positions(None, None, None) == INVALID
    assert lib.st_plan_positions(a.handle, (ctypes.c_void_p * 1)(0), None) == INVALID
    assert lib.st_plan_positions(a.handle, (ctypes.c_void_p * 1)(20), None) == ALIGN


class Device:
    """A tensor of some type on the GPU, at an address that no call accepts."""
    is_cuda = True

    def __init__(self, dtype, n=1 << 20):
        self.dtype, self.nbytes = dtype, n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4


def test_types_that_are_not_read_as_bits():
    """Every buffer of the layer norm, the positions and lse has its type or is
    raw bits; the right types get as far as the address."""
    f32, bf16 = hsc.st_plan_shards(2, 1, 8, (4, 4), ((4,), (4,)), (0, 0), "f32"), hsc.st_plan_shards(
        2, 1, 8, (4, 4), ((4,), (4,)), (0, 0), "bf16")
    t = hsc._torch()
    x, y, s = Device(t.float32), Device(t.bfloat16), Device(t.float32)

    def status(f):
        with pytest.raises(hsc.ShardConvError) as e:
            f()
        return e.value.status

    def forward(x=x, y=y, g=s, b=s, st=s):
        return status(lambda: hsc.st_layernorm_sharded(f32, [x], g, b, 1e-5, bf16, [y], st, stream=0))

    def backward(x=x, dy=y, g=s, st=s, dx=x, dg=s, db=s):
        return status(lambda: hsc.st_layernorm_backward(f32, [x], bf16, [dy], g, st, f32, [dx], dg, db, s, stream=0))

    assert forward() == ALIGN and backward() == ALIGN
    assert forward(x=Device(t.int32), y=Device(t.int16), st=Device(t.uint8)) == ALIGN
    for wrong in (t.float64, t.float16, t.bfloat16, t.int64):
        w = Device(wrong)
        assert [forward(x=w), forward(g=w), forward(b=w), forward(st=w)] == [INVALID] * 4, wrong
        assert [backward(x=w), backward(g=w), backward(st=w), backward(dx=w), backward(dg=w), backward(db=w)] == [INVALID] * 6
    for wrong in (t.float32, t.float16, t.int32):
        assert forward(y=Device(wrong)) == INVALID and backward(dy=Device(wrong)) == INVALID, wrong
    assert status(lambda: hsc.st_plan_positions(f32, [Device(t.int32)], stream=0)) == ALIGN
    for wrong in (t.int64, t.int16, t.float32):
        assert status(lambda: hsc.st_plan_positions(f32, [Device(wrong)], stream=0)) == INVALID
    one = seqs([8])
    for wrong in (t.float64, t.bfloat16, t.int64):
        assert status(lambda: hsc.st_attention_packed(one, None, None, None, 0.1, None, Device(wrong), stream=0)) == INVALID
        assert status(lambda: hsc.st_attention_packed_backward(one, *[None] * 4, Device(wrong), None, 0.1, *[None] * 4, stream=0)) == INVALID


def test_backward_strides():
    """Token strides up to 2^30 bytes over a tile's tokens pass (the call then
    lacks its workspace); the outputs' have the forward call's limit."""
    def back(s, es, **big):
        q, k = view(1 << 20), view(1 << 20, 128)
        args = dict(q=q, k=k, v=k, out=q, dout=q, dq=q, dk=k, dv=k)
        args.update({n: view(1 << 20, t // es) for n, t in big.items()})
        a = [args[n] for n in ("q", "k", "v", "out")] + [1 << 20, args["dout"], 0.1] + [args[n] for n in ("dq", "dk", "dv")]
        return lib.st_attention_packed_backward(s.handle, *a, None, 0, None)

    half, single, wide = seqs([8]), seqs([8], dtype="f32"), seqs([8], dim=128, dtype="f32", heads=2, kv=2)
    for s, es in ((half, 2), (single, 4)):
        assert back(s, es, **{n: 1 << 24 for n in ("q", "k", "v", "dout")}) == WORKSPACE
        assert back(s, es, **{n: 1 << 30 for n in ("out", "dq", "dk", "dv")}) == WORKSPACE
        for n in ("q", "k", "v", "dout"):
            assert back(s, es, **{n: (1 << 24) + 16}) == UNSUPPORTED, n
        for n in ("out", "dq", "dk", "dv"):
            assert back(s, es, **{n: (1 << 30) + 16}) == UNSUPPORTED, n
    kv = view(1 << 20, 256, 128)

    def wide_v(t):
        q, v = view(1 << 20, 256, 128), view(1 << 20, t // 4, 128)
        return lib.st_attention_packed_backward(wide.handle, q, kv, v, q, 1 << 20, q, 0.1, q, kv, kv, None, 0, None)

    assert wide_v(1 << 23) == WORKSPACE and wide_v((1 << 23) + 16) == UNSUPPORTED


def test_every_entry_point_is_exported():
    """`from halo_sharded_conv_amd import *` brings every function of the binding
    and the classes they return."""
    functions = {n for n in vars(hsc) if n.startswith("st_") and callable(getattr(hsc, n))}
    assert functions | {"Plan", "Sequences"} <= set(hsc.__all__)
    assert all(hasattr(hsc, n) for n in hsc.__all__)


def test_positions_are_not_read_across_rows():
    """[tokens, 3] positions with two sections."""
    t = hsc._torch()

    class Rows(Device):
        def __init__(self, dtype, *shape):
            super().__init__(dtype)
            self.shape = shape

        def dim(self):
            return len(self.shape)

        def numel(self):
            return 1

        def stride(self, i):
            return (128, 64, 1)[i]

    x = Rows(t.float32, 6, 2, 64)

    def status(*shape):
        with pytest.raises(hsc.ShardConvError) as e:
            hsc.st_rope_axes(x, Rows(t.int32, *shape), [32, 32], x, stream=0)
        return e.value.status

    assert status(6, 3) == BAD_SHAPE and status(6, 1) == BAD_SHAPE and status(2, 3, 3) == BAD_SHAPE
    assert status(6, 2) == ALIGN and status(12) == ALIGN and status(2, 3, 2) == ALIGN

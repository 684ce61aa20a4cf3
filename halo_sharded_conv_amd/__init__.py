"""Python binding of libshardconv (the halo-sharded conv + GroupNorm library).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  torch tensors supply device memory and the current stream.  The
binding fails loudly if the library is missing or a tensor is not on a GPU;
there is no CPU fallback.

Names match the C-ABI in include/shardconv.h (st_plan_shards, st_halo_pack,
st_halo_unpack, st_conv_sharded, st_groupnorm_sharded, ...).
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import List, Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libshardconv.so")

ST_F32, ST_BF16 = 0, 1
ST_MAX_SHARDS = 64
DTYPES = {"f32": ST_F32, "bf16": ST_BF16}
ESIZE = {ST_F32: 4, ST_BF16: 2}


class ShardConvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class _ShardInfo(ctypes.Structure):
    _fields_ = [("index", ctypes.c_int32), ("grid", ctypes.c_int32 * 3),
                ("offset", ctypes.c_int64 * 3), ("extent", ctypes.c_int64 * 3),
                ("padded", ctypes.c_int64 * 3), ("elems", ctypes.c_int64),
                ("bytes", ctypes.c_int64)]


class _HaloBox(ctypes.Structure):
    _fields_ = [("src_shard", ctypes.c_int32), ("dst_shard", ctypes.c_int32),
                ("dir", ctypes.c_int32 * 3), ("dst_lo", ctypes.c_int64 * 3),
                ("src_lo", ctypes.c_int64 * 3), ("ext", ctypes.c_int64 * 3),
                ("msg_offset", ctypes.c_int64)]


class _Tokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _GnLayout(ctypes.Structure):
    _fields_ = [("partials_offset", ctypes.c_size_t), ("stats_offset", ctypes.c_size_t),
                ("scales_offset", ctypes.c_size_t), ("ymax_offset", ctypes.c_size_t),
                ("chan_offset", ctypes.c_size_t), ("total_bytes", ctypes.c_size_t)]


def _hip_runtimes() -> list:
    """Paths of every HIP runtime library mapped into this process."""
    try:
        with open("/proc/self/maps") as f:
            return sorted({ln.split()[-1] for ln in f if "libamdhip64" in ln})
    except OSError:
        return []


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python halo_sharded_conv_amd/build.py`")
    # torch ships its own HIP runtime and its libraries ask for it by a name
    # that does not match an already loaded libamdhip64.so.7.  Loading torch
    # first lets this library bind to torch's runtime (same soname), so
    # torch's streams and allocations and these kernels share one runtime.
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    runtimes = _hip_runtimes()
    if len(runtimes) > 1:
        raise ImportError(f"two HIP runtimes are loaded ({runtimes}); import torch before any other HIP library")
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    PP = ctypes.POINTER(ctypes.c_void_p)
    PI32, PT = ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(_Tokens)
    PR = ctypes.c_char_p                     # an st_rows, packed
    sig = {
        "st_version": (ctypes.c_char_p, []),
        "st_last_error": (ctypes.c_char_p, []),
        "st_status_string": (ctypes.c_char_p, [I32]),
        "st_plan_shards": (I32, [I32, I64, I64, ctypes.POINTER(I64), ctypes.POINTER(I32),
                                 ctypes.POINTER(I64), ctypes.POINTER(I32), I32, ctypes.POINTER(P)]),
        "st_plan_destroy": (I32, [P]),
        "st_plan_num_shards": (I64, [P]),
        "st_plan_msg_bytes": (I64, [P]),
        "st_plan_num_halo_boxes": (I64, [P]),
        "st_plan_num_zero_boxes": (I64, [P]),
        "st_plan_upload": (I32, [P, P]),
        "st_plan_shard_info": (I32, [P, I32, ctypes.POINTER(_ShardInfo)]),
        "st_plan_halo_box": (I32, [P, I32, ctypes.POINTER(_HaloBox)]),
        "st_halo_pack": (I32, [P, PP, P, P]),
        "st_halo_unpack": (I32, [P, P, PP, I32, P]),
        "st_halo_exchange": (I32, [P, PP, I32, P]),
        "st_conv_weight_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "st_conv_pack_weights": (I32, [I32, I32, I32, I32, I32, P, P, P]),
        "st_conv_dgrad_weights": (I32, [I32, I32, I32, I32, I32, P, P, P]),
        "st_conv_workspace_bytes": (SZ, [P, I32, I32]),
        "st_conv_sharded": (I32, [P, PP, P, P, I32, I32, PP, P, I32, P, SZ, P]),
        "st_conv_sharded_packed": (I32, [P, PP, P, P, I32, I32, PP, P, I32, P]),
        "st_plan_pooled": (I32, [P, I32, I32, ctypes.POINTER(I32), I32, ctypes.POINTER(P)]),
        "st_pool_sharded": (I32, [P, PP, I32, I32, I32, P, PP, P]),
        "st_plan_strided": (I32, [P, I32, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(P)]),
        "st_conv_strided_workspace_bytes": (SZ, [P, I32, I32]),
        "st_conv_strided_sharded": (I32, [P, PP, P, P, I32, I32, P, PP, P, SZ, P]),
        "st_plan_transposed": (I32, [P, I32, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(P)]),
        "st_conv_transposed_workspace_bytes": (SZ, [P, I32, I32]),
        "st_conv_transposed_sharded": (I32, [P, PP, P, P, I32, I32, P, PP, P, SZ, P]),
        "st_conv_wgrad_workspace_bytes": (SZ, [P, I32, I32]),
        "st_conv_wgrad": (I32, [P, PP, P, PP, I32, P, P, SZ, P]),
        "st_groupnorm_workspace_bytes": (SZ, [P, I32]),
        "st_groupnorm_workspace_layout": (I32, [P, I32, ctypes.POINTER(_GnLayout)]),
        "st_groupnorm_sharded": (I32, [P, PP, P, I32, ctypes.c_float, P, P, PP, P, SZ, P]),
        "st_groupnorm_sharded_noalloc": (I32, [P, PP, P, I32, ctypes.c_float, P, P, PP, P]),
        "st_groupnorm_partials": (I32, [P, PP, P, I32, P, SZ, P]),
        "st_groupnorm_combine": (I32, [P, I32, ctypes.c_float, P, P, P, SZ, P]),
        "st_groupnorm_apply": (I32, [P, PP, I32, PP, P, SZ, P]),
        "st_groupnorm_combine_apply": (I32, [P, PP, I32, ctypes.c_float, P, P, PP, P, SZ, P]),
        "st_groupnorm_backward_workspace_bytes": (SZ, [P, I32]),
        "st_groupnorm_backward": (I32, [P, PP, PP, P, P, I32, P, P, SZ, P, PP, P, P, P, SZ, P]),
        "st_layernorm_sharded": (I32, [P, PP, P, P, ctypes.c_float, P, PP, P, P]),
        "st_layernorm_backward_workspace_bytes": (SZ, [P]),
        "st_layernorm_backward": (I32, [P, PP, P, PP, P, P, P, PP, P, P, P, SZ, P]),
        "st_plan_positions": (I32, [P, PP, P]),
        "st_rope_axes": (I32, [P, I32, I64, I64, I64, I32, I32, I32, P, I32, PI32, ctypes.c_double, I32, I32, P, I32,
                               I64, I64, P]),
        "st_plan_sequences": (I32, [I32, PI32, PI32, I32, I32, I32, I32, I32, ctypes.POINTER(P)]),
        "st_seqs_destroy": (I32, [P]),
        "st_seqs_upload": (I32, [P, P]),
        "st_attention_workspace_bytes": (SZ, [P, I32]),
        "st_attention_packed": (I32, [P, PT, PT, PT, ctypes.c_float, PT, P, P, SZ, P]),
        "st_attention_packed_backward": (I32, [P, PT, PT, PT, PT, P, PT, ctypes.c_float, PT, PT, PT, P, SZ, P]),
        "st_mx8_store": (I32, [I64, I64, PR, PR, P]),
        "st_mx8_load": (I32, [I64, I64, PR, I32, PR, P]),
        "st_rmsnorm": (I32, [I64, I64, PR, PR, P, ctypes.c_float, PR, PR, PR, P, P]),
        "st_rmsnorm_backward_workspace_bytes": (SZ, [I64, I64]),
        "st_rmsnorm_backward": (I32, [I64, I64, PR, PR, PR, P, P, PR, P, P, SZ, P]),
        "st_linear_workspace_bytes": (SZ, [I64, I64, I64, I32, I32]),
        "st_linear": (I32, [I64, I64, I64, PR, PR, P, I32, PR, PR, PR, P, SZ, P]),
        "st_linear_backward": (I32, [I64, I64, I64, PR, PR, I32, PR, PR, PR, PR, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _check(status: int, what: str) -> None:
    if status != 0:
        msg = lib.st_last_error().decode()
        name = lib.st_status_string(status).decode()
        raise ShardConvError(status, f"{what}: {name}: {msg}")


def st_version() -> str:
    return lib.st_version().decode()


# ---------------------------------------------------------------- plans

class Plan:
    """Owns an st_plan*; released on destroy() or garbage collection."""

    def __init__(self, handle: int, ndim: int, batch: int, channels: int, dtype: int,
                 shards: Sequence[Sequence[int]], halo: Sequence[int]):
        self._h = ctypes.c_void_p(handle)
        self.ndim, self.batch, self.channels, self.dtype = ndim, batch, channels, dtype
        self.shards = tuple(tuple(s) for s in shards)
        self.halo = tuple(halo)
        self._bytes = self._cells = self._stats = None

    @property
    def handle(self) -> ctypes.c_void_p:
        if not self._h:
            raise ShardConvError(1, "plan already destroyed")
        return self._h

    def destroy(self) -> None:
        if self._h:
            _check(lib.st_plan_destroy(self._h), "st_plan_destroy")
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    @property
    def num_shards(self) -> int:
        return int(lib.st_plan_num_shards(self.handle))

    @property
    def msg_bytes(self) -> int:
        return int(lib.st_plan_msg_bytes(self.handle))

    @property
    def num_halo_boxes(self) -> int:
        return int(lib.st_plan_num_halo_boxes(self.handle))

    @property
    def num_zero_boxes(self) -> int:
        return int(lib.st_plan_num_zero_boxes(self.handle))

    def upload(self, stream=None) -> None:
        """Put the halo descriptor table on the current device now (needed
        before a graph capture that contains the plan's first halo call)."""
        _check(lib.st_plan_upload(self.handle, _stream(stream)), "st_plan_upload")

    def shard_info(self, i: int) -> dict:
        info = _ShardInfo()
        _check(lib.st_plan_shard_info(self.handle, i, ctypes.byref(info)), "st_plan_shard_info")
        d = self.ndim
        return {"index": info.index, "grid": tuple(info.grid[:d]), "offset": tuple(info.offset[:d]),
                "extent": tuple(info.extent[:d]), "padded": tuple(info.padded[:d]),
                "elems": info.elems, "bytes": info.bytes}

    def padded_shape(self, i: int) -> tuple:
        return (self.batch, *self.shard_info(i)["padded"], self.channels)

    def halo_box(self, i: int) -> dict:
        b = _HaloBox()
        _check(lib.st_plan_halo_box(self.handle, i, ctypes.byref(b)), "st_plan_halo_box")
        d = self.ndim
        return {"src": b.src_shard, "dst": b.dst_shard, "dir": tuple(b.dir[:d]),
                "dst_lo": tuple(b.dst_lo[:d]), "src_lo": tuple(b.src_lo[:d]),
                "ext": tuple(b.ext[:d]), "msg_offset": b.msg_offset}


def st_plan_shards(ndim: int, batch: int, channels: int, spatial: Sequence[int],
                   shard_sizes: Sequence[Sequence[int]], halo: Sequence[int], dtype) -> Plan:
    """Plan over per-axis shard sizes (axis 0 outermost); dtype 'f32'/'bf16' or 0/1."""
    dt = DTYPES.get(dtype, dtype)
    n_axes = len(spatial)
    sp = (ctypes.c_int64 * max(1, n_axes))(*spatial)
    counts = (ctypes.c_int32 * max(1, len(shard_sizes)))(*[len(s) for s in shard_sizes])
    flat = [int(v) for s in shard_sizes for v in s]
    sizes = (ctypes.c_int64 * max(1, len(flat)))(*flat)
    hl = (ctypes.c_int32 * max(1, len(halo)))(*halo)
    out = ctypes.c_void_p()
    _check(lib.st_plan_shards(ndim, batch, channels, sp, counts, sizes, hl, dt, ctypes.byref(out)),
           "st_plan_shards")
    return Plan(out.value, ndim, batch, channels, dt, shard_sizes, halo)


# ------------------------------------------------------------ device calls

def _torch():
    import torch
    return torch


def _current_stream() -> int:
    """Handle of the current device's current stream, without building a
    torch.cuda.Stream object (4 us of a 12 us call)."""
    torch = _torch()
    try:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:                   # a torch without these two
        return torch.cuda.current_stream().cuda_stream


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(_current_stream())
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dev_ptr(t, what: str, min_bytes: int = 0) -> int:
    if t is None:
        return 0
    if not getattr(t, "is_cuda", False):
        raise ShardConvError(1, f"{what}: expected a GPU tensor (no CPU fallback exists)")
    if not t.is_contiguous():
        raise ShardConvError(1, f"{what}: tensor must be contiguous")
    if t.nbytes < min_bytes:
        raise ShardConvError(2, f"{what}: tensor holds {t.nbytes} bytes, needs {min_bytes}")
    return t.data_ptr()


def _ptr_array(tensors, what: str, sizes: List[int]):
    if len(tensors) != len(sizes):
        raise ShardConvError(2, f"{what}: expected {len(sizes)} shard buffers, got {len(tensors)}")
    arr = (ctypes.c_void_p * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        if t is not None and getattr(t, "is_cuda", False) and t.is_contiguous() and t.nbytes >= sizes[i]:
            arr[i] = t.data_ptr()
        else:
            arr[i] = _dev_ptr(t, f"{what}[{i}]", sizes[i])   # its message
    return arr


def _shard_bytes(plan: Plan) -> List[int]:
    if plan._bytes is None:                  # fixed for a plan's life
        plan._bytes = [plan.shard_info(i)["bytes"] for i in range(plan.num_shards)]
    return plan._bytes


def st_halo_pack(plan: Plan, shard_bufs, msg, stream=None) -> None:
    arr = _ptr_array(shard_bufs, "st_halo_pack shard", _shard_bytes(plan))
    m = _dev_ptr(msg, "st_halo_pack msg", plan.msg_bytes) if plan.msg_bytes else 0
    _check(lib.st_halo_pack(plan.handle, arr, ctypes.c_void_p(m), _stream(stream)), "st_halo_pack")


def st_halo_unpack(plan: Plan, msg, shard_bufs, zero_global_margins: bool = True, stream=None) -> None:
    arr = _ptr_array(shard_bufs, "st_halo_unpack shard", _shard_bytes(plan))
    m = _dev_ptr(msg, "st_halo_unpack msg", plan.msg_bytes) if plan.msg_bytes else 0
    _check(lib.st_halo_unpack(plan.handle, ctypes.c_void_p(m), arr, int(bool(zero_global_margins)),
                              _stream(stream)), "st_halo_unpack")



def st_halo_exchange(plan: Plan, shard_bufs, zero_global_margins: bool = True, stream=None) -> None:
    arr = _ptr_array(shard_bufs, "st_halo_exchange shard", _shard_bytes(plan))
    _check(lib.st_halo_exchange(plan.handle, arr, int(bool(zero_global_margins)), _stream(stream)),
           "st_halo_exchange")

def st_conv_weight_bytes(ndim: int, cin: int, cout: int, ksize: int, dtype) -> int:
    return int(lib.st_conv_weight_bytes(ndim, cin, cout, ksize, DTYPES.get(dtype, dtype)))


def st_conv_pack_weights(ndim: int, cin: int, cout: int, ksize: int, dtype, weight, packed,
                         stream=None) -> None:
    dt = DTYPES.get(dtype, dtype)
    need = st_conv_weight_bytes(ndim, cin, cout, ksize, dt)
    raw = cout * cin * ksize ** ndim * ESIZE[dt]
    _check(lib.st_conv_pack_weights(ndim, cin, cout, ksize, dt,
                                    ctypes.c_void_p(_dev_ptr(weight, "weight", raw)),
                                    ctypes.c_void_p(_dev_ptr(packed, "packed weight", need)),
                                    _stream(stream)), "st_conv_pack_weights")


def st_conv_dgrad_weights(ndim: int, cin: int, cout: int, ksize: int, dtype, weight, out,
                          stream=None) -> None:
    dt = DTYPES.get(dtype, dtype)
    raw = cout * cin * ksize ** ndim * ESIZE[dt]
    _check(lib.st_conv_dgrad_weights(ndim, cin, cout, ksize, dt,
                                     ctypes.c_void_p(_dev_ptr(weight, "weight", raw)),
                                     ctypes.c_void_p(_dev_ptr(out, "dgrad weight", raw)),
                                     _stream(stream)), "st_conv_dgrad_weights")


def _y_bytes(in_plan: Plan, cout: int) -> List[int]:
    """Bytes of each shard's unpadded fp32 conv output [N][extent...][cout]."""
    out = []
    for i in range(in_plan.num_shards):
        n = in_plan.batch * cout * 4
        for e in in_plan.shard_info(i)["extent"]:
            n *= e
        out.append(n)
    return out


def st_conv_workspace_bytes(in_plan: Plan, cout: int, ksize: int) -> int:
    return int(lib.st_conv_workspace_bytes(in_plan.handle, cout, ksize))


def st_conv_sharded(in_plan: Plan, in_bufs, weight, bias, cout: int, ksize: int, y_bufs, ymax=None,
                    groups: int = 1, workspace=None, stream=None) -> None:
    """weight: raw [Cout][Cin][k..] in the plan's dtype (bf16 as int16/uint16
    bits); workspace: >= st_conv_workspace_bytes bytes."""
    ins = _ptr_array(in_bufs, "st_conv_sharded input", _shard_bytes(in_plan))
    outs = _ptr_array(y_bufs, "st_conv_sharded y", _y_bytes(in_plan, cout))
    raw = cout * in_plan.channels * ksize ** in_plan.ndim * ESIZE[in_plan.dtype]
    w = _dev_ptr(weight, "weight", raw)
    b = _dev_ptr(bias, "bias", 4 * cout)
    ym = _dev_ptr(ymax, "ymax", 4 * in_plan.batch * groups) if ymax is not None else 0
    ws, nb = _ws(workspace)
    _check(lib.st_conv_sharded(in_plan.handle, ins, ctypes.c_void_p(w), ctypes.c_void_p(b), cout, ksize, outs,
                               ctypes.c_void_p(ym), groups, ctypes.c_void_p(ws), nb, _stream(stream)),
           "st_conv_sharded")


def st_conv_sharded_packed(in_plan: Plan, in_bufs, packed_weight, bias, cout: int, ksize: int, y_bufs, ymax=None,
                           groups: int = 1, stream=None) -> None:
    """packed_weight: from st_conv_pack_weights."""
    ins = _ptr_array(in_bufs, "st_conv_sharded_packed input", _shard_bytes(in_plan))
    outs = _ptr_array(y_bufs, "st_conv_sharded_packed y", _y_bytes(in_plan, cout))
    need_w = st_conv_weight_bytes(in_plan.ndim, in_plan.channels, cout, ksize, in_plan.dtype)
    w = _dev_ptr(packed_weight, "packed weight", need_w)
    b = _dev_ptr(bias, "bias", 4 * cout)
    ym = _dev_ptr(ymax, "ymax", 4 * in_plan.batch * groups) if ymax is not None else 0
    _check(lib.st_conv_sharded_packed(in_plan.handle, ins, ctypes.c_void_p(w), ctypes.c_void_p(b), cout, ksize,
                                      outs, ctypes.c_void_p(ym), groups, _stream(stream)),
           "st_conv_sharded_packed")


def st_plan_pooled(in_plan: Plan, ksize: int, stride: int, out_halo=None, out_dtype=None) -> Plan:
    """Output plan of a 'valid' pooling; its shard sizes are derived by the library."""
    dt = in_plan.dtype if out_dtype is None else DTYPES.get(out_dtype, out_dtype)
    hl = (ctypes.c_int32 * 3)(*(list(out_halo) + [0] * (3 - len(out_halo)))) if out_halo is not None else None
    out = ctypes.c_void_p()
    _check(lib.st_plan_pooled(in_plan.handle, ksize, stride, hl, dt, ctypes.byref(out)), "st_plan_pooled")
    halo = tuple(out_halo) if out_halo is not None else (0,) * in_plan.ndim
    probe = Plan(out.value, in_plan.ndim, in_plan.batch, in_plan.channels, dt, (), halo)
    # per-axis shard sizes from the shard table (shards are row-major over the grid)
    n = probe.num_shards
    infos = [probe.shard_info(i) for i in range(n)]
    sizes = []
    for a in range(in_plan.ndim):
        seen = {}
        for inf in infos:
            seen.setdefault(inf["grid"][a], inf["extent"][a])
        sizes.append(tuple(seen[g] for g in sorted(seen)))
    probe.shards = tuple(sizes)
    return probe


def st_pool_sharded(in_plan: Plan, in_bufs, ksize: int, stride: int, mode: str, out_plan: Plan, out_bufs,
                    stream=None) -> None:
    """mode 'avg' or 'max'."""
    ins = _ptr_array(in_bufs, "st_pool_sharded input", _shard_bytes(in_plan))
    outs = _ptr_array(out_bufs, "st_pool_sharded output", _shard_bytes(out_plan))
    m = {"avg": 0, "max": 1}[mode]
    _check(lib.st_pool_sharded(in_plan.handle, ins, ksize, stride, m, out_plan.handle, outs, _stream(stream)),
           "st_pool_sharded")


def _plan_from_handle(handle, ndim, batch, channels, dtype, halo) -> Plan:
    """Wrap a library-derived plan, recovering its per-axis shard sizes."""
    plan = Plan(handle, ndim, batch, channels, dtype, (), halo)
    infos = [plan.shard_info(i) for i in range(plan.num_shards)]
    sizes = []
    for a in range(ndim):
        seen = {}
        for inf in infos:
            seen.setdefault(inf["grid"][a], inf["extent"][a])
        sizes.append(tuple(seen[g] for g in sorted(seen)))
    plan.shards = tuple(sizes)
    return plan


def st_plan_strided(in_plan: Plan, ksize: int, stride: int, cout: int, out_halo=None) -> Plan:
    """fp32 output plan of a strided 'same'-padded conv; shard sizes derived by the library."""
    hl = (ctypes.c_int32 * 3)(*(list(out_halo) + [0] * (3 - len(out_halo)))) if out_halo is not None else None
    out = ctypes.c_void_p()
    _check(lib.st_plan_strided(in_plan.handle, ksize, stride, cout, hl, ctypes.byref(out)), "st_plan_strided")
    return _plan_from_handle(out.value, in_plan.ndim, in_plan.batch, cout, ST_F32,
                             tuple(out_halo) if out_halo is not None else (0,) * in_plan.ndim)


def st_conv_strided_workspace_bytes(in_plan: Plan, cout: int, ksize: int) -> int:
    return int(lib.st_conv_strided_workspace_bytes(in_plan.handle, cout, ksize))


def st_conv_strided_sharded(in_plan: Plan, in_bufs, weight, bias, ksize: int, stride: int, out_plan: Plan,
                            out_bufs, workspace, stream=None) -> None:
    """weight: raw [Cout][Cin][k..] in the input plan's dtype."""
    ins = _ptr_array(in_bufs, "st_conv_strided_sharded input", _shard_bytes(in_plan))
    outs = _ptr_array(out_bufs, "st_conv_strided_sharded output", _shard_bytes(out_plan))
    taps = ksize ** in_plan.ndim
    w = _dev_ptr(weight, "weight", ESIZE[in_plan.dtype] * taps * in_plan.channels * out_plan.channels)
    b = _dev_ptr(bias, "bias", 4 * out_plan.channels)
    ws, nb = _ws(workspace)
    _check(lib.st_conv_strided_sharded(in_plan.handle, ins, ctypes.c_void_p(w), ctypes.c_void_p(b), ksize, stride,
                                       out_plan.handle, outs, ctypes.c_void_p(ws), nb, _stream(stream)),
           "st_conv_strided_sharded")


def st_plan_transposed(in_plan: Plan, ksize: int, stride: int, cout: int, out_halo=None) -> Plan:
    """fp32 output plan of a transposed (upsampling) conv: every shard's extents times stride."""
    hl = (ctypes.c_int32 * 3)(*(list(out_halo) + [0] * (3 - len(out_halo)))) if out_halo is not None else None
    out = ctypes.c_void_p()
    _check(lib.st_plan_transposed(in_plan.handle, ksize, stride, cout, hl, ctypes.byref(out)), "st_plan_transposed")
    return _plan_from_handle(out.value, in_plan.ndim, in_plan.batch, cout, ST_F32,
                             tuple(out_halo) if out_halo is not None else (0,) * in_plan.ndim)


def st_conv_transposed_workspace_bytes(in_plan: Plan, cout: int, ksize: int) -> int:
    return int(lib.st_conv_transposed_workspace_bytes(in_plan.handle, cout, ksize))


def st_conv_transposed_sharded(in_plan: Plan, in_bufs, weight, bias, ksize: int, stride: int, out_plan: Plan,
                               out_bufs, workspace, stream=None) -> None:
    """weight: raw [Cin][Cout][k..] (Cin = in_plan.channels) in the input plan's dtype."""
    ins = _ptr_array(in_bufs, "st_conv_transposed_sharded input", _shard_bytes(in_plan))
    outs = _ptr_array(out_bufs, "st_conv_transposed_sharded output", _shard_bytes(out_plan))
    taps = ksize ** in_plan.ndim
    w = _dev_ptr(weight, "weight", ESIZE[in_plan.dtype] * taps * in_plan.channels * out_plan.channels)
    b = _dev_ptr(bias, "bias", 4 * out_plan.channels)
    ws, nb = _ws(workspace)
    _check(lib.st_conv_transposed_sharded(in_plan.handle, ins, ctypes.c_void_p(w), ctypes.c_void_p(b), ksize,
                                          stride, out_plan.handle, outs, ctypes.c_void_p(ws), nb, _stream(stream)),
           "st_conv_transposed_sharded")


def st_conv_wgrad_workspace_bytes(x_plan: Plan, cout: int, ksize: int) -> int:
    return int(lib.st_conv_wgrad_workspace_bytes(x_plan.handle, cout, ksize))


def st_conv_wgrad(x_plan: Plan, x_bufs, dy_plan: Plan, dy_bufs, ksize: int, dweight, workspace,
                  stream=None) -> None:
    xs = _ptr_array(x_bufs, "st_conv_wgrad x", _shard_bytes(x_plan))
    dys = _ptr_array(dy_bufs, "st_conv_wgrad dy", _shard_bytes(dy_plan))
    elems = dy_plan.channels * x_plan.channels * ksize ** x_plan.ndim
    dw = _dev_ptr(dweight, "dweight", 4 * elems)
    ws, nb = _ws(workspace)
    _check(lib.st_conv_wgrad(x_plan.handle, xs, dy_plan.handle, dys, ksize, ctypes.c_void_p(dw),
                             ctypes.c_void_p(ws), nb, _stream(stream)), "st_conv_wgrad")


def st_groupnorm_workspace_bytes(y_plan: Plan, groups: int) -> int:
    return int(lib.st_groupnorm_workspace_bytes(y_plan.handle, groups))


def st_groupnorm_workspace_layout(y_plan: Plan, groups: int) -> dict:
    l = _GnLayout()
    _check(lib.st_groupnorm_workspace_layout(y_plan.handle, groups, ctypes.byref(l)),
           "st_groupnorm_workspace_layout")
    return {f: getattr(l, f) for f, _ in _GnLayout._fields_}


def st_groupnorm_sharded(y_plan: Plan, y_bufs, ymax, groups: int, eps: float, gamma, beta,
                         z_bufs, workspace, stream=None) -> None:
    sizes = _shard_bytes(y_plan)
    ys = _ptr_array(y_bufs, "st_groupnorm_sharded y", sizes)
    zs = _ptr_array(z_bufs, "st_groupnorm_sharded z", sizes)
    ym = _dev_ptr(ymax, "ymax", 4 * y_plan.batch * groups) if ymax is not None else 0
    g = _dev_ptr(gamma, "gamma", 4 * y_plan.channels)
    b = _dev_ptr(beta, "beta", 4 * y_plan.channels)
    ws = _dev_ptr(workspace, "workspace")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.st_groupnorm_sharded(y_plan.handle, ys, ctypes.c_void_p(ym), groups, float(eps),
                                    ctypes.c_void_p(g), ctypes.c_void_p(b), zs, ctypes.c_void_p(ws),
                                    ws_bytes, _stream(stream)), "st_groupnorm_sharded")


def st_groupnorm_sharded_noalloc(y_plan: Plan, y_bufs, ymax, groups: int, eps: float, gamma, beta,
                                 z_bufs, stream=None) -> None:
    """st_groupnorm_sharded with the library's static scratch as workspace
    (no device allocation; calls that overlap on one GPU race)."""
    sizes = _shard_bytes(y_plan)
    ys = _ptr_array(y_bufs, "st_groupnorm_sharded_noalloc y", sizes)
    zs = _ptr_array(z_bufs, "st_groupnorm_sharded_noalloc z", sizes)
    ym = _dev_ptr(ymax, "ymax", 4 * y_plan.batch * groups) if ymax is not None else 0
    g = _dev_ptr(gamma, "gamma", 4 * y_plan.channels)
    b = _dev_ptr(beta, "beta", 4 * y_plan.channels)
    _check(lib.st_groupnorm_sharded_noalloc(y_plan.handle, ys, ctypes.c_void_p(ym), groups, float(eps),
                                            ctypes.c_void_p(g), ctypes.c_void_p(b), zs, _stream(stream)),
           "st_groupnorm_sharded_noalloc")


def _ws(workspace):
    ws = _dev_ptr(workspace, "workspace")
    return ws, (workspace.nbytes if workspace is not None else 0)


def st_groupnorm_partials(y_plan: Plan, y_bufs, ymax, groups: int, workspace, stream=None) -> None:
    ys = _ptr_array(y_bufs, "st_groupnorm_partials y", _shard_bytes(y_plan))
    ym = _dev_ptr(ymax, "ymax", 4 * y_plan.batch * groups) if ymax is not None else 0
    ws, nb = _ws(workspace)
    _check(lib.st_groupnorm_partials(y_plan.handle, ys, ctypes.c_void_p(ym), groups, ctypes.c_void_p(ws), nb,
                                     _stream(stream)), "st_groupnorm_partials")


def st_groupnorm_combine(y_plan: Plan, groups: int, eps: float, gamma, beta, workspace, stream=None) -> None:
    g = _dev_ptr(gamma, "gamma", 4 * y_plan.channels)
    b = _dev_ptr(beta, "beta", 4 * y_plan.channels)
    ws, nb = _ws(workspace)
    _check(lib.st_groupnorm_combine(y_plan.handle, groups, float(eps), ctypes.c_void_p(g), ctypes.c_void_p(b),
                                    ctypes.c_void_p(ws), nb, _stream(stream)), "st_groupnorm_combine")


def st_groupnorm_apply(y_plan: Plan, y_bufs, groups: int, z_bufs, workspace, stream=None) -> None:
    sizes = _shard_bytes(y_plan)
    ys = _ptr_array(y_bufs, "st_groupnorm_apply y", sizes)
    zs = _ptr_array(z_bufs, "st_groupnorm_apply z", sizes)
    ws, nb = _ws(workspace)
    _check(lib.st_groupnorm_apply(y_plan.handle, ys, groups, zs, ctypes.c_void_p(ws), nb, _stream(stream)),
           "st_groupnorm_apply")


def st_groupnorm_combine_apply(y_plan: Plan, y_bufs, groups: int, eps: float, gamma, beta, z_bufs, workspace,
                               stream=None) -> None:
    sizes = _shard_bytes(y_plan)
    ys = _ptr_array(y_bufs, "st_groupnorm_combine_apply y", sizes)
    zs = _ptr_array(z_bufs, "st_groupnorm_combine_apply z", sizes)
    g = _dev_ptr(gamma, "gamma", 4 * y_plan.channels)
    b = _dev_ptr(beta, "beta", 4 * y_plan.channels)
    ws, nb = _ws(workspace)
    _check(lib.st_groupnorm_combine_apply(y_plan.handle, ys, groups, float(eps), ctypes.c_void_p(g),
                                          ctypes.c_void_p(b), zs, ctypes.c_void_p(ws), nb, _stream(stream)),
           "st_groupnorm_combine_apply")


def st_groupnorm_backward_workspace_bytes(y_plan: Plan, groups: int) -> int:
    return int(lib.st_groupnorm_backward_workspace_bytes(y_plan.handle, groups))


def st_groupnorm_backward(y_plan: Plan, y_bufs, dz_bufs, ymax, dzmax, groups: int, gamma, fwd_workspace,
                          dy_bufs, dgamma, dbeta, workspace, stream=None, dy_plan: Optional[Plan] = None) -> None:
    """dy_plan None: dy in y's fp32 layout; else dy written into dy_plan's
    (padded, fp32 or bf16) shard interiors."""
    sizes = _shard_bytes(y_plan)
    ys = _ptr_array(y_bufs, "st_groupnorm_backward y", sizes)
    dzs = _ptr_array(dz_bufs, "st_groupnorm_backward dz", sizes)
    dys = _ptr_array(dy_bufs, "st_groupnorm_backward dy", sizes if dy_plan is None else _shard_bytes(dy_plan))
    ng = 4 * y_plan.batch * groups
    ym = _dev_ptr(ymax, "ymax", ng) if ymax is not None else 0
    dm = _dev_ptr(dzmax, "dzmax", ng) if dzmax is not None else 0
    g = _dev_ptr(gamma, "gamma", 4 * y_plan.channels)
    dg = _dev_ptr(dgamma, "dgamma", 4 * y_plan.channels)
    db = _dev_ptr(dbeta, "dbeta", 4 * y_plan.channels)
    fws, fnb = _ws(fwd_workspace)
    ws, nb = _ws(workspace)
    _check(lib.st_groupnorm_backward(y_plan.handle, ys, dzs, ctypes.c_void_p(ym), ctypes.c_void_p(dm), groups,
                                     ctypes.c_void_p(g), ctypes.c_void_p(fws), fnb,
                                     dy_plan.handle if dy_plan is not None else None, dys, ctypes.c_void_p(dg),
                                     ctypes.c_void_p(db), ctypes.c_void_p(ws), nb, _stream(stream)),
           "st_groupnorm_backward")


__all__ = [
    "lib", "LIB_PATH", "ShardConvError", "Plan", "ST_F32", "ST_BF16", "st_version",
    "st_plan_shards", "st_halo_pack", "st_halo_unpack", "st_halo_exchange", "st_conv_weight_bytes", "st_conv_dgrad_weights",
    "st_conv_pack_weights", "st_conv_workspace_bytes", "st_conv_sharded", "st_conv_sharded_packed",
    "st_groupnorm_workspace_bytes", "st_conv_strided_workspace_bytes", "st_conv_transposed_workspace_bytes",
    "st_groupnorm_workspace_layout", "st_groupnorm_sharded", "st_groupnorm_sharded_noalloc", "st_groupnorm_partials",
    "st_groupnorm_combine", "st_groupnorm_apply", "st_groupnorm_backward_workspace_bytes",
    "st_groupnorm_backward", "st_conv_wgrad_workspace_bytes", "st_conv_wgrad", "st_plan_pooled",
    "st_pool_sharded", "st_plan_strided", "st_conv_strided_sharded", "st_plan_transposed",
    "st_conv_transposed_sharded", "st_layernorm_sharded", "st_layernorm_backward",
    "st_layernorm_backward_workspace_bytes", "st_plan_positions", "st_rope_axes", "Sequences", "st_plan_sequences",
    "st_attention_workspace_bytes", "st_attention_packed", "st_attention_packed_backward", "st_groupnorm_combine_apply",
    "ST_MX8", "Mx8", "mx8_empty", "st_mx8_store", "st_mx8_load", "st_rmsnorm", "st_rmsnorm_backward_workspace_bytes",
    "st_rmsnorm_backward", "st_linear_workspace_bytes", "st_linear", "st_linear_backward",
]


# ------------------------------------------------------------ token operators

def _bits(*names):
    return frozenset(getattr(_torch(), n) for n in names)


# What the token operators take as fp32, bf16 and int32: the type itself, or its
# bits (integers of its width, bytes).  Any other type is refused, not read as bits.
_FP32, _INT32 = _bits("float32", "int32", "uint8"), _bits("int32", "uint8")
_TYPES = {ST_F32: _FP32, ST_BF16: _bits("bfloat16", "int16", "uint8")}


def _typed(t, what: str, types, min_bytes: int = 0) -> int:
    """_dev_ptr of a tensor of one of these types, or of None."""
    if t is not None and getattr(t, "is_cuda", False) and t.dtype in types and t.is_contiguous() and t.nbytes >= min_bytes:
        return t.data_ptr()
    ptr = _dev_ptr(t, what, min_bytes)       # its message, or the dtype's
    if t is not None:
        raise ShardConvError(1, f"{what}: unexpected dtype {t.dtype}")
    return ptr


def _typed_array(tensors, what: str, types, sizes: List[int]):
    if len(tensors) != len(sizes):
        return _ptr_array(tensors, what, sizes)   # its message
    arr = (ctypes.c_void_p * max(1, len(sizes)))()
    for i, t in enumerate(tensors):
        if t is not None and getattr(t, "is_cuda", False) and t.dtype in types and t.is_contiguous() and t.nbytes >= sizes[i]:
            arr[i] = t.data_ptr()
        else:
            arr[i] = _typed(t, f"{what}[{i}]", types, sizes[i])   # its message
    return arr


def _plan_array(plan: Plan, tensors, what: str):
    """Shard buffers of a plan, in its dtype."""
    return _typed_array(tensors, what, _TYPES[plan.dtype], _shard_bytes(plan))


def _cells(plan: Plan) -> List[int]:
    """Interior cells of every shard."""
    if plan._cells is None:
        out = []
        for i in range(plan.num_shards):
            n = plan.batch
            for e in plan.shard_info(i)["extent"]:
                n *= e
            out.append(n)
        plan._cells = out
    return plan._cells


def _stats_bytes(plan: Plan) -> int:
    """Of the layer norm's statistics: 2 floats per cell."""
    if plan._stats is None:
        plan._stats = 8 * sum(_cells(plan))
    return plan._stats


def st_layernorm_sharded(x_plan: Plan, x_bufs, gamma, beta, eps: float, y_plan: Plan, y_bufs, stats=None,
                         stream=None) -> None:
    """Layer norm over the channels of every cell; stats: 2 floats per cell
    (mean, 1 / sqrt(var + eps)), shard by shard, or None."""
    xs = _plan_array(x_plan, x_bufs, "st_layernorm_sharded x")
    ys = _plan_array(y_plan, y_bufs, "st_layernorm_sharded y")
    g = _typed(gamma, "gamma", _FP32, 4 * x_plan.channels)
    b = _typed(beta, "beta", _FP32, 4 * x_plan.channels)
    st = _typed(stats, "stats", _FP32, _stats_bytes(x_plan))
    _check(lib.st_layernorm_sharded(x_plan.handle, xs, g, b, float(eps), y_plan.handle, ys, st, _stream(stream)),
           "st_layernorm_sharded")


def st_layernorm_backward_workspace_bytes(x_plan: Plan) -> int:
    return int(lib.st_layernorm_backward_workspace_bytes(x_plan.handle))


def st_layernorm_backward(x_plan: Plan, x_bufs, dy_plan: Plan, dy_bufs, gamma, stats, dx_plan: Plan, dx_bufs, dgamma,
                          dbeta, workspace, stream=None) -> None:
    """stats: as st_layernorm_sharded wrote them; dgamma, dbeta: C floats or None."""
    xs = _plan_array(x_plan, x_bufs, "st_layernorm_backward x")
    dys = _plan_array(dy_plan, dy_bufs, "st_layernorm_backward dy")
    dxs = _plan_array(dx_plan, dx_bufs, "st_layernorm_backward dx")
    c = 4 * x_plan.channels
    ws, nb = _ws(workspace)
    _check(lib.st_layernorm_backward(x_plan.handle, xs, dy_plan.handle, dys, _typed(gamma, "gamma", _FP32, c),
                                     _typed(stats, "stats", _FP32, _stats_bytes(x_plan)), dx_plan.handle, dxs,
                                     _typed(dgamma, "dgamma", _FP32, c), _typed(dbeta, "dbeta", _FP32, c), ws, nb,
                                     _stream(stream)), "st_layernorm_backward")


def st_plan_positions(plan: Plan, pos_bufs, stream=None) -> None:
    """Global int32 grid positions [N][extent...][ndim] of every shard's cells."""
    ps = _typed_array(pos_bufs, "st_plan_positions", _INT32, [4 * plan.ndim * n for n in _cells(plan)])
    _check(lib.st_plan_positions(plan.handle, ps, _stream(stream)), "st_plan_positions")


_TENSOR_DTYPES = {_torch().float32: ST_F32, _torch().bfloat16: ST_BF16, _torch().int16: ST_BF16}


def _float_dtype(t, what: str) -> int:
    """ST_F32 or ST_BF16 of a tensor (bf16 also as int16 bit patterns)."""
    dt = _TENSOR_DTYPES.get(t.dtype)
    if dt is None:
        raise ShardConvError(1, f"{what}: expected float32 or bfloat16, got {t.dtype}")
    return dt


def _rows3(t, what: str):
    """Checks of a [tokens, heads, head_dim] tensor with contiguous channels."""
    if not getattr(t, "is_cuda", False):
        raise ShardConvError(1, f"{what}: expected a GPU tensor (no CPU fallback exists)")
    if t.dim() != 3:
        raise ShardConvError(2, f"{what}: expected [tokens, heads, head_dim], got {tuple(t.shape)}")
    if t.numel() and t.shape[2] > 1 and t.stride(2) != 1:
        raise ShardConvError(2, f"{what}: channels must be contiguous")


_PAIRS = {"halves": 0, "adjacent": 1}


def st_rope_axes(x, positions, axis_dims: Sequence[int], out, rotated_heads: Optional[int] = None,
                 base: float = 10000.0, pairs: str = "halves", inverse: bool = False, stream=None) -> None:
    """Rotary positions with one section of channels per axis.

    x, out: [tokens, heads, head_dim], float32 or bfloat16 each, any token and
    head strides; out may be x.  positions: int32 [tokens, axes] (or flat).
    rotated_heads: heads that turn (default all), the others are copied.
    """
    _rows3(x, "st_rope_axes x")
    _rows3(out, "st_rope_axes out")
    tokens, heads, dim = x.shape
    if tuple(out.shape) != (tokens, heads, dim):
        raise ShardConvError(2, f"st_rope_axes: out is {tuple(out.shape)}, x is {tuple(x.shape)}")
    if pairs not in _PAIRS:
        raise ShardConvError(1, f"st_rope_axes: unknown pairing {pairs!r}")
    n = len(axis_dims)
    if positions.dtype != _torch().int32:
        raise ShardConvError(1, "st_rope_axes: positions must be int32")
    if n and positions.dim() > 1 and positions.shape[-1] != n:
        raise ShardConvError(2, f"st_rope_axes: positions are {tuple(positions.shape)}, axis_dims names {n} axes")
    pos = _dev_ptr(positions, "positions", 4 * tokens * n)
    dims = (ctypes.c_int32 * max(1, n))(*axis_dims)
    _check(lib.st_rope_axes(x.data_ptr(), _float_dtype(x, "st_rope_axes x"), x.stride(0), x.stride(1), tokens, heads,
                            heads if rotated_heads is None else rotated_heads, dim, pos, n, dims, float(base),
                            _PAIRS[pairs], int(bool(inverse)), out.data_ptr(), _float_dtype(out, "st_rope_axes out"),
                            out.stride(0), out.stride(1), _stream(stream)), "st_rope_axes")


class Sequences:
    """Owns an st_seqs*: the work plan of attention over packed sequences."""

    def __init__(self, handle: int, q_lens, k_lens, heads: int, kv_heads: int, head_dim: int, dtype: int, causal: bool):
        self._h = ctypes.c_void_p(handle)
        self.total_q, self.total_k = sum(q_lens), sum(k_lens)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.dtype, self.causal = dtype, causal
        self.q_shape, self.k_shape = (self.total_q, heads, head_dim), (self.total_k, kv_heads, head_dim)

    @property
    def handle(self) -> ctypes.c_void_p:
        if not self._h:
            raise ShardConvError(1, "sequences already destroyed")
        return self._h

    def destroy(self) -> None:
        if self._h:
            _check(lib.st_seqs_destroy(self._h), "st_seqs_destroy")
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def upload(self, stream=None) -> None:
        """Put the work tables on the current device now (needed before a graph
        capture that contains the first attention call)."""
        _check(lib.st_seqs_upload(self.handle, _stream(stream)), "st_seqs_upload")


def st_plan_sequences(q_lens: Sequence[int], k_lens: Optional[Sequence[int]], heads: int, kv_heads: int, head_dim: int,
                      dtype, causal: bool) -> Sequences:
    """Plan of attention over packed sequences of q_lens queries and k_lens
    (None: q_lens) keys; dtype 'f32'/'bf16' or 0/1."""
    q = list(q_lens)
    k = q if k_lens is None else list(k_lens)
    if len(q) != len(k):
        raise ShardConvError(2, f"st_plan_sequences: {len(q)} query lengths and {len(k)} key lengths")
    if any(n < 0 or n >= 1 << 31 for n in q + k):
        raise ShardConvError(1, "st_plan_sequences: a length is negative or past 2^31")
    dt = DTYPES.get(dtype, dtype)
    qa = (ctypes.c_int32 * max(1, len(q)))(*q)
    ka = (ctypes.c_int32 * max(1, len(k)))(*k)
    out = ctypes.c_void_p()
    _check(lib.st_plan_sequences(len(q), qa, ka, heads, kv_heads, head_dim, dt, int(bool(causal)), ctypes.byref(out)),
           "st_plan_sequences")
    return Sequences(out.value, q, k, heads, kv_heads, head_dim, dt, bool(causal))


def st_attention_workspace_bytes(seqs: Sequences, backward: bool = False) -> int:
    return int(lib.st_attention_workspace_bytes(seqs.handle, int(bool(backward))))


def _tokens(t, what: str, seqs: Sequences, keys: bool) -> _Tokens:
    want = seqs.k_shape if keys else seqs.q_shape
    if t.shape != want or not t.is_cuda:
        _rows3(t, what)
        raise ShardConvError(2, f"{what}: expected {want}, got {tuple(t.shape)}")
    if _TENSOR_DTYPES.get(t.dtype) != seqs.dtype:
        raise ShardConvError(1, f"{what}: dtype {t.dtype} is not the plan's")
    st, sh, sc = t.stride()
    if sc != 1:
        _rows3(t, what)
    return _Tokens(t.data_ptr(), st, sh)


def st_attention_packed(seqs: Sequences, q, k, v, scale: float, out, lse=None, workspace=None, stream=None) -> None:
    """q, out: [total queries, heads, head_dim]; k, v: [total keys, kv_heads,
    head_dim]; any strides that are multiples of 16 bytes; lse: float32
    [total queries, heads] or None."""
    what = "st_attention_packed"
    l = _typed(lse, "st_attention_packed lse", _FP32, 4 * seqs.total_q * seqs.heads)
    ws, nb = _ws(workspace)
    _check(lib.st_attention_packed(seqs.handle, _tokens(q, "st_attention_packed q", seqs, False),
                                   _tokens(k, "st_attention_packed k", seqs, True),
                                   _tokens(v, "st_attention_packed v", seqs, True), scale,
                                   _tokens(out, "st_attention_packed out", seqs, False), l, ws, nb, _stream(stream)), what)


def st_attention_packed_backward(seqs: Sequences, q, k, v, out, lse, dout, scale: float, dq, dk, dv, workspace,
                                 stream=None) -> None:
    """dq, dk, dv of st_attention_packed; out and lse as it wrote them."""
    def view(t, n, keys):
        return _tokens(t, n, seqs, keys)

    what = "st_attention_packed_backward"
    l = _typed(lse, "st_attention_packed_backward lse", _FP32, 4 * seqs.total_q * seqs.heads)
    ws, nb = _ws(workspace)
    _check(lib.st_attention_packed_backward(
        seqs.handle, view(q, "st_attention_packed_backward q", False), view(k, "st_attention_packed_backward k", True),
        view(v, "st_attention_packed_backward v", True), view(out, "st_attention_packed_backward out", False), l,
        view(dout, "st_attention_packed_backward dout", False), scale, view(dq, "st_attention_packed_backward dq", False),
        view(dk, "st_attention_packed_backward dk", True), view(dv, "st_attention_packed_backward dv", True), ws, nb,
        _stream(stream)), what)


# ------------------------------------------- MLP branch: rows of channels, 8 bits

ST_MX8 = 2
_ROW_TYPES = {"f32": ST_F32, "bf16": ST_BF16, "mx8": ST_MX8}
_ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}


# An operand's st_rows as bytes: data, scales, stride, scale stride, type.  (Packed
# by struct and passed as a pointer to the bytes: a third of the time of a ctypes
# structure, of which a call takes up to six.)
_PACK = struct.Struct("=QQqqi4x").pack


class Mx8:
    """Rows of `channels` values in the 8-bit form: codes (bytes, [rows, at least
    channels]) and scales (bytes, [rows, at least a byte per 32 channels]).  The
    codes' row stride is a multiple of 16, the scales' of 4."""

    __slots__ = ("codes", "scales", "channels", "rows")

    def __init__(self, codes, scales, channels: int):
        self.codes, self.scales, self.channels = codes, scales, int(channels)
        blocks = -(-self.channels // 32)
        for t, what, least in ((codes, "codes", self.channels), (scales, "scales", blocks)):
            if t.dim() != 2 or t.element_size() != 1 or t.shape[1] < least or (t.shape[1] > 1 and t.numel() and t.stride(1) != 1):
                raise ShardConvError(2, f"Mx8: {what} are not bytes [rows, >= {least}] with contiguous rows")
        if codes.shape[0] != scales.shape[0]:
            raise ShardConvError(2, f"Mx8: {codes.shape[0]} rows of codes and {scales.shape[0]} of scales")
        self.rows = int(codes.shape[0])


def mx8_empty(rows: int, channels: int, device: str = "cuda") -> Mx8:
    """An unwritten Mx8 whose strides every operator takes."""
    torch = _torch()
    return Mx8(torch.empty(rows, -(-channels // 16) * 16, dtype=torch.uint8, device=device),
               torch.empty(rows, -(-channels // 128) * 4, dtype=torch.uint8, device=device), channels)


_ROW_DTYPES = {_torch().float32: ST_F32, _torch().bfloat16: ST_BF16}


def _device() -> int:
    return _torch()._C._cuda_getDevice()


def _here(t, what: str, device: int) -> None:
    """The kernels run on the current device: operands of another one are refused."""
    if not getattr(t, "is_cuda", False):
        raise ShardConvError(1, f"{what}: expected a GPU tensor (no CPU fallback exists)")
    if t.get_device() != device:
        raise ShardConvError(1, f"{what}: on device {t.get_device()}, which is not the current one")


def _rows(t, call: str, name: str, rows: int, channels: int, device: int):
    """st_rows of a [rows, channels] tensor or an Mx8; None stays None."""
    if t is None:
        return None
    if t.__class__ is Mx8:
        if t.rows != rows or t.channels != channels:
            raise ShardConvError(2, f"{call} {name}: expected {(rows, channels)}, got {(t.rows, t.channels)}")
        c, s = t.codes, t.scales
        if not (c.is_cuda and s.is_cuda and c.get_device() == device and s.get_device() == device):
            _here(c, f"{call} {name}", device)
            _here(s, f"{call} {name}", device)
        return _PACK(c.data_ptr(), s.data_ptr(), c.stride(0), s.stride(0), ST_MX8)
    if not (getattr(t, "is_cuda", False) and t.get_device() == device):
        _here(t, f"{call} {name}", device)
    if t.shape != (rows, channels):
        raise ShardConvError(2, f"{call} {name}: expected {(rows, channels)}, got {tuple(t.shape)}")
    dt = _ROW_DTYPES.get(t.dtype)
    if dt is None:
        raise ShardConvError(1, f"{call} {name}: expected float32, bfloat16 or Mx8, got {t.dtype}")
    st, sc = t.stride()
    if sc != 1 and channels > 1 and rows:
        raise ShardConvError(2, f"{call} {name}: channels must be contiguous")
    return _PACK(t.data_ptr(), 0, st, 0, dt)


def _shape(t, what: str):
    if isinstance(t, Mx8):
        return t.rows, t.channels
    if t is None or getattr(t, "dim", lambda: 0)() != 2:
        raise ShardConvError(2, f"{what}: expected [rows, channels]")
    return t.shape[0], t.shape[1]


def _act(act: str, what: str) -> int:
    if act not in _ACTS:
        raise ShardConvError(1, f"{what}: unknown activation {act!r}")
    return _ACTS[act]


def _floats(t, what: str, min_bytes: int, device: int):
    """Floats of the current device, or None."""
    if t is not None and not (getattr(t, "is_cuda", False) and t.get_device() == device):
        _here(t, what, device)
    return _typed(t, what, _FP32, min_bytes)


def _ws_here(workspace, device: int):
    if workspace is not None:
        _here(workspace, "workspace", device)
    return _ws(workspace)


def st_mx8_store(x, out: Mx8, stream=None) -> None:
    """x: [rows, channels], float32 or bfloat16, into the 8-bit form."""
    dev = _device()
    n, c = _shape(x, "st_mx8_store x")
    _check(lib.st_mx8_store(n, c, _rows(x, "st_mx8_store", "x", n, c, dev), _rows(out, "st_mx8_store", "out", n, c, dev), _stream(stream)),
           "st_mx8_store")


def st_mx8_load(x: Mx8, out, act: str = "none", stream=None) -> None:
    """act(x) into [rows, channels], float32 or bfloat16."""
    dev = _device()
    n, c = _shape(x, "st_mx8_load x")
    _check(lib.st_mx8_load(n, c, _rows(x, "st_mx8_load", "x", n, c, dev), _act(act, "st_mx8_load"),
                           _rows(out, "st_mx8_load", "out", n, c, dev), _stream(stream)), "st_mx8_load")


def st_rmsnorm(x, residual, gamma, eps: float, total=None, y=None, y8: Optional[Mx8] = None, rstd=None, stream=None) -> None:
    """s = x + residual (None: x) into total, s * rstd * gamma into y and y8 (the
    8-bit form); rows of channels in float32 or bfloat16; gamma: C floats or
    None; rstd: a float per row or None."""
    what = "st_rmsnorm"
    dev = _device()
    n, c = _shape(x, "st_rmsnorm x")
    _check(lib.st_rmsnorm(n, c, _rows(x, "st_rmsnorm", "x", n, c, dev), _rows(residual, "st_rmsnorm", "residual", n, c, dev),
                          _floats(gamma, "gamma", 4 * c, dev), float(eps), _rows(total, "st_rmsnorm", "total", n, c, dev),
                          _rows(y, "st_rmsnorm", "y", n, c, dev), _rows(y8, "st_rmsnorm", "y8", n, c, dev),
                          _floats(rstd, "rstd", 4 * n, dev), _stream(stream)), what)


def st_rmsnorm_backward_workspace_bytes(rows: int, channels: int) -> int:
    return int(lib.st_rmsnorm_backward_workspace_bytes(rows, channels))


def st_rmsnorm_backward(s, dy, dtotal, gamma, rstd, dx, dgamma, workspace, stream=None) -> None:
    """s: the forward call's total (a tensor, or the Mx8 it was kept in); dtotal:
    gradient at s from the residual stream, or None; dgamma: C floats or None."""
    what = "st_rmsnorm_backward"
    dev = _device()
    n, c = _shape(s, "st_rmsnorm_backward s")
    ws, nb = _ws_here(workspace, dev)
    _check(lib.st_rmsnorm_backward(n, c, _rows(s, "st_rmsnorm_backward", "s", n, c, dev), _rows(dy, "st_rmsnorm_backward", "dy", n, c, dev),
                                   _rows(dtotal, "st_rmsnorm_backward", "dtotal", n, c, dev), _floats(gamma, "gamma", 4 * c, dev),
                                   _floats(rstd, "rstd", 4 * n, dev), _rows(dx, "st_rmsnorm_backward", "dx", n, c, dev),
                                   _floats(dgamma, "dgamma", 4 * c, dev), ws, nb, _stream(stream)), what)


def st_linear_workspace_bytes(rows: int, channels_in: int, channels_out: int, dtype, backward: bool = False) -> int:
    """dtype: 'f32', 'bf16' or 'mx8' of the products."""
    return int(lib.st_linear_workspace_bytes(rows, channels_in, channels_out, _ROW_TYPES.get(dtype, dtype), int(bool(backward))))


def st_linear(x, w, bias, y, act: str = "none", residual=None, pre=None, workspace=None, stream=None) -> None:
    """y = act(x w^T + bias) + residual.  x: [rows, in], w: [out, in], both of one
    type (float32, bfloat16, Mx8); y, pre: [rows, out] in any of the three, pre
    receives x w^T + bias; bias: float32 [out] or None."""
    what = "st_linear"
    dev = _device()
    n, k = _shape(x, "st_linear x")
    m = _shape(w, "st_linear w")[0]
    ws, nb = _ws_here(workspace, dev)
    _check(lib.st_linear(n, k, m, _rows(x, "st_linear", "x", n, k, dev), _rows(w, "st_linear", "w", m, k, dev),
                         _floats(bias, "bias", 4 * m, dev), _act(act, what), _rows(residual, "st_linear", "residual", n, m, dev),
                         _rows(y, "st_linear", "y", n, m, dev), _rows(pre, "st_linear", "pre", n, m, dev), ws, nb, _stream(stream)), what)


def st_linear_backward(x, w, dy, dx, dw, dbias, act: str = "none", pre=None, workspace=None, stream=None) -> None:
    """Gradients of st_linear at x, w and bias (each None: not computed).  x: w's
    type, or the Mx8 it was kept in; pre: as st_linear wrote it."""
    what = "st_linear_backward"
    dev = _device()
    n, k = _shape(x, "st_linear_backward x")
    m = _shape(w, "st_linear_backward w")[0]
    ws, nb = _ws_here(workspace, dev)
    _check(lib.st_linear_backward(n, k, m, _rows(x, "st_linear_backward", "x", n, k, dev), _rows(w, "st_linear_backward", "w", m, k, dev),
                                  _act(act, what), _rows(pre, "st_linear_backward", "pre", n, m, dev),
                                  _rows(dy, "st_linear_backward", "dy", n, m, dev), _rows(dx, "st_linear_backward", "dx", n, k, dev),
                                  _rows(dw, "st_linear_backward", "dw", m, k, dev), _floats(dbias, "dbias", 4 * m, dev), ws, nb,
                                  _stream(stream)), what)

"""Attention over packed sequences against the fp64 definition: forward and
gradients, lengths from zero and one up to several tiles, grouped heads,
strides, masks that leave rows empty, NaN and infinities where a row does not
look, splits over the keys, streams and graphs.

Tolerances, element by element, from the roundings of each type (u = 2^-8 of a
bf16, 2^-24 of an fp32 value):
  bf16  the output's rounding and that of the weights (p in out and dv, ds in
        dq and dk) are u of what they multiply each, and D = dout * out comes
        from the rounded output: 2 u = 2^-7 of the sum of absolute values
        (tokens.attention_bounds), plus 10% for the second order and fp32 parts
  fp32  a score is a sum of head_dim products: its error grows as a few u
        sqrt(head_dim) of scale * sum |q||k|; the sums over keys add a few u:
        2^-20 (1 + largest scale * sum |q||k|) of the sum of absolute values
  lse   the score's error alone, absolute: 2^-20 (1 + largest score)
"""
import math

import numpy as np
import pytest
import torch

from helpers import say
from oracle import tokens

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(q_lens, k_lens, heads, kv_heads, dim, dtype, seed=0):
    rng = np.random.default_rng(seed)
    t = TORCH[dtype]
    q, dout = (torch.from_numpy(rng.normal(size=(sum(q_lens), heads, dim))).to(t) for _ in range(2))
    k, v = (torch.from_numpy(rng.normal(size=(sum(k_lens), kv_heads, dim))).to(t) for _ in range(2))
    return q, k, v, dout


def f64(t):
    return t.double().cpu().numpy()


def run(lib, q, k, v, dout, q_lens, k_lens, dtype, causal, scale, train=True, lse=True):
    seqs = lib.st_plan_sequences(q_lens, k_lens, q.shape[1], k.shape[1], q.shape[2], dtype, causal)
    # no byte past what is asked for: a guard behind it must stay
    need = lib.st_attention_workspace_bytes(seqs, backward=train)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    l = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
    lib.st_attention_packed(seqs, q, k, v, scale, out, l, ws[:need] if need else None)
    r = {"out": out, "lse": l}
    if train:
        r.update(dq=torch.full_like(q, 7.0), dk=torch.full_like(k, 7.0), dv=torch.full_like(v, 7.0))
        lib.st_attention_packed_backward(seqs, q, k, v, out, l, dout, scale, r["dq"], r["dk"], r["dv"],
                                         ws[:need] if need else None)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all()), "written past the workspace"
    return r


def check(r, q, k, v, dout, q_lens, k_lens, dtype, causal, scale):
    a = [f64(t) for t in (q, k, v)]
    want = tokens.attention(*a, q_lens, k_lens, scale, causal, f64(dout))
    b = tokens.attention_bounds(*a, q_lens, k_lens, scale, causal, f64(dout))
    eps = 1.1 * 2.0 ** -7 if dtype == "bf16" else 2.0 ** -20 * (1 + b["score"])
    for name in ("out", "dq", "dk", "dv"):
        if r.get(name) is None:
            continue
        off = np.abs(f64(r[name]) - want[name])
        assert np.all(off <= eps * b[name] + 1e-30), f"{name}: {np.max(off - eps * b[name])} over, {np.max(off)} off"
    if r["lse"] is not None:
        got = f64(r["lse"])
        empty = np.isneginf(want["lse"])
        assert np.array_equal(np.isneginf(got), empty)
        assert np.all(np.abs(got[~empty] - want["lse"][~empty]) <= 2.0 ** -20 * (1 + b["score"]))


# lengths around the 32-row blocks and the 64-key and 128-row tiles
RAGGED = ([1, 0, 33, 64, 129, 200, 31], None)
OTHER = ([1, 5, 0, 70, 130, 3, 65], [200, 0, 9, 33, 131, 1, 64])
CASES = [
    (RAGGED, 2, 2, 64, False), (RAGGED, 2, 2, 64, True), (OTHER, 4, 2, 64, False), (OTHER, 4, 2, 64, True),
    (RAGGED, 6, 2, 128, True), (OTHER, 3, 1, 128, False), (OTHER, 8, 1, 32, True), (RAGGED, 5, 5, 40, False),
    (OTHER, 7, 1, 96, True), (RAGGED, 2, 1, 8, True), (OTHER, 2, 2, 72, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,kv_heads,dim,causal", CASES)
def test_forward_and_gradients(gpu_lib, lens, heads, kv_heads, dim, causal, dtype):
    q_lens, k_lens = lens[0], lens[1] or lens[0]
    say(f"attention {dtype} {heads}/{kv_heads} x {dim} causal={causal} q={q_lens} k={k_lens}")
    host = inputs(q_lens, k_lens, heads, kv_heads, dim, dtype)
    dev = [t.cuda() for t in host]
    scale = 1 / math.sqrt(dim)
    r = run(gpu_lib, *dev, q_lens, k_lens, dtype, causal, scale)
    check(r, *host, q_lens, k_lens, dtype, causal, scale)
    # the same bits again, and without the optional lse
    again = run(gpu_lib, *dev, q_lens, k_lens, dtype, causal, scale)
    assert all(torch.equal(r[n].view(torch.int16), again[n].view(torch.int16)) for n in r)
    bare = run(gpu_lib, *dev, q_lens, k_lens, dtype, causal, scale, train=False, lse=False)
    assert torch.equal(bare["out"].view(torch.int16), r["out"].view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,k_lens,heads,kv_heads,dim,causal", [
    ([1, 1, 1], [5000, 700, 1], 8, 2, 64, False),         # single tokens, keys split and joined
    ([1, 3], [3001, 2000], 4, 1, 128, True),
    ([700], [40], 2, 2, 64, False),                       # few keys: rows split for dk and dv
    ([1500], [1500], 1, 1, 32, True),                     # one long sequence, one head
])
def test_split_work(gpu_lib, q_lens, k_lens, heads, kv_heads, dim, causal, dtype):
    say(f"split attention {dtype} q={q_lens} k={k_lens}")
    host = inputs(q_lens, k_lens, heads, kv_heads, dim, dtype, seed=1)
    dev = [t.cuda() for t in host]
    scale = 1 / math.sqrt(dim)
    r = run(gpu_lib, *dev, q_lens, k_lens, dtype, causal, scale)
    check(r, *host, q_lens, k_lens, dtype, causal, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_do_not_touch_each_other(gpu_lib, dtype):
    """A sequence's bits are those it has with NaN and infinities next door."""
    q_lens = k_lens = [40, 97, 33]
    say(f"attention next to NaN {dtype}")
    host = inputs(q_lens, k_lens, 4, 2, 64, dtype, seed=2)
    for causal in (False, True):
        clean = run(gpu_lib, *[t.cuda() for t in host], q_lens, k_lens, dtype, causal, 0.2)
        bad = [t.clone() for t in host]
        for i, t in enumerate(bad):
            t[:40] = math.nan if i % 2 else math.inf
            t[137:] = math.nan
        r = run(gpu_lib, *[t.cuda() for t in bad], q_lens, k_lens, dtype, causal, 0.2)
        for n in r:
            assert torch.equal(r[n][40:137], clean[n][40:137]), f"{n} causal={causal}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 2, 2), (128, 4, 2), (40, 3, 1)])
def test_later_keys_do_not_reach_earlier_rows(gpu_lib, dtype, dim, heads, kv_heads):
    """NaN, +inf and -inf in a key or value reach the rows that see them, as the
    definition says, and no row before them."""
    n, at = 150, 77
    say(f"special values under the causal mask {dtype} {dim}")
    host = inputs([n], [n], heads, kv_heads, dim, dtype, seed=3)
    clean = run(gpu_lib, *[t.cuda() for t in host], [n], [n], dtype, True, 0.2, train=False)
    for where in ("k", "v"):
        for value in (math.nan, math.inf, -math.inf):
            bad = [t.clone() for t in host]
            bad["qkv".index(where)][at, 0, 5] = value
            r = run(gpu_lib, *[t.cuda() for t in bad], [n], [n], dtype, True, 0.2, train=False)
            assert torch.equal(r["out"][:at], clean["out"][:at]), (where, value)
            group = heads // kv_heads
            if where == "v":
                got = r["out"][at:, :group, 5].float()
                assert bool((torch.isnan(got) if math.isnan(value) else got == value).all()), value
                got = r["out"][at:].clone()
                got[:, :group, 5] = clean["out"][at:, :group, 5]
                assert torch.equal(got, clean["out"][at:])
            elif math.isnan(value):
                assert bool(torch.isnan(r["out"][at:, :group].float()).all())


def test_large_scores(gpu_lib):
    """Scores of several hundred: no overflow, the running maximum moves."""
    n = 300
    for dtype in ("bf16", "f32"):
        host = inputs([n], [n], 2, 2, 64, dtype, seed=4)
        host[1].mul_(torch.linspace(0.1, 8.0, n, dtype=torch.float64)[:, None, None].to(host[1].dtype))
        r = run(gpu_lib, *[t.cuda() for t in host], [n], [n], dtype, False, 0.5)
        check(r, *host, [n], [n], dtype, False, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,k_lens,heads,kv_heads,dim", [
    ([0, 1, 0, 1, 1], None, 8, 1, 128),
    ([1, 200, 33], [1, 1, 1], 4, 2, 64),
    ([300], [1], 3, 3, 96)])
def test_a_single_key_leaves_no_gradient_of_its_weight(gpu_lib, q_lens, k_lens, heads, kv_heads, dim, dtype):
    # its weight is one whatever q and k are: exact zeros, not the roundings of p dp - D
    k_lens = k_lens or q_lens
    t = [x.cuda() for x in inputs(q_lens, k_lens, heads, kv_heads, dim, dtype, seed=12)]
    r = run(gpu_lib, *t, q_lens, k_lens, dtype, False, dim ** -0.5)
    check(r, *t, q_lens, k_lens, dtype, False, dim ** -0.5)
    assert not r["dq"].any() and not r["dk"].any()


@pytest.mark.parametrize("layout", ["joint", "heads first", "spaced"])
def test_strides(gpu_lib, layout):
    """Views: a joint projection, heads outermost, rows with gaps; values
    between the rows stay as they were."""
    q_lens = k_lens = [50, 81]
    t, heads, kv_heads, dim = 131, 4, 2, 64
    host = inputs(q_lens, k_lens, heads, kv_heads, dim, "bf16", seed=5)
    want = run(gpu_lib, *[x.cuda() for x in host], q_lens, k_lens, "bf16", True, 0.125)

    def buffers():
        if layout == "joint":
            b = torch.full((t, heads + 2 * kv_heads, dim), 3.0, dtype=torch.bfloat16, device="cuda")
            return b, [b[:, :heads], b[:, heads:heads + kv_heads], b[:, heads + kv_heads:]]
        if layout == "heads first":
            b = torch.full((heads + 2 * kv_heads, t, dim), 3.0, dtype=torch.bfloat16, device="cuda")
            return b, [b[:heads].transpose(0, 1), b[heads:heads + kv_heads].transpose(0, 1), b[heads + kv_heads:].transpose(0, 1)]
        b = torch.full((t, heads + 2 * kv_heads, dim + 8), 3.0, dtype=torch.bfloat16, device="cuda")
        c = b[:, :, :dim]
        return b, [c[:, :heads], c[:, heads:heads + kv_heads], c[:, heads + kv_heads:]]

    _, (q, k, v) = buffers()
    for dst, src in ((q, host[0]), (k, host[1]), (v, host[2])):
        dst.copy_(src)
    grads, (dq, dk, dv) = buffers()
    outs, (out, dout, _) = buffers()
    dout = torch.empty_like(out)
    dout.copy_(host[3])
    lse = torch.empty(t, heads, device="cuda")
    seqs = gpu_lib.st_plan_sequences(q_lens, k_lens, heads, kv_heads, dim, "bf16", True)
    ws = torch.empty(max(16, gpu_lib.st_attention_workspace_bytes(seqs, True)), dtype=torch.uint8, device="cuda")
    gpu_lib.st_attention_packed(seqs, q, k, v, 0.125, out, lse, ws)
    gpu_lib.st_attention_packed_backward(seqs, q, k, v, out, lse, dout, 0.125, dq, dk, dv, ws)
    for got, name in ((out, "out"), (lse, "lse"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        assert torch.equal(got, want[name]), name
    if layout == "spaced":
        assert bool((grads[:, :, dim:] == 3.0).all()) and bool((outs[:, :, dim:] == 3.0).all())


def test_gradient_against_differences(gpu_lib):
    """fp32: the directional derivative of sum(out * dout), by central
    differences of the library's own forward pass in steps h: truncation ~ h^2
    and rounding ~ 2^-20 |f| / h; with h = 2^-5 both stay below 1% here."""
    q_lens = k_lens = [60, 37]
    host = inputs(q_lens, k_lens, 2, 1, 32, "f32", seed=6)
    dev = [t.cuda() for t in host]
    r = run(gpu_lib, *dev, q_lens, k_lens, "f32", True, 0.2)
    rng = np.random.default_rng(7)
    h = 2.0 ** -5
    for i, name in enumerate(("dq", "dk", "dv")):
        t = torch.from_numpy(rng.normal(size=tuple(host[i].shape))).cuda()
        f = []
        for sign in (1, -1):
            moved = list(dev)
            moved[i] = (dev[i].double() + sign * h * t).float()
            out = run(gpu_lib, *moved, q_lens, k_lens, "f32", True, 0.2, train=False)["out"]
            f.append(float((out.double() * dev[3].double()).sum()))
        got, want = (f[0] - f[1]) / (2 * h), float((r[name].double() * t).sum())
        size = float(torch.linalg.vector_norm(r[name].double()))
        assert abs(got - want) <= 0.02 * size, (name, got, want)


def test_streams_and_graphs(gpu_lib):
    """On a stream of its own, and captured: every replay gives the eager bits."""
    q_lens, k_lens = [1, 70, 1], [900, 70, 40]
    host = inputs(q_lens, k_lens, 4, 2, 64, "bf16", seed=8)
    q, k, v, dout = [t.cuda() for t in host]
    want = run(gpu_lib, q, k, v, dout, q_lens, k_lens, "bf16", True, 0.125)
    seqs = gpu_lib.st_plan_sequences(q_lens, k_lens, 4, 2, 64, "bf16", True)
    ws = torch.empty(gpu_lib.st_attention_workspace_bytes(seqs, True), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(72, 4, device="cuda")
    grads = [torch.empty_like(t) for t in (q, k, v)]

    def step():
        gpu_lib.st_attention_packed(seqs, q, k, v, 0.125, out, lse, ws)
        gpu_lib.st_attention_packed_backward(seqs, q, k, v, out, lse, dout, 0.125, *grads, ws)

    def same():
        torch.cuda.synchronize()
        for got, name in zip([out, lse] + grads, ("out", "lse", "dq", "dk", "dv")):
            assert torch.equal(got, want[name]), name

    # a first call inside a capture is refused and records nothing
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(gpu_lib.ShardConvError) as e:
            gpu_lib.st_attention_packed(seqs, q, k, v, 0.125, out, lse, ws)
        out.fill_(1.0)
    assert e.value.status == 4
    seqs.upload()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(3):
        for t in [out, lse] + grads:
            t.fill_(float(r))
        ws.fill_(r)
        g.replay()
        same()


@pytest.mark.parametrize("q_lens,k_lens", [([5, 70], [0, 0]), ([0, 0], [40, 3]), ([3, 0], [0, 9])])
def test_no_keys_or_no_queries(gpu_lib, q_lens, k_lens):
    """Rows without a key give zeros and -inf, keys without a row zero gradients."""
    for causal in (False, True):
        host = inputs(q_lens, k_lens, 4, 2, 64, "bf16", seed=9)
        r = run(gpu_lib, *[t.cuda() for t in host], q_lens, k_lens, "bf16", causal, 0.1)
        assert all(bool((r[n] == 0).all()) for n in ("out", "dq", "dk", "dv")) and bool(torch.isneginf(r["lse"]).all())


def test_offsets_past_32_bits(gpu_lib):
    """Keys and values 128 KiB apart: the last lie 8.6 GB into their buffer."""
    n, gap = 65600, 65536
    rng = np.random.default_rng(10)
    k, v = (torch.from_numpy(rng.normal(size=(n, 1, 64))).bfloat16().cuda() for _ in range(2))
    q = torch.from_numpy(rng.normal(size=(3, 2, 64))).bfloat16().cuda()
    big = torch.empty(n, 1, gap, dtype=torch.bfloat16, device="cuda")
    kb, vb = big[:, :, :64], big[:, :, gap - 64:]
    kb.copy_(k)
    vb.copy_(v)
    dout = torch.ones_like(q)
    want = run(gpu_lib, q, k, v, dout, [3], [n], "bf16", True, 0.125)
    got = run(gpu_lib, q, kb, vb, dout, [3], [n], "bf16", True, 0.125)
    for name in ("out", "lse", "dq", "dk", "dv"):
        assert torch.equal(got[name], want[name]), name


def test_refusals_on_the_gpu(gpu_lib):
    seqs = gpu_lib.st_plan_sequences([8], None, 2, 2, 64, "bf16", False)
    t = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")

    def status(f):
        with pytest.raises(gpu_lib.ShardConvError) as e:
            f()
        return e.value.status

    st = gpu_lib.st_attention_packed
    assert status(lambda: st(seqs, t.float(), t, t, 0.1, t)) == 1          # dtype
    assert status(lambda: st(seqs, t[:4], t, t, 0.1, t)) == 2              # shape
    assert status(lambda: st(seqs, t, t, t, 0.0, t)) == 1                  # scale
    assert status(lambda: st(seqs, t, t, t, float("nan"), t)) == 1
    assert status(lambda: st(seqs, t.cpu(), t, t, 0.1, t)) == 1            # not on the GPU
    odd = torch.zeros(8, 2, 68, dtype=torch.bfloat16, device="cuda")[:, :, :64]
    assert status(lambda: st(seqs, odd, t, t, 0.1, t)) == 7                # 136-byte strides
    shifted = torch.zeros(8 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 2, 64)
    assert status(lambda: st(seqs, t, t, shifted, 0.1, t)) == 7            # pointer off by 2 bytes
    wide = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(8, 2, 64)
    assert status(lambda: st(seqs, t, t, t, 0.1, wide)) == 2               # rows overlap
    long = gpu_lib.st_plan_sequences([1], [9000], 2, 2, 64, "bf16", False)
    q, k = t[:1], torch.zeros(9000, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.st_attention_workspace_bytes(long) > 0
    assert status(lambda: st(long, q, k, k, 0.1, torch.empty_like(q))) == 5  # no workspace
    b = gpu_lib.st_attention_packed_backward
    lse = torch.zeros(8, 2, device="cuda")
    assert status(lambda: b(seqs, t, t, t, t, lse, t, 0.1, t, t, t, None)) == 5
    assert status(lambda: b(seqs, t, t, t, t, None, t, 0.1, t, t, t, lse)) == 1


def test_more_tiles_than_one_launch_holds(gpu_lib):
    """2^22 sequences of one token with 16 heads are 2^26 one-wave workgroups, one
    more than a launch takes.  A single key weighs one: out = v, dv = dout, and
    nothing is left of dq and dk."""
    n, heads, dim = (1 << 22) + 3, 16, 8
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v, dout = (torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(4))
    r = run(gpu_lib, q, k, v, dout, [1] * n, [1] * n, "bf16", False, 0.3)
    assert torch.equal(r["out"], v) and torch.equal(r["dv"], dout)
    assert not r["dq"].any() and not r["dk"].any()
    assert bool(((r["lse"] - 0.3 * (q.float() * k.float()).sum(-1)).abs() < 1e-4).all())


@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [("bf16", 4, 2, 64), ("f32", 2, 1, 128), ("f32", 2, 2, 64)])
def test_token_strides_at_the_limit(gpu_lib, dtype, heads, kv_heads, dim):
    """Tokens as far apart as both calls take: 16 MiB, 8 MiB of v of wide fp32 heads."""
    n = 150
    host = inputs([n], [n], heads, kv_heads, dim, dtype, seed=13)
    dev = [t.cuda() for t in host]
    want = run(gpu_lib, *dev, [n], [n], dtype, True, 0.1)
    es = 2 if dtype == "bf16" else 4

    def far(t, stride, at):
        big = torch.empty(n * stride // es, dtype=t.dtype, device="cuda")
        v = big[at:].as_strided(t.shape, (stride // es, dim, 1), at)
        v.copy_(t)
        return v

    q, k, v, dout = dev
    wide = dtype == "f32" and dim > 64
    q, k, dout = far(q, 1 << 24, 64), far(k, 1 << 24, 0), far(dout, 1 << 24, 128)
    v = far(v, 1 << 23 if wide else 1 << 24, 0)
    seqs = gpu_lib.st_plan_sequences([n], [n], heads, kv_heads, dim, dtype, True)
    ws = torch.empty(gpu_lib.st_attention_workspace_bytes(seqs, True), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want["out"]), torch.empty_like(want["lse"])
    gpu_lib.st_attention_packed(seqs, q, k, v, 0.1, out, lse, ws)
    grads = [torch.empty_like(want[g]) for g in ("dq", "dk", "dv")]
    gpu_lib.st_attention_packed_backward(seqs, q, k, v, out, lse, dout, 0.1, *grads, ws)
    for got, name in zip([out, lse] + grads, ("out", "lse", "dq", "dk", "dv")):
        assert torch.equal(got, want[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,heads,kv_heads,dim", [
    ([130], [3000], 2, 1, 96), ([130], [3000], 2, 2, 128), ([140], [1700], 1, 1, 72),     # keys split for out and dq
    ([1, 20], [900, 2500], 4, 2, 96), ([2], [3000], 3, 1, 128),                           # one-wave tiles
    ([3000], [130], 1, 1, 96), ([1500], [20], 2, 1, 128),                                 # rows split for dk and dv
])
def test_split_work_of_wide_heads(gpu_lib, q_lens, k_lens, heads, kv_heads, dim, causal, dtype):
    say(f"split attention {dtype} {heads}/{kv_heads} x {dim} causal={causal} q={q_lens} k={k_lens}")
    host = inputs(q_lens, k_lens, heads, kv_heads, dim, dtype, seed=14)
    dev = [t.cuda() for t in host]
    seqs = gpu_lib.st_plan_sequences(q_lens, k_lens, heads, kv_heads, dim, dtype, causal)
    if not causal or max(q_lens) <= max(k_lens):           # (few rows see a key otherwise)
        assert gpu_lib.st_attention_workspace_bytes(seqs, backward=True) > 4 * sum(q_lens) * heads + 256   # partial results
    r = run(gpu_lib, *dev, q_lens, k_lens, dtype, causal, dim ** -0.5)
    check(r, *host, q_lens, k_lens, dtype, causal, dim ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk,at", [(130, 1500, 300), (130, 1500, 1450), (3, 2000, 700), (600, 600, 290)])
def test_special_values_in_split_and_whole_tiles(gpu_lib, dtype, lq, lk, at):
    """A NaN or infinite value of a key in a tile that every row sees, in a masked
    one of a split row, and a NaN in K, with the scores too close together for any
    weight to underflow: what the rows that see the key get, and no other."""
    heads, kv_heads, dim = 4, 2, 64
    group, first = heads // kv_heads, max(0, at - (lk - lq))
    host = inputs([lq], [lk], heads, kv_heads, dim, dtype, seed=15)
    clean = run(gpu_lib, *[t.cuda() for t in host], [lq], [lk], dtype, True, 0.05, train=False)
    for where in ("k", "v"):
        for value in (math.nan, math.inf, -math.inf):
            if where == "k" and not math.isnan(value):
                continue
            bad = [t.clone() for t in host]
            bad["qkv".index(where)][at, 0, 5] = value
            r = run(gpu_lib, *[t.cuda() for t in bad], [lq], [lk], dtype, True, 0.05, train=False)
            assert torch.equal(r["out"][:first], clean["out"][:first])
            assert torch.equal(r["out"][:, group:], clean["out"][:, group:])
            if where == "k":
                assert bool(torch.isnan(r["out"][first:, :group].float()).all())
                continue
            got = r["out"][first:, :group, 5].float()
            assert bool((torch.isnan(got) if math.isnan(value) else got == value).all()), value
            rest = r["out"].clone()
            rest[first:, :group, 5] = clean["out"][first:, :group, 5]
            assert torch.equal(rest, clean["out"])

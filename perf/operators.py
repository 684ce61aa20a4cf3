"""Cases of the token operators: layer norm over sharded volumes, rotary
positions with several axes, attention over packed sequences.

Each case names one call (or one forward and backward pair) as a program on
this library makes it.  run() computes it either in its plain form
(elementary torch operations in 32 bits, rounded once at the end) or, where
`own` is true, through the library's entry points; exact() computes it in 64
bits from the definition.

Formulas
  layer norm   y = (x - mean) * rstd * gamma + beta over the channels of one
               cell; mean and the biased variance of that cell's channels
               dx = rstd * (g - mean(g) - xhat * mean(g * xhat)), g = dy * gamma
               dgamma = sum over cells of dy * xhat, dbeta = sum of dy
  rotation     pair i of an axis section of d channels turns by
               position * base^(-2i/d)
  attention    out = softmax(scale * q k^T) v per sequence and head; lse = log
               of the softmax's denominator; causal: query i of lq sees keys
               0 .. i + lk - lq; a row that sees no key gives 0 and -inf
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one small fp32 volume cut 17/15 along depth (the 4-to-8-channel
        # layer's output): a call where only latency counts
        norm_case("norm vol32 f32", 32, 32, 32, 8, 0, "17,15", "f32", "f32", 0, False),
        # a training step's norm over the 2048^2 image layer's 64 channels in
        # four uneven row shards: narrow rows, pure memory traffic
        norm_case("norm img2048 train", 1, 2048, 2048, 64, 1, "603,470,519,456", "bf16", "bf16", 0, True),
        # the weather grid's fp32 conv output, W cut 900/892, normalised
        # straight into the next conv's padded bf16 shards, and back
        norm_case("norm grid train", 1, 1024, 1792, 256, 2, "900,892", "f32", "bf16", 1, True),
        # a token list with odd sizes: rows that are no power of two wide
        norm_case("norm tokens1000 train", 1, 1, 4099, 1000, 2, "4099", "bf16", "bf16", 0, True),
        # one small image's queries and keys, two axes: latency
        rope_case("rope image small", 0, 37, 70, 8, 8, 64, "32,32", "bf16", "bf16", "halves", False),
        # a video's joint q, k, v projection in fp32, rotated (q and k) and
        # rounded to bf16 for the attention
        rope_case("rope video", 16, 64, 112, 36, 24, 64, "16,24,24", "f32", "bf16", "halves", False),
        # four windows of 8 x 8 tokens: the smallest attention, latency
        attend_case("attend windows small", "64,64,64,64", "", 4, 4, 32, "bf16", False, False, False),
        # a training batch of images at their own resolutions, packed
        attend_case("attend images train", "2590,1,300,1369,961,64,2590,17", "", 8, 8, 64, "bf16", False, True, False),
        # one long causal sequence (time-ordered tokens), grouped heads,
        # q, k and v as views of one projection, trained
        attend_case("attend causal train", "8192", "", 16, 2, 128, "bf16", True, True, True),
        # a long prompt, causal, forward only, odd length
        attend_case("attend prompt", "16001", "", 16, 4, 128, "bf16", True, False, False),
        # attention pooling and single-token serving: one query per sample
        # over long key lists (256^2 tokens and shorter)
        attend_case("attend single tokens", "1,1,1,1", "65536,40000,12345,777", 16, 4, 64, "bf16", False, False, False),
        # fp32 operands, a head width off the powers of two
        attend_case("attend f32 train", "1000,777", "", 4, 4, 40, "f32", False, True, False),
    ]


def norm_case(name, d, h, w, c, axis, sizes, x, y, y_halo, train):
    return {"name": name, "op": "norm", "d": d, "h": h, "w": w, "c": c, "axis": axis, "sizes": sizes, "x": x, "y": y,
            "y_halo": y_halo, "train": train}


def rope_case(name, t, h, w, heads, rotated, dim, axis_dims, x, out, pairs, inverse):
    return {"name": name, "op": "rope", "t": t, "h": h, "w": w, "heads": heads, "rotated": rotated, "dim": dim,
            "axis_dims": axis_dims, "x": x, "out": out, "pairs": pairs, "inverse": inverse}


def attend_case(name, q_lens, k_lens, heads, kv_heads, dim, dtype, causal, train, fused):
    return {"name": name, "op": "attend", "q_lens": q_lens, "k_lens": k_lens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "causal": causal, "train": train, "fused": fused}


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["norm", "rope", "attend", "attend"])
    if kind == "norm":
        c = spread(rng, 8, 8192)
        cells = min(spread(rng, 1, 1 << 22), (1 << 28) // c)
        h = spread(rng, 1, max(1, int(math.sqrt(cells))))
        w = max(1, cells // h)
        parts = rng.randint(1, min(4, h))
        cuts = sorted(rng.sample(range(1, h), parts - 1)) if parts > 1 else []
        sizes = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [h]))
        c_ = norm_case("", 1, h, w, c, 1, sizes, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]),
                       rng.choice([0, 0, 1]) if min(map(int, sizes.split(","))) > 1 else 0, rng.random() < 0.7)
    elif kind == "rope":
        t = rng.choice([0, spread(rng, 1, 32)])
        h, w = spread(rng, 1, 512), spread(rng, 1, 512)
        axes = 3 if t else 2
        parts = [2 * rng.randint(1, 20) for _ in range(axes)]
        dim = sum(parts)
        dim += (-dim) % 8
        tokens = max(1, t) * h * w
        heads = max(1, min(rng.randint(1, 48), (1 << 28) // (tokens * dim)))
        c_ = rope_case("", t, h, w, heads, rng.randint((heads + 1) // 2, heads), dim, ",".join(map(str, parts)),
                       rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]), rng.choice(["halves", "adjacent"]),
                       rng.random() < 0.5)
    else:
        kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 1, 2, 3, 4, 8])
        heads, dim = kv * group, rng.choice([16, 32, 40, 64, 64, 72, 96, 128, 128])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        train, causal = rng.random() < 0.5, rng.random() < 0.5
        most = spread(rng, 1, 8192 if dtype == "bf16" else 2048)
        count = spread(rng, 1, 64)
        room = (1 << 29) // heads  # padded scores
        while most > 1 and count * most * most > room:
            count, most = (count + 1) // 2 if count > 1 else 1, most if count > 1 else most // 2
        lens = [most] + [rng.randint(0, most) for _ in range(count - 1)]
        rng.shuffle(lens)
        kind = rng.choice(["self", "self", "single", "cross"])
        k_lens = ""
        if kind == "single":
            k_lens = ",".join(str(min(65536, n * 8)) for n in lens)
            lens = [1] * count
        elif kind == "cross":
            k_lens = ",".join(str(rng.randint(0, most)) for _ in lens)
        if k_lens and not any(map(int, k_lens.split(","))):
            k_lens = ",".join(["1"] * count)
        c_ = attend_case("", ",".join(map(str, lens)), k_lens, heads, kv, dim, dtype, causal, train,
                         kind == "self" and rng.random() < 0.5)
    del c_["name"]
    return c_


def ints(text):
    return [int(v) for v in text.split(",")]


def lens_of(case):
    q = ints(case["q_lens"])
    return q, ints(case["k_lens"]) if case["k_lens"] else q


def pairs_seen(case):
    """Query-key pairs that the masks leave, per head."""
    n = 0
    for lq, lk in zip(*lens_of(case)):
        if not case["causal"]:
            n += lq * lk
        else:  # rows see lk - lq + 1 .. lk keys, those below one see none
            first = max(1, lk - lq + 1)
            n += (first + lk) * (lk - first + 1) // 2 if lk else 0
    return n


def work(case):
    if case["op"] == "norm":
        n = case["d"] * case["h"] * case["w"] * case["c"]
        ex, ey = SIZE[case["x"]], SIZE[case["y"]]
        per = (ex + ey) + ((ey + ex) if case["train"] else 0)
        return {"bytes": n * per + 8 * case["c"] + (8 * case["c"] if case["train"] else 0),
                "flops": n * (8 + (14 if case["train"] else 0))}
    if case["op"] == "rope":
        tokens = max(1, case["t"]) * case["h"] * case["w"]
        n = tokens * case["heads"] * case["dim"]
        axes = len(ints(case["axis_dims"]))
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["out"]]) + 4 * axes * tokens,
                "flops": 3 * tokens * case["rotated"] * sum(ints(case["axis_dims"]))}
    q, k = lens_of(case)
    d, e = case["dim"], SIZE[case["dtype"]]
    nq, nk = sum(q) * case["heads"] * d * e, sum(k) * case["kv_heads"] * d * e
    flops = 4 * pairs_seen(case) * d * case["heads"]
    bytes_ = 2 * nq + 2 * nk + 4 * sum(q) * case["heads"]
    if case["train"]:
        flops = flops // 4 * 14
        bytes_ += 2 * nq + 2 * nk
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    {"norm": prepare_norm, "rope": prepare_rope, "attend": prepare_attend}[case["op"]](case, g, s)
    if own:
        import halo_sharded_conv_amd
        s["lib"] = halo_sharded_conv_amd
        make_plans(case, s)
    return s


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def shard_shapes(case):
    """Interior extents (d, h, w) of every shard: one axis is cut."""
    full = [case["d"], case["h"], case["w"]]
    return [tuple(n if a == case["axis"] else full[a] for a in range(3)) for n in ints(case["sizes"])]


def padded(case, shape, halo):
    """Shape of a shard buffer [1][d][h][w][c] with its margins (a volume of
    one plane is 2D and has none along depth)."""
    d, h, w = shape
    return (1, d + (2 * halo if case["d"] > 1 else 0), h + 2 * halo, w + 2 * halo, case["c"])


def inner(case, buf, halo):
    if halo == 0:
        return buf
    lo = halo if case["d"] > 1 else 0
    return buf[:, lo:buf.shape[1] - lo, halo:-halo, halo:-halo]


def prepare_norm(case, g, s):
    c, halo = case["c"], case["y_halo"]
    mean, spread_ = normal(g, c), torch.rand(c, generator=g, device="cuda") * 2 + 0.1
    tx, ty = TORCH[case["x"]], TORCH[case["y"]]
    shapes = shard_shapes(case)
    s["x"] = [(mean + spread_ * normal(g, *padded(case, sh, 0))).to(tx) for sh in shapes]
    s["gamma"] = 1 + 0.1 * normal(g, c)
    s["beta"] = 0.1 * normal(g, c)
    s["y"] = [torch.zeros(padded(case, sh, halo), dtype=ty, device="cuda") for sh in shapes]
    s["stats"] = torch.empty(case["d"] * case["h"] * case["w"], 2, device="cuda")
    s["eps"] = 1e-5
    if case["train"]:
        s["dy"] = [normal(g, *padded(case, sh, halo)).to(ty) for sh in shapes]
        s["dx"] = [torch.empty_like(x) for x in s["x"]]
        s["dgamma"], s["dbeta"] = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")


def prepare_rope(case, g, s):
    h, w = case["h"], case["w"]
    # a shard's tokens: their positions start at the shard's offset
    axes = ([torch.arange(case["t"])] if case["t"] else []) + [torch.arange(h) + h // 2, torch.arange(w)]
    grid = torch.meshgrid(*axes, indexing="ij")
    s["positions"] = torch.stack([a.reshape(-1) for a in grid], -1).to(torch.int32).cuda()
    tokens = s["positions"].shape[0]
    s["x"] = normal(g, tokens, case["heads"], case["dim"]).to(TORCH[case["x"]])
    s["out"] = torch.empty(tokens, case["heads"], case["dim"], dtype=TORCH[case["out"]], device="cuda")
    s["axis_dims"] = ints(case["axis_dims"])
    s["base"] = 10000.0


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


def prepare_attend(case, g, s):
    q_lens, k_lens = lens_of(case)
    tq, tk = sum(q_lens), sum(k_lens)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    t = TORCH[case["dtype"]]
    if case["fused"]:
        joint = normal(g, tq, hq + 2 * hk, d).to(t)
        s["q"], s["k"], s["v"] = joint[:, :hq], joint[:, hq:hq + hk], joint[:, hq + hk:]
    else:
        s["q"], s["k"], s["v"] = normal(g, tq, hq, d).to(t), normal(g, tk, hk, d).to(t), normal(g, tk, hk, d).to(t)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty(tq, hq, d, dtype=t, device="cuda")
    s["lse"] = torch.empty(tq, hq, device="cuda")
    for n, v in (("q_len", q_lens), ("k_len", k_lens), ("q_at", starts(q_lens)), ("k_at", starts(k_lens))):
        s[n] = torch.tensor(v, device="cuda")
    s["q_max"], s["k_max"] = max(q_lens), max(k_lens)
    if case["train"]:
        s["dout"] = normal(g, tq, hq, d).to(t)
        if case["fused"]:
            joint = torch.empty(tq, hq + 2 * hk, d, dtype=t, device="cuda")
            s["dq"], s["dk"], s["dv"] = joint[:, :hq], joint[:, hq:hq + hk], joint[:, hq + hk:]
        else:
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))


def make_plans(case, s):
    """The plans and workspaces that a program on the library keeps."""
    lib = s["lib"]
    if case["op"] == "norm":
        full = [case["d"], case["h"], case["w"]]
        cuts = [ints(case["sizes"]) if a == case["axis"] else [full[a]] for a in range(3)]
        nd = 3 if case["d"] > 1 else 2
        plan = lambda halo, t: lib.st_plan_shards(nd, 1, case["c"], full[3 - nd:], cuts[3 - nd:], [halo] * nd, t)  # noqa: E731
        s["x_plan"], s["y_plan"] = plan(0, case["x"]), plan(case["y_halo"], case["y"])
        if case["train"]:
            n = lib.st_layernorm_backward_workspace_bytes(s["x_plan"])
            s["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    elif case["op"] == "attend":
        q_lens, k_lens = lens_of(case)
        s["seqs"] = lib.st_plan_sequences(q_lens, k_lens, case["heads"], case["kv_heads"], case["dim"], case["dtype"],
                                          case["causal"])
        n = lib.st_attention_workspace_bytes(s["seqs"], backward=case["train"])
        s["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------- run

def run(s):
    op, train = s["case"]["op"], s["case"].get("train")
    if op == "norm":
        return (run_norm if own else plain_norm)(s, train)
    if op == "rope":
        return (run_rope if own else plain_rope)(s)
    return (run_attend if own else plain_attend)(s, train)


def run_norm(s, train):
    lib = s["lib"]
    lib.st_layernorm_sharded(s["x_plan"], s["x"], s["gamma"], s["beta"], s["eps"], s["y_plan"], s["y"], s["stats"])
    if not train:
        return {"y": s["y"], "stats": s["stats"]}
    lib.st_layernorm_backward(s["x_plan"], s["x"], s["y_plan"], s["dy"], s["gamma"], s["stats"], s["x_plan"], s["dx"],
                              s["dgamma"], s["dbeta"], s["workspace"])
    return {"y": s["y"], "stats": s["stats"], "dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def run_rope(s):
    c = s["case"]
    s["lib"].st_rope_axes(s["x"], s["positions"], s["axis_dims"], s["out"], rotated_heads=c["rotated"], base=s["base"],
                          pairs=c["pairs"], inverse=c["inverse"])
    return s["out"]


def run_attend(s, train):
    lib = s["lib"]
    lib.st_attention_packed(s["seqs"], s["q"], s["k"], s["v"], s["scale"], s["out"], s["lse"], s["workspace"])
    if not train:
        return {"out": s["out"], "lse": s["lse"]}
    lib.st_attention_packed_backward(s["seqs"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["scale"],
                                     s["dq"], s["dk"], s["dv"], s["workspace"])
    return {n: s[n] for n in ("out", "lse", "dq", "dk", "dv")}


# ------------------------------------------------------------ plain forms

def plain_norm(s, train):
    case, halo = s["case"], s["case"]["y_halo"]
    parts = [plain_norm_shard(s, x, inner(case, dy, halo).float() if train else None)
             for x, dy in zip(s["x"], s["dy"] if train else s["x"])]
    ys = [put(case, buf, p[0], halo) for buf, p in zip(s["y"], parts)]
    stats = torch.cat([p[1] for p in parts])
    if not train:
        return {"y": ys, "stats": stats}
    return {"y": ys, "stats": stats, "dx": [p[2] for p in parts], "dgamma": sum(p[3] for p in parts),
            "dbeta": sum(p[4] for p in parts)}


def put(case, buf, y, halo):
    inner(case, buf, halo).copy_(y)
    return buf


def plain_norm_shard(s, x, dy):
    c = s["case"]["c"]
    t = x.dtype
    x = x.float()
    mean = x.mean(-1, keepdim=True)
    x = x - mean
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    xhat = x * rstd
    y = xhat * s["gamma"] + s["beta"]
    stats = torch.cat([mean, rstd], -1).reshape(-1, 2)
    if dy is None:
        return y, stats
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return y, stats, dx.to(t), (dy * xhat).reshape(-1, c).sum(0), dy.reshape(-1, c).sum(0)


def plain_rope(s):
    case, x = s["case"], s["x"]
    r, dims = case["rotated"], s["axis_dims"]
    lo = [sum(dims[:a]) for a in range(len(dims))]
    turned = [plain_section(x[:, :r, lo[a]:lo[a] + d].float(), s["positions"][:, a], d, s) for a, d in enumerate(dims)]
    turned = torch.cat(turned + [x[:, :r, sum(dims):].float()], -1)
    return torch.cat([turned, x[:, r:].float()], 1).to(s["out"].dtype)


def plain_section(x, position, d, s):
    case = s["case"]
    turn = s["base"] ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float32) / d)
    angle = position.float()[:, None, None] * turn
    cos, sin = torch.cos(angle), torch.sin(angle)
    if case["inverse"]:
        sin = -sin
    if case["pairs"] == "halves":
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def pad(x, at, length, most):
    """Packed [T][H][D] as [B][H][most][D] in 32 bits, zeros past each length."""
    i = torch.arange(most, device=x.device)
    rows = x.float()[(at[:, None] + i).clamp(max=x.shape[0] - 1)]
    return torch.where((i < length[:, None])[:, :, None, None], rows, 0.0).transpose(1, 2).contiguous()


def pack(x, at, length, total):
    """[B][H][most][...] back to packed [T][H][...]."""
    b = torch.repeat_interleave(torch.arange(len(at), device=x.device), length, output_size=total)
    return x[b, :, torch.arange(total, device=x.device) - at[b]]


def plain_attend(s, train):
    case, t = s["case"], s["q"].dtype
    group = case["heads"] // case["kv_heads"]
    q = pad(s["q"], s["q_at"], s["q_len"], s["q_max"])
    k = pad(s["k"], s["k_at"], s["k_len"], s["k_max"]).repeat_interleave(group, 1)
    v = pad(s["v"], s["k_at"], s["k_len"], s["k_max"]).repeat_interleave(group, 1)
    i = torch.arange(s["q_max"], device=q.device)[:, None]
    j = torch.arange(s["k_max"], device=q.device)[None, :]
    seen = (j < s["k_len"][:, None, None]) & (i < s["q_len"][:, None, None])
    if case["causal"]:
        seen = seen & (j <= i + (s["k_len"] - s["q_len"])[:, None, None])
    seen = seen[:, None]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~seen, -math.inf)
    most = p.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    p = p.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, 1.0, total))
    o = torch.matmul(p, v)
    tq, tk = s["q"].shape[0], s["k"].shape[0]
    out = pack(o, s["q_at"], s["q_len"], tq).to(t)
    lse = pack((most + total.log())[..., 0], s["q_at"], s["q_len"], tq)
    if not train:
        return {"out": out, "lse": lse}
    do = pad(s["dout"], s["q_at"], s["q_len"], s["q_max"])
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    shared = (len(dk), case["kv_heads"], group, s["k_max"], case["dim"])
    dk, dv = dk.reshape(shared).sum(2), dv.reshape(shared).sum(2)
    return {"out": out, "lse": lse, "dq": pack(dq, s["q_at"], s["q_len"], tq).to(t),
            "dk": pack(dk, s["k_at"], s["k_len"], tk).to(t), "dv": pack(dv, s["k_at"], s["k_len"], tk).to(t)}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    {"norm": prepare_norm, "rope": prepare_rope, "attend": prepare_attend}[case["op"]](case, g, s)
    return {"norm": exact_norm, "rope": exact_rope, "attend": exact_attend}[case["op"]](case, s)


def exact_norm(case, s):
    halo, c = case["y_halo"], case["c"]
    gamma, beta = s["gamma"].double(), s["beta"].double()
    out = {"y": [], "stats": [], "dx": []}
    dgamma = torch.zeros(c, dtype=torch.float64, device="cuda")
    dbeta = torch.zeros_like(dgamma)
    for i, x in enumerate(s["x"]):
        x = x.double()
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        rstd = (var + s["eps"]) ** -0.5
        y = torch.zeros(s["y"][i].shape, dtype=torch.float64, device="cuda")
        inner(case, y, halo).copy_((x - mean) * rstd * gamma + beta)
        out["y"].append(y)
        out["stats"].append(torch.stack([mean.reshape(-1), rstd.reshape(-1)], 1))
        if case["train"]:
            dy = inner(case, s["dy"][i], halo).double()
            u = (x - mean) * rstd
            h = dy * gamma
            out["dx"].append(rstd / c * (c * h - h.sum(-1, keepdim=True) - u * (h * u).sum(-1, keepdim=True)))
            dgamma += (dy * u).sum((0, 1, 2, 3))
            dbeta += dy.sum((0, 1, 2, 3))
    out["stats"] = torch.cat(out["stats"])
    if not case["train"]:
        return {"y": out["y"], "stats": out["stats"]}
    return {**out, "dgamma": dgamma, "dbeta": dbeta}


def exact_rope(case, s):
    out = s["x"].double()
    lo = 0
    for a, d in enumerate(s["axis_dims"]):
        for i in range(d // 2):
            m, n = (lo + i, lo + d // 2 + i) if case["pairs"] == "halves" else (lo + 2 * i, lo + 2 * i + 1)
            angle = s["positions"][:, a].double() * s["base"] ** (-2.0 * i / d) * (-1 if case["inverse"] else 1)
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            z = torch.complex(s["x"][:, :case["rotated"], m].double(), s["x"][:, :case["rotated"], n].double()) * turn
            out[:, :case["rotated"], m], out[:, :case["rotated"], n] = z.real, z.imag
        lo += d
    return out


def exact_attend(case, s):
    q_lens, k_lens = lens_of(case)
    group = case["heads"] // case["kv_heads"]
    like = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"out": like(s["out"]), "lse": like(s["lse"])}
    if case["train"]:
        out.update(dq=like(s["q"]), dk=like(s["k"]), dv=like(s["v"]))
    q0 = k0 = 0
    for lq, lk in zip(q_lens, k_lens):
        rows, keys = slice(q0, q0 + lq), slice(k0, k0 + lk)
        q0, k0 = q0 + lq, k0 + lk
        for h in range(case["heads"]) if lq else ():
            if not lk:
                out["lse"][rows, h] = -math.inf
                continue
            q, k, v = s["q"][rows, h].double(), s["k"][keys, h // group].double(), s["v"][keys, h // group].double()
            z = s["scale"] * (q @ k.mT)
            if case["causal"]:
                z += torch.full((lq, lk), -math.inf, dtype=torch.float64, device="cuda").triu_(lk - lq + 1)
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None])
            out["out"][rows, h], out["lse"][rows, h] = p @ v, lse
            if case["train"]:
                do = s["dout"][rows, h].double()
                dp = do @ v.mT
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                out["dq"][rows, h] = ds @ k
                out["dk"][keys, h // group] += ds.mT @ q
                out["dv"][keys, h // group] += p.mT @ do
    return out

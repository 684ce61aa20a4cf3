"""Cases of the MLP branch's operators: matrix products with bias, activation and
residual, root-mean-square norm with the residual's addition, activations held
in 8 bits.

Each case names one call (or one forward and backward pair) as a program on
this library makes it.  run() computes it either in its plain form (elementary
torch operations in 32 bits, rounded once at the end) or, where `own` is true,
through the library's entry points; exact() computes it in 64 bits from the
definition.

Formulas (M rows)
  linear    z = x w^T + bias;  y = act(z) + residual;  pre = z, kept for the
            backward pass
            p = dy * act'(pre);  dx = p w;  dw = p^T x;  dbias = sum of p
            act: none, relu, gelu (z * Phi(z)), silu (z * sigmoid(z))
  rms norm  s = x + residual, in the type it is kept in
            y = s * rstd * gamma, rstd = 1 / sqrt(mean(s^2) + eps)
            dx = ds + rstd * (g - xh * mean(g * xh)), g = dy * gamma, xh = s * rstd
            dgamma = sum over rows of dy * xh
  mx8       blocks of 32 channels of a row: k the smallest power with
            max |v| <= 448 * 2^k; codes v * 2^-k rounded to e4m3 (nearest even);
            held as code bytes and a byte k + 127 (1 .. 254) per block
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4.0, "bf16": 2.0, "mx8": 1 + 1 / 32, "": 0.0}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of 16 heads of 128 through the widening product: serving, the
        # weights' bytes count
        linear_case("linear token", 1, 2048, 8192, "bf16", "gelu", "", "bf16", ""),
        # a small batch of tokens through the narrowing product in 8 bits
        linear_case("linear few tokens mx8", 33, 8192, 2048, "mx8", "none", "bf16", "bf16", ""),
        # odd sizes in fp32: rows that are no power of two wide, a residual
        linear_case("linear odd f32", 4099, 1000, 257, "f32", "silu", "f32", "f32", ""),
        # a 128^2 volume's tokens through the widening product in training: the
        # pre-activation is kept in 8 bits
        linear_case("linear up kept", 16384, 2048, 8192, "bf16", "gelu", "", "bf16", "mx8"),
        # the narrowing product with both operands in 8 bits, onto the fp32 stream
        linear_case("linear down mx8", 16384, 8192, 2048, "mx8", "none", "f32", "bf16", ""),
        # gradients of the joint q, k, v projection of 12 heads of 64 over 16 x 32^2 cells
        backward_case("linear joint backward", 16384, 768, 2304, "bf16", "none", "bf16", ""),
        # gradients of the widening product, its input and its pre-activation kept
        # in 8 bits since the forward pass
        backward_case("linear up kept backward", 16384, 2048, 8192, "bf16", "gelu", "mx8", "mx8"),
        # one token's norm: latency
        norm_case("norm token", 1, 2048, "f32", "bf16", "f32", "mx8", False, ""),
        # the weather grid's cells, a bf16 branch added to the fp32 stream, the
        # output in 8 bits for the next product
        norm_case("norm grid mx8", 1024 * 1792, 256, "f32", "bf16", "f32", "mx8", False, ""),
        # a token list with odd sizes, trained, the sum kept in bf16
        norm_case("norm tokens1000 train", 65536, 1000, "bf16", "bf16", "bf16", "bf16", True, "bf16"),
        # an image layer's activations to 8 bits and back
        store_case("checkpoint img2048", 2048 * 2048, 64, "bf16", "none", "bf16"),
        # odd sizes: blocks that end before 32 channels; read back through the activation
        store_case("checkpoint odd gelu", 4099, 1001, "f32", "gelu", "bf16"),
    ]


def linear_case(name, m, k, n, dtype, act, residual, y, pre):
    """pre: the type that the pre-activation is kept in ("": it is not)."""
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "residual": residual, "y": y,
            "pre": pre}


def backward_case(name, m, k, n, dtype, act, x, pre):
    """x, pre: the types that the input and the pre-activation were kept in."""
    return {"name": name, "op": "backward", "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "x": x, "pre": pre}


def norm_case(name, m, c, x, residual, total, y, train, kept):
    """kept: the type that the sum has in the backward pass."""
    return {"name": name, "op": "norm", "m": m, "c": c, "x": x, "residual": residual, "total": total, "y": y,
            "train": train, "kept": kept}


def store_case(name, m, c, x, act, out):
    return {"name": name, "op": "store", "m": m, "c": c, "x": x, "act": act, "out": out}


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "backward", "norm", "store"])
    if kind in ("linear", "backward"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"] if kind == "backward" else ["bf16", "bf16", "mx8", "f32"])
        k, n = spread(rng, 8, 8192), spread(rng, 8, 8192)
        if rng.random() < 0.6:
            k, n = max(8, k // 8 * 8), max(8, n // 8 * 8)
        room = (1 << 38) // (8 if dtype == "f32" else 1)
        m = min(spread(rng, 1, 1 << 16), max(1, room // (k * n)))
        act = rng.choice(["none", "relu", "gelu", "silu"])
        plain = "f32" if dtype == "f32" else "bf16"
        if kind == "linear":
            c = linear_case("", m, k, n, dtype, act, rng.choice(["", "f32", "bf16"]), rng.choice([plain, plain, "f32", "mx8"]),
                            rng.choice(["", plain, "mx8"]))
        else:
            pre = rng.choice([plain, "mx8"])
            c = backward_case("", m, k, n, dtype, act, rng.choice([plain, "mx8"]), "" if act == "none" else pre)
    else:
        c = spread(rng, 8, 8192)
        if rng.random() < 0.6:
            c = max(8, c // 8 * 8)
        m = min(spread(rng, 1, 1 << 22), (1 << 28) // c)
        if kind == "norm":
            train, total = rng.random() < 0.5, rng.choice(["f32", "bf16"])
            c = norm_case("", m, c, rng.choice(["f32", "bf16"]), rng.choice(["", "f32", "bf16"]), total,
                          rng.choice(["f32", "bf16", "mx8"]) if not train else rng.choice(["f32", "bf16"]), train,
                          rng.choice([total, "mx8"]) if train else "")
        else:
            c = store_case("", m, c, rng.choice(["f32", "bf16"]), rng.choice(["none", "relu", "gelu", "silu"]),
                           rng.choice(["f32", "bf16"]))
    del c["name"]
    return c


def work(case):
    if case["op"] in ("linear", "backward"):
        m, k, n, e = case["m"], case["k"], case["n"], SIZE[case["dtype"]]
        if case["op"] == "linear":
            return {"bytes": (m * k + n * k) * e + m * n * (SIZE[case["y"]] + SIZE[case["residual"]] + SIZE[case["pre"]]) + 4 * n,
                    "flops": 2 * m * k * n}
        return {"bytes": m * k * (SIZE[case["x"]] + e) + 2 * n * k * e + m * n * (e + SIZE[case["pre"]]) + 4 * n,
                "flops": 4 * m * k * n}
    n = case["m"] * case["c"]
    if case["op"] == "norm":
        once = n * (SIZE[case["x"]] + SIZE[case["residual"]] + SIZE[case["total"]] + SIZE[case["y"]]) + 4 * case["c"]
        if case["train"]:  # dy, ds in; dx, dgamma out
            once += n * (SIZE[case["y"]] + 2 * SIZE[case["total"]]) + 4 * case["c"]
        return {"bytes": once, "flops": n * (12 if case["train"] else 5)}
    return {"bytes": n * (SIZE[case["x"]] + SIZE[case["out"]]), "flops": n * 6}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    s = inputs(case, seed)
    if own:
        import halo_sharded_conv_amd
        s["lib"] = halo_sharded_conv_amd
        make_own(case, s)
    return s


def inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    {"linear": prepare_linear, "backward": prepare_backward, "norm": prepare_norm, "store": prepare_store}[case["op"]](case, g, s)
    return s


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def empty(dtype, *shape):
    return torch.empty(*shape, dtype=TORCH[dtype], device="cuda")


def held(v, dtype):
    """v in the type that a program has it in."""
    return mx8_held(v) if dtype == "mx8" else v.to(TORCH[dtype])


def returned(dtype):
    """8-bit outputs are returned as the values they stand for, which bf16 holds."""
    return "bf16" if dtype == "mx8" else dtype


def tokens_and_weight(case, g):
    # a norm's output, with channels of different size; weights that keep it
    m, k, n = case["m"], case["k"], case["n"]
    return normal(g, m, k) * (0.25 + 1.5 * torch.rand(k, generator=g, device="cuda")), normal(g, n, k) / math.sqrt(k)


def prepare_linear(case, g, s):
    m, n = case["m"], case["n"]
    x, w = tokens_and_weight(case, g)
    s["x"], s["w"] = held(x, case["dtype"]), held(w, case["dtype"])
    s["bias"] = 0.2 * normal(g, n)
    s["residual"] = normal(g, m, n).to(TORCH[case["residual"]]) if case["residual"] else None
    s["y"] = empty(returned(case["y"]), m, n)
    s["pre"] = empty(returned(case["pre"]), m, n) if case["pre"] else None


def prepare_backward(case, g, s):
    m, k, n = case["m"], case["k"], case["n"]
    x, w = tokens_and_weight(case, g)
    s["x"], s["w"] = held(x, case["x"]), held(w, case["dtype"])
    s["pre"] = held(1.2 * normal(g, m, n) + 0.2 * normal(g, n), case["pre"]) if case["pre"] else None
    s["dy"] = normal(g, m, n).to(TORCH[case["dtype"]])
    s["dx"], s["dw"], s["dbias"] = empty(case["dtype"], m, k), empty(case["dtype"], n, k), empty("f32", n)


def prepare_norm(case, g, s):
    m, c = case["m"], case["c"]
    size = 0.1 + 2 * torch.rand(c, generator=g, device="cuda")
    s["x"] = (normal(g, m, c) * size).to(TORCH[case["x"]])
    s["residual"] = (0.5 * normal(g, m, c)).to(TORCH[case["residual"]]) if case["residual"] else None
    s["gamma"] = 1 + 0.1 * normal(g, c)
    s["eps"] = 1e-6
    s["total"] = empty(case["total"], m, c)
    s["rstd"] = torch.empty(m, device="cuda")
    s["y"] = empty(returned(case["y"]), m, c)
    if case["train"]:
        s["dy"] = normal(g, m, c).to(TORCH[case["y"]])
        s["dtotal"] = normal(g, m, c).to(TORCH[case["total"]])
        s["dx"], s["dgamma"] = empty(case["total"], m, c), torch.empty(c, device="cuda")


def prepare_store(case, g, s):
    m, c = case["m"], case["c"]
    s["x"] = (normal(g, m, c) * (0.05 + 2 * torch.rand(c, generator=g, device="cuda"))).to(TORCH[case["x"]])
    s["out"] = empty(case["out"], m, c)


def mx8_held(v):
    """Codes [m, c rounded up to 16] and scales [m, blocks rounded up to 4] as bytes."""
    m, c = v.shape
    codes = torch.zeros(m, -(-c // 16) * 16, dtype=torch.uint8, device=v.device)
    scales = torch.zeros(m, -(-c // 128) * 4, dtype=torch.uint8, device=v.device)
    byte = block_scale(v)
    grid = v * power(254 - byte).repeat_interleave(32, 1)[:, :c]
    codes[:, :c] = grid.to(torch.float8_e4m3fn).view(torch.uint8)
    scales[:, :byte.shape[1]] = byte.to(torch.uint8)
    return codes, scales, c


def make_own(case, s):
    """The holders and workspaces that a program on the library keeps."""
    lib = s["lib"]
    for name in ("x", "w", "pre"):
        if isinstance(s.get(name), tuple):
            s[name] = lib.Mx8(*s[name])
    if case["op"] in ("linear", "backward"):
        m, k, n = case["m"], case["k"], case["n"]
        need = lib.st_linear_workspace_bytes(m, k, n, case["dtype"], backward=case["op"] == "backward")
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
        for name in ("y", "pre") if case["op"] == "linear" else ():
            if case[name] == "mx8":
                s[name + "8"] = lib.mx8_empty(m, n)
    elif case["op"] == "norm":
        m, c = case["m"], case["c"]
        if case["y"] == "mx8":
            s["y8"] = lib.mx8_empty(m, c)
        if case["kept"] == "mx8":
            s["total8"] = lib.mx8_empty(m, c)
        if case["train"]:
            need = lib.st_rmsnorm_backward_workspace_bytes(m, c)
            s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    else:
        s["x8"] = lib.mx8_empty(case["m"], case["c"])


# --------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if op == "linear":
        return (run_linear if own else plain_linear)(s, s["case"])
    if op == "backward":
        return (run_backward if own else plain_backward)(s, s["case"])
    if op == "norm":
        return (run_norm if own else plain_norm)(s, s["case"])
    return (run_store if own else plain_store)(s, s["case"])


def run_linear(s, case):
    lib = s["lib"]
    lib.st_linear(s["x"], s["w"], s["bias"], s.get("y8", s["y"]), act=case["act"], residual=s["residual"],
                  pre=s.get("pre8", s["pre"]), workspace=s["workspace"])
    if "y8" in s:
        lib.st_mx8_load(s["y8"], s["y"])
    if "pre8" in s:
        lib.st_mx8_load(s["pre8"], s["pre"])
    return {"y": s["y"], "pre": s["pre"]}


def run_backward(s, case):
    s["lib"].st_linear_backward(s["x"], s["w"], s["dy"], s["dx"], s["dw"], s["dbias"], act=case["act"], pre=s["pre"],
                                workspace=s["workspace"])
    return {n: s[n] for n in ("dx", "dw", "dbias")}


def run_norm(s, case):
    lib = s["lib"]
    y8 = s.get("y8")
    lib.st_rmsnorm(s["x"], s["residual"], s["gamma"], s["eps"], total=s["total"], y=None if y8 else s["y"], y8=y8,
                   rstd=s["rstd"])
    if y8:
        lib.st_mx8_load(y8, s["y"])
    if not case["train"]:
        return {"total": s["total"], "y": s["y"], "rstd": s["rstd"]}
    total = s["total"]
    if case["kept"] == "mx8":
        total = s["total8"]
        lib.st_mx8_store(s["total"], total)
    lib.st_rmsnorm_backward(total, s["dy"], s["dtotal"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["workspace"])
    return {n: s[n] for n in ("total", "y", "rstd", "dx", "dgamma")}


def run_store(s, case):
    s["lib"].st_mx8_store(s["x"], s["x8"])
    s["lib"].st_mx8_load(s["x8"], s["out"], act=case["act"])
    return s["out"]


# ------------------------------------------------------------ plain forms

def power(byte):
    """2^(byte - 127) for whole numbers 1 .. 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def block_scale(v):
    """The scale byte of every block of 32 channels, from the largest value's bits."""
    m, c = v.shape
    v = torch.nn.functional.pad(v.abs(), (0, -c % 32)).reshape(m, -1, 32)
    bits = v.amax(-1).view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(1, 254)


def through_mx8(v):
    """The values that the 8-bit form of v stands for, in 32 bits."""
    byte = block_scale(v)
    c = v.shape[1]
    up, down = (power(b).repeat_interleave(32, 1)[:, :c] for b in (254 - byte, byte))
    return (v * up).to(torch.float8_e4m3fn).float() * down


def values(a):
    """A held tensor's values in 32 bits."""
    if isinstance(a, torch.Tensor):
        return a.float()
    codes, scales, c = a
    blocks = -(-c // 32)
    return codes[:, :c].contiguous().view(torch.float8_e4m3fn).float() * power(scales[:, :blocks]).repeat_interleave(32, 1)[:, :c]


def kept(v, dtype):
    """v as it comes back from the type it is kept in."""
    return through_mx8(v) if dtype == "mx8" else v.to(TORCH[dtype]).float()


def activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    t = 1 / (1 + torch.exp(-z))
    return t * (1 + z * (1 - t))


def plain_linear(s, case):
    z = torch.matmul(values(s["x"]), values(s["w"]).T) + s["bias"]
    y = activate(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = kept(y, case["y"]).to(s["y"].dtype)
    return {"y": y, "pre": kept(z, case["pre"]).to(s["pre"].dtype) if case["pre"] else None}


def plain_backward(s, case):
    p = s["dy"].float()
    if case["act"] != "none":
        p = p * slope(values(s["pre"]), case["act"])
    t = s["dx"].dtype
    return {"dx": torch.matmul(p, values(s["w"])).to(t), "dw": torch.matmul(p.T, values(s["x"])).to(t), "dbias": p.sum(0)}


def plain_norm(s, case):
    total = s["x"].float()
    if s["residual"] is not None:
        total = total + s["residual"].float()
    total = total.to(s["total"].dtype)
    v = total.float()
    rstd = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + s["eps"])
    y = v * rstd * s["gamma"]
    y = (through_mx8(y) if case["y"] == "mx8" else y).to(s["y"].dtype)
    if not case["train"]:
        return {"total": total, "y": y, "rstd": rstd[:, 0]}
    xh = kept(v, case["kept"]) * rstd
    dy = s["dy"].float()
    g = dy * s["gamma"]
    dx = s["dtotal"].float() + rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    return {"total": total, "y": y, "rstd": rstd[:, 0], "dx": dx.to(s["dx"].dtype), "dgamma": (dy * xh).sum(0)}


def plain_store(s, case):
    return activate(through_mx8(s["x"].float()), case["act"]).to(s["out"].dtype)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    return {"linear": exact_linear, "backward": exact_backward, "norm": exact_norm,
            "store": exact_store}[case["op"]](case, inputs(case, seed))


def two64(e):
    """2^e for whole numbers in fp64's range, by its exponent bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def read64(a):
    if isinstance(a, torch.Tensor):
        return a.double()
    codes, scales, c = a
    v = codes[:, :c].int()
    exponent, mantissa = (v >> 3) & 15, (v & 7).double()
    size = torch.where(exponent == 0, mantissa / 512, (8 + mantissa) * two64(exponent - 10))
    block = torch.arange(c, device=v.device) // 32
    return torch.where(v > 127, -size, size) * two64(scales.int()[:, block] - 127)


def grid64(v):
    """Rounded to the 8-bit form: step by step from the block's largest value."""
    m, c = v.shape
    out = torch.empty_like(v)
    for lo in range(0, c, 32):
        part = v[:, lo:lo + 32]
        top = part.abs().amax(1, keepdim=True)
        e = torch.frexp(top / 448)[1]
        k = torch.where(top <= 448 * two64(e - 1), e - 1, e).clamp(-126, 127)
        u = part * two64(-k)
        step = two64((torch.frexp(u)[1] - 1).clamp(min=-6) - 3)
        out[:, lo:lo + 32] = torch.round(u / step) * step * two64(k)
    return out


def keep64(v, dtype):
    return grid64(v) if dtype == "mx8" else v.to(TORCH[dtype]).double()


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(z) if act == "silu" else z


def exact_linear(case, s):
    z = read64(s["x"]) @ read64(s["w"]).mT + s["bias"].double()
    y = act64(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": grid64(y) if case["y"] == "mx8" else y, "pre": None if not case["pre"] else grid64(z) if case["pre"] == "mx8" else z}


def exact_backward(case, s):
    p = s["dy"].double()
    if case["pre"]:
        z = read64(s["pre"])
        if case["act"] == "relu":
            p = p * (z > 0)
        elif case["act"] == "gelu":
            p = p * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5)
        else:
            t = torch.sigmoid(z)
            p = p * (t + z * t * torch.sigmoid(-z))
    return {"dx": p @ read64(s["w"]), "dw": p.mT @ read64(s["x"]), "dbias": p.sum(0)}


def exact_norm(case, s):
    out = {n: [] for n in ("total", "y", "rstd", "dx")}
    dgamma = 0.0
    for rows in torch.arange(case["m"], device="cuda").split(1 << 18):
        part = slice(int(rows[0]), int(rows[-1]) + 1)
        total = s["x"][part].double()
        if s["residual"] is not None:
            total = total + s["residual"][part].double()
        total = total.float().to(TORCH[case["total"]]).double()  # 32 bits, then its type
        rstd = (total.square().sum(1) / case["c"] + s["eps"]) ** -0.5
        y = s["gamma"].double() * total * rstd[:, None]
        out["total"].append(total)
        out["y"].append(grid64(y) if case["y"] == "mx8" else y)
        out["rstd"].append(rstd)
        if case["train"]:
            dy, u = s["dy"][part].double(), keep64(total, case["kept"]) * rstd[:, None]
            h = dy * s["gamma"].double()
            out["dx"].append(s["dtotal"][part].double() + rstd[:, None] * (h - u * (h * u).sum(1, keepdim=True) / case["c"]))
            dgamma = dgamma + (dy * u).sum(0)
    out = {n: torch.cat(v) for n, v in out.items() if v}
    return {**out, "dgamma": dgamma} if case["train"] else out


def exact_store(case, s):
    return act64(grid64(s["x"].double()), case["act"])

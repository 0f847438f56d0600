"""Measured cases of the packed-row operators: matrices kept in 8 bits with one scale for each row, written from and read
into floating-point tensors, multiplied as integers (a linear layer's forward pass), and used in the backward pass (the
weight gradient from the layer's packed input, the input gradient from packed weights, an activation function's gradient
from its packed input).

Rows are tokens (activations) or output channels (weights).  With `own` false everything is computed by elementary torch
operations; with `own` true by the library's calls."""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    # widths: 256/688 are the small model's, 1600/6400 the 1.5B-shaped model's, 4096/11008 those of the 7.5B list
    return [
        # --- keep: pack a tensor into 8 bits, later restore it (an activation checkpoint by itself)
        # one short sequence of the small model: latency of two launches
        dict(name="keep-mini-bf16", op="keep", rows=509, cols=256, src="bf16", dst="bf16", rule="pow2"),
        # the MLP's inner activations of a long batch
        dict(name="keep-7p5b-bf16", op="keep", rows=16384, cols=11008, src="bf16", dst="bf16", rule="pow2"),
        # --- linear: y = x w^T in 8-bit integers, scales for each token and channel
        # one new token through the widest layer: bound by the weights' bytes
        dict(name="linear-token-bf16", op="linear", rows=1, k=4096, n=11008, dst="bf16", rule="max"),
        # the query, key and value projection of one sequence of the 1.5B shape, with its bias
        dict(name="linear-gpt2-bf16", op="linear", rows=1024, k=1600, n=4800, dst="bf16", rule="max", bias="bf16"),
        # the widest layer over a long batch: the largest product
        dict(name="linear-7p5b-bf16", op="linear", rows=16384, k=4096, n=11008, dst="bf16", rule="pow2"),
        # --- weight gradient from the packed input
        # two micro-steps of the 1.5B shape accumulated in fp32, with the bias's gradient
        dict(name="weight-gpt2-bf16-f32", op="weight", rows=4096, k=1600, n=6400, dy="bf16", dst="f32", steps=2,
             bias="f32"),
        # a layer of the 7.5B list into the 16-bit send buffer
        dict(name="weight-7p5b-bf16", op="weight", rows=8192, k=4096, n=11008, dy="bf16", dst="bf16", steps=1),
        # a ragged fp16 batch with odd widths
        dict(name="weight-odd-f16", op="weight", rows=1003, k=333, n=1043, dy="f16", dst="f32", steps=1),
        # --- input gradient from packed weights
        # the 1.5B shape's second MLP layer
        dict(name="input-gpt2-bf16", op="input", rows=4096, k=6400, n=1600, dy="bf16", dst="bf16", rule="pow2"),
        # a ragged fp16 batch of the 7.5B list's attention projection
        dict(name="input-7p5b-odd-f16", op="input", rows=2047, k=4096, n=4096, dy="f16", dst="f16", rule="max"),
        # --- activation function: forward (packing its input), backward from the packed input
        # GELU between the 1.5B shape's MLP layers
        dict(name="act-gpt2-gelu-bf16", op="act", rows=2048, cols=6400, kind="gelu", src="bf16", dst="bf16"),
        # gated SiLU of the 7.5B list, the result packed for the next layer
        dict(name="act-7p5b-gated-bf16", op="act", rows=8192, cols=11008, kind="silu", gated=True, src="bf16",
             dst="bf16", packed=True),
    ]


def draw(rng):
    def size(lo, hi, odd=0.4):
        v = int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
        return max(lo, v if rng.random() < odd else (v + 15) // 16 * 16 if v >= 16 else v)

    op = rng.choice(["keep", "linear", "linear", "weight", "weight", "input", "act"])
    half = lambda: rng.choice(["bf16", "bf16", "f16"])
    c = dict(op=op, dst=half())
    if op in ("keep", "act"):
        c.update(rows=size(1, 32768), cols=size(8, 12000), src=rng.choice(["bf16", "bf16", "f16", "f32"]))
        while c["rows"] * c["cols"] > 1.0e8:
            c["rows"] //= 2
        if op == "keep":
            c.update(rule=rng.choice(["pow2", "pow2", "max"]), overflow=rng.random() < 0.1)
        else:
            c.update(kind=rng.choice(["gelu", "silu"]), gated=rng.random() < 0.5, packed=rng.random() < 0.4)
    else:
        c.update(rows=size(1, 32768), k=size(32, 12000), n=size(32, 12000))
        while c["rows"] * c["k"] * c["n"] > 6.0e11:
            big = max(("rows", "k", "n"), key=lambda d: c[d])
            c[big] //= 2
        if op == "linear":
            if rng.random() < 0.4:
                c["rows"] = rng.randint(1, 24)         # generation: a few tokens
            c.update(dst=rng.choice(["bf16", "f16", "f32"]), rule=rng.choice(["max", "max", "pow2"]))
            if rng.random() < 0.4:
                c["bias"] = rng.choice(["bf16", "f32"])
        elif op == "weight":
            c.update(dy=half(), dst=rng.choice(["f32", "f32", "bf16", "f16"]), steps=rng.choice([1, 1, 2]))
            if rng.random() < 0.4:
                c["bias"] = c["dst"]
        else:
            c.update(dy=c["dst"], rule=rng.choice(["pow2", "pow2", "max"]))
    c["strided"] = rng.random() < 0.25
    return c


# --- inputs

def floats(gen, rows, cols, dtype, strided):
    """A matrix, with `strided` the columns of a wider one."""
    wide = cols + 24 if strided else cols
    return torch.randn(rows, wide, generator=gen, dtype=DTYPES[dtype], device="cuda")[:, :cols]


def activations(gen, rows, cols, dtype, strided):
    """Tokens of different magnitude; some channels stand out, as they do behind a norm with learned weights."""
    x = floats(gen, rows, cols, dtype, strided)
    channel = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    token = torch.exp(0.4 * torch.randn(rows, 1, generator=gen, device="cuda"))
    x.mul_(channel.to(x.dtype)).mul_(token.to(x.dtype))
    return x


def gradients(gen, rows, cols, dtype, strided):
    """Gradients of a layer's result: small, tokens differ by decades; fp16 under a loss scale."""
    dy = floats(gen, rows, cols, dtype, strided)
    token = torch.exp(1.0 * torch.randn(rows, 1, generator=gen, device="cuda")) * (0.1 if dtype == "f16" else 1e-4)
    return dy.mul_(token.to(dy.dtype))


def packed(gen, rows, cols, rule, spread):
    """Packed rows as a program has them in hand: q, its rows on 16-byte boundaries with zeros behind them, and scale."""
    pitch = (cols + 15) // 16 * 16
    q = torch.zeros(rows, pitch, dtype=torch.int8, device="cuda")
    # about normal, and the row's largest value is 127 steps (pow2: 64 to 127)
    top = torch.full((rows, 1), 127.0, device="cuda")
    scale = torch.exp(spread * torch.randn(rows, generator=gen, device="cuda")) * 2e-2
    if rule == "pow2":
        top = 64 + 63 * torch.rand(rows, 1, generator=gen, device="cuda")
        scale = torch.exp2(torch.round(torch.log2(scale)))
    v = torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float16)
    v.mul_((top / 3.5).half()).round_().clamp_(-127, 127)
    q[:, :cols] = v.to(torch.int8)
    return dict(q=q, scale=scale, rule=rule, cols=cols)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, strided, dev = case, case.get("strided", False), dict(device="cuda")
    s = dict(case=c)
    if c["op"] == "keep":
        s["x"] = activations(gen, c["rows"], c["cols"], c["src"], strided)
        if c.get("overflow"):
            s["x"][seed % c["rows"], -1] = math.inf
    elif c["op"] == "act":
        wide = 2 * c["cols"] if c.get("gated") else c["cols"]
        s["x"] = activations(gen, c["rows"], wide, c["src"], strided)
        s["dy"] = gradients(gen, c["rows"], c["cols"], c["dst"], strided)
    elif c["op"] == "linear":
        s["xs"] = [packed(gen, c["rows"], c["k"], "pow2", 0.5)]
        s["w"] = packed(gen, c["n"], c["k"], c["rule"], 0.2)
        s["bias"] = torch.randn(c["n"], generator=gen, dtype=DTYPES[c["bias"]], **dev) if "bias" in c else None
    elif c["op"] == "weight":
        s["xs"] = [packed(gen, c["rows"], c["k"], "pow2", 0.5) for _ in range(c["steps"])]
        s["dys"] = [gradients(gen, c["rows"], c["n"], c["dy"], strided) for _ in range(c["steps"])]
    else:
        s["w"] = packed(gen, c["n"], c["k"], c["rule"], 0.2)
        s["dys"] = [gradients(gen, c["rows"], c["n"], c["dy"], strided)]
    if own:
        import zero_partitioned_mixed_reduce_amd as zpm
        wrap = lambda p: zpm.ZeroPacked.of(p["q"], p["scale"], p["cols"], zpm.ZERO_SCALE_POW2 if p["rule"] == "pow2"
                                           else zpm.ZERO_SCALE_MAX)
        s["own_xs"] = [wrap(p) for p in s.get("xs", [])]
        s["own_w"] = wrap(s["w"]) if "w" in s else None
        empty = lambda rows, cols, rule: zpm.ZeroPacked(rows, cols, rule, device="cuda")
        if c["op"] == "keep":
            s["keep"] = empty(c["rows"], c["cols"], zpm.ZERO_SCALE_POW2 if c["rule"] == "pow2" else zpm.ZERO_SCALE_MAX)
        elif c["op"] == "act":
            s["keep"] = empty(*s["x"].shape, zpm.ZERO_SCALE_POW2)
            s["next"] = empty(c["rows"], c["cols"], zpm.ZERO_SCALE_POW2) if c.get("packed") else None
            s["kind"] = zpm.ZERO_ACT_GELU if c["kind"] == "gelu" else zpm.ZERO_ACT_SILU
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    c = s["case"]
    out = DTYPES[c["dst"]]
    if c["op"] == "keep":
        s["keep"].zero_packed_write(s["x"])
        return dict(x=s["keep"].zero_packed_read(dtype=out), scale=s["keep"].scale)
    if c["op"] == "linear":
        return dict(y=s["own_xs"][0].zero_packed_linear(s["own_w"], bias=s["bias"], dtype=out))
    if c["op"] == "input":
        return dict(dx=s["own_w"].zero_packed_input_grad(s["dys"][0], dtype=out))
    if c["op"] == "weight":
        db = torch.empty(c["n"], dtype=out, device="cuda") if "bias" in c else None
        dw = s["own_xs"][0].zero_packed_weight_grad(s["dys"][0], dtype=out, bias_grad=db)
        if c["steps"] == 2:
            s["own_xs"][1].zero_packed_weight_grad(s["dys"][1], out=dw, bias_grad=db, accumulate=True)
        return dict(dw=dw) if db is None else dict(dw=dw, db=db)
    gated = c.get("gated", False)
    if c.get("packed"):
        s["keep"].zero_packed_act(s["x"], s["kind"], gated=gated, packed=s["next"])
        y = s["next"].zero_packed_read(dtype=out)
    else:
        y = s["keep"].zero_packed_act(s["x"], s["kind"], gated=gated, dtype=out)
    return dict(y=y, dx=s["keep"].zero_packed_act_grad(s["dy"], s["kind"], gated=gated))


# --- plain forms, in 32 bits

def plain_write(x, rule):
    """(q, scale) with one column of scales."""
    x = x.float()
    top = x.abs().amax(1, keepdim=True)
    if rule == "pow2":
        m, e = torch.frexp(top)                        # top = m 2^e: the smallest power of two with top <= 127 of it
        s = torch.ldexp(torch.ones_like(top), (e - torch.where(m <= 127 / 128, 7, 6)).clamp(min=-126))
        q = torch.round(x / s)
    else:
        s = (top / 127).clamp(min=2.0 ** -126)
        q = torch.round(x.double() / s.double()).float().clamp(-127, 127)
    s = torch.where(top == 0, 0.0, s)
    fine = torch.isfinite(top)
    s = torch.where(fine, s, math.nan)
    return torch.where(fine & (top > 0), q, 0.0), s


def plain_values(p):
    return p["q"][:, :p["cols"]].float() * p["scale"][:, None]


def plain_curve(x, kind):
    """f(x) and f'(x): x times the logistic function of h(x)."""
    if kind == "gelu":
        a = 2 * math.sqrt(2 / math.pi)
        g = 1 / (1 + torch.exp(-a * (x + 0.044715 * x * x * x)))
        return x * g, g + x * g * (1 - g) * a * (1 + 3 * 0.044715 * x * x)
    g = 1 / (1 + torch.exp(-x))
    return x * g, g + x * g * (1 - g)


def run_plain(s):
    c = s["case"]
    out = DTYPES[c["dst"]]
    if c["op"] == "keep":
        q, scale = plain_write(s["x"], c["rule"])
        return dict(x=(q * scale).to(out), scale=scale[:, 0])
    if c["op"] == "linear":
        x, w = s["xs"][0], s["w"]
        y = x["q"].float() @ w["q"].float().T
        y = y * x["scale"][:, None] * w["scale"]
        return dict(y=(y if s["bias"] is None else y + s["bias"].float()).to(out))
    if c["op"] == "input":
        return dict(dx=(s["dys"][0].float() @ plain_values(s["w"])).to(out))
    if c["op"] == "weight":
        dw = (s["dys"][0].float().T @ plain_values(s["xs"][0])).to(out)
        db = s["dys"][0].float().sum(0).to(out)
        if c["steps"] == 2:
            dw = (dw.float() + s["dys"][1].float().T @ plain_values(s["xs"][1])).to(out)
            db = (db.float() + s["dys"][1].float().sum(0)).to(out)
        return dict(dw=dw, db=db) if "bias" in c else dict(dw=dw)
    x, dy, n = s["x"].float(), s["dy"].float(), c["cols"]
    q, scale = plain_write(x, "pow2")
    kept = q * scale
    if c.get("gated"):
        y = plain_curve(x[:, :n], c["kind"])[0] * x[:, n:]
        f, df = plain_curve(kept[:, :n], c["kind"])
        dx = torch.cat([dy * kept[:, n:] * df, dy * f], 1)
    else:
        y = plain_curve(x, c["kind"])[0]
        dx = dy * plain_curve(kept, c["kind"])[1]
    if c.get("packed"):
        q, scale = plain_write(y, "pow2")
        y = q * scale
    return dict(y=y.to(out), dx=dx.to(s["dy"].dtype))


def work(case):
    c, m = case, case["rows"]
    out = BYTES[c["dst"]]
    if c["op"] == "keep":
        return dict(bytes=m * c["cols"] * (BYTES[c["src"]] + 1 + 1 + out) + 8 * m, flops=3 * m * c["cols"])
    if c["op"] == "act":
        f, wide = c["cols"], c["cols"] * (2 if c.get("gated") else 1)
        y = 2 + out if c.get("packed") else out
        return dict(bytes=m * (wide * (BYTES[c["src"]] + 2 + out) + f * (y + out)), flops=30 * m * f)
    k, n = c["k"], c["n"]
    if c["op"] == "linear":
        return dict(bytes=m * k + n * k + m * n * out + 4 * (m + n) + (n * BYTES[c["bias"]] if "bias" in c else 0),
                    flops=2 * m * k * n)
    if c["op"] == "input":
        return dict(bytes=m * n * 2 + n * k + m * k * out + 4 * n, flops=2 * m * k * n)
    steps = c["steps"]
    return dict(bytes=steps * (m * n * 2 + m * k + 4 * m) + (2 * steps - 1) * (n * k + (n if "bias" in c else 0)) * out,
                flops=2 * steps * m * k * n)


# --- the definitions in 64 bits

def exact_write(x, rule):
    x = x.double()
    top = x.abs().amax(1)
    s = torch.exp2(torch.ceil(torch.log2(top / 127))) if rule == "pow2" else (top / 127).float().double()
    s = torch.where(top > 0, s.clamp(min=2.0 ** -126), torch.zeros_like(s))
    q = torch.where(top[:, None] > 0, x / s[:, None], torch.zeros_like(x)).round().clamp(-127, 127)
    bad = ~torch.isfinite(top)
    q[bad], s[bad] = 0, math.nan
    return q * s[:, None], s


def exact_f(x, kind):
    t = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return 0.5 * x * (1 + torch.tanh(t)) if kind == "gelu" else x * torch.sigmoid(x)


def exact_slope(x, kind):
    if kind == "silu":
        g = torch.sigmoid(x)
        return g * (1 + x * (1 - g))
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * x * x)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    value = lambda p: p["q"][:, :p["cols"]].double() * p["scale"].double()[:, None]
    if op == "keep":
        x, scale = exact_write(s["x"], c["rule"])
        return dict(x=x, scale=scale)
    if op == "linear":
        y = value(s["xs"][0]) @ value(s["w"]).T
        return dict(y=y if s["bias"] is None else y + s["bias"].double())
    if op == "input":
        return dict(dx=s["dys"][0].double() @ value(s["w"]))
    if op == "weight":
        dw = sum(dy.double().T @ value(x) for x, dy in zip(s["xs"], s["dys"]))
        return dict(dw=dw, db=sum(dy.double().sum(0) for dy in s["dys"])) if "bias" in c else dict(dw=dw)
    kept, _ = exact_write(s["x"], "pow2")
    x, dy, n, kind = s["x"].double(), s["dy"].double(), c["cols"], c["kind"]
    if c.get("gated"):
        y = exact_f(x[:, :n], kind) * x[:, n:]
        dx = torch.cat([dy * kept[:, n:] * exact_slope(kept[:, :n], kind), dy * exact_f(kept[:, :n], kind)], 1)
    else:
        y, dx = exact_f(x, kind), dy * exact_slope(kept, kind)
    # a packed result has no exact value: a step either way at a border
    return dict(y=None if c.get("packed") else y, dx=dx)

"""Measured cases of the gradient-list operators: the norm over many tensors, clipping by it (the whole list by the
global norm, or each tensor by its own), and scaling into another buffer.

A list is what a training program holds after the backward pass: one gradient per parameter, of the shapes of a whole
model or of a few of its layers, in fp16, bf16 or fp32.  Results go into one flat buffer in list order, the layout in
which a rank hands its gradients to the sharded step's reduce.  With `own` false everything is computed by elementary
torch operations; with `own` true by the library's calls."""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GPT2 = dict(model="gpt2", d=1600)                      # the 1.5B-shaped list: 48 layers, vocabulary 50257
LLAMA = dict(model="llama", d=4096, mlp=11008)         # a layer of the 7.5B list
MINI = dict(model="llama", d=256, mlp=688, layers=4, vocab=2000)


def listed():
    return [
        # --- norm: what a run logs every step, and the first half of every clip
        # per-tensor norms of a small model's list: tens of small launches' worth of work, latency counts
        dict(name="norm-mini-bf16", op="norm", src="bf16", each=True, **MINI),
        # the whole 1.5B list, per-tensor norms beside the global one
        dict(name="norm-gpt2-bf16", op="norm", src="bf16", each=True, layers=48, vocab=50257, **GPT2),
        # largest magnitude over a thousand ragged fp16 tensors under a loss scale (an overflow margin)
        dict(name="norm-max-odd-f16", op="norm", kind="max", src="f16", scale=4096.0, model="odd", count=1000,
             total=3_000_017, each=True),
        # --- clip by the global norm
        # low-rank adapters: eight small fp32 tensors, the smallest call
        dict(name="clip-adapters-f32", op="clip", src="f32", dst="bf16", model="odd", count=8, total=20_011),
        # twelve layers whose gradients are views of one flat bf16 buffer, back to back, onto the rank's send buffer
        dict(name="clip-gpt2-12-bf16", op="clip", src="bf16", dst="bf16", packed=True, layers=12, vocab=0, **GPT2),
        # fp32 gradients of two large layers, cast to the 16-bit send buffer
        dict(name="clip-7p5b-2-f32-bf16", op="clip", src="f32", dst="bf16", layers=2, vocab=0, **LLAMA),
        # the whole 1.5B list
        dict(name="clip-gpt2-bf16", op="clip", src="bf16", dst="bf16", layers=48, vocab=50257, **GPT2),
        # gradients of mixed types, some of them column slices of fused matrices, at new addresses every step
        dict(name="clip-mixed-moving", op="clip", src="mix", dst="f32", model="odd", count=150, total=5_000_011,
             strided=True, moving=True),
        # --- clip each tensor by its own norm
        # four layers in fp16 under a loss scale
        dict(name="each-gpt2-4-f16", op="clip", scope="each", src="f16", dst="f16", scale=1024.0, layers=4, vocab=0,
             **GPT2),
        # three thousand small fp32 tensors
        dict(name="each-odd-f32", op="clip", scope="each", src="f32", dst="f32", model="odd", count=3000,
             total=2_500_003),
        # --- scale: unscale and convert into the send buffer, no norm
        # fp32 gradients of the small model into fp16, with the loss scale kept in
        dict(name="scale-mini-f32-f16", op="scale", src="f32", dst="f16", factor=1024.0, **MINI),
        # one 117M-element bf16 gradient (a 1/64 shard of 7.5B) unscaled into fp32
        dict(name="scale-shard-bf16-f32", op="scale", src="bf16", dst="f32", factor=2.0 ** -16, model="odd", count=1,
             total=117_187_520),
    ]


def draw(rng):
    op = rng.choice(["norm", "clip", "clip", "each", "scale"])
    c = dict(op="clip" if op == "each" else op, src=rng.choice(["f16", "bf16", "bf16", "f32", "mix"]))
    if op == "each":
        c["scope"] = "each"
    if c["op"] == "norm":
        c["kind"] = rng.choice(["l2", "l2", "max"])
        c["each"] = rng.random() < 0.7
    else:
        c["dst"] = rng.choice(["f16", "bf16", "bf16", "f32"])
    if c["op"] == "scale":
        c["factor"] = 2.0 ** rng.randint(-12, 6) * rng.choice([1.0, 1.0, 1.25])
    else:
        c["scale"] = 2.0 ** rng.randint(0, 12)
        c["overflow"] = rng.random() < 0.1             # a step that a loss scale too large has spoilt
    if c["op"] == "clip":
        c["slack"] = rng.random() < 0.2                # a norm below the limit: nothing to clip
        c["kind"] = rng.choice(["l2", "l2", "l2", "max"])
    c["packed"] = rng.random() < 0.4
    c["strided"] = rng.random() < 0.3
    c["moving"] = rng.random() < 0.2
    total = int(math.exp(rng.uniform(math.log(2e3), math.log(2e8))))
    if rng.random() < 0.5:
        c.update(model="odd", total=total, count=max(1, min(total // 4, int(math.exp(rng.uniform(0, math.log(2000)))))))
    else:
        d = max(8, int(math.sqrt(total / 12 / rng.randint(1, 24))))
        if rng.random() < 0.5:
            d = (d + 7) // 8 * 8
        kind = rng.choice(["gpt2", "llama"])
        c.update(model=kind, d=d, vocab=rng.choice([0, 0, 3 * d + 1]), layers=max(1, min(48, total // (13 * d * d))))
        if kind == "llama":
            c["mlp"] = 8 * d // 3
    return c


def shapes(case):
    """(rows, cols) of every tensor of the list; rows == 1 for vectors."""
    if case["model"] == "odd":
        n, total = case["count"], case["total"]
        r = random.Random(n * 1000003 + total)
        w = [math.exp(r.uniform(0, 5)) for _ in range(n)]
        s = sum(w)
        out = []
        for x in w:
            k = max(1, int(total * x / s))
            rows = r.choice([1, 1, r.randint(2, 64)]) if n > 1 else 1
            out.append((rows, max(1, k // rows)))
        out[-1] = (1, max(1, total - sum(a * b for a, b in out[:-1])))
        return out
    d, v = case["d"], case["vocab"]
    out = [(v, d)] if v else []
    for _ in range(case["layers"]):
        if case["model"] == "gpt2":
            out += [(1, d), (1, d), (d, 3 * d), (d, d), (1, d), (1, d), (d, 4 * d), (4 * d, d)]
        else:
            m = case["mlp"]
            out += [(1, d), (d, d), (d, d), (d, d), (d, d), (1, d), (m, d), (m, d), (d, m)]
    return out + ([(1, d), (v, d)] if v and case["model"] == "llama" else [])


def elements(case):
    return sum(a * b for a, b in shapes(case))


def make_list(case, seed):
    """The gradients, as views of one allocation per type: back to back (`packed`), or each on a 256-byte boundary as
    an allocator places them; with `strided` every third matrix is a column slice of one that is wider by 24."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kinds = ["bf16", "f32", "bf16", "bf16"] if case["src"] == "mix" else [case["src"]]
    sh = shapes(case)
    place, used = [], dict.fromkeys(kinds, 0)
    for i, (rows, cols) in enumerate(sh):
        k = kinds[i % len(kinds)]
        pitch = cols + 24 if case.get("strided") and rows > 1 and i % 3 == 1 else cols
        at = used[k] if case.get("packed") else (used[k] + 127) // 128 * 128
        place.append((k, at, pitch))
        used[k] = at + rows * pitch
    store = {k: torch.randn(n + 1, generator=gen, dtype=DTYPES[k], device="cuda") for k, n in used.items()}
    r = random.Random(len(sh))
    out = []
    for (rows, cols), (k, at, pitch) in zip(sh, place):
        t = store[k][at:at + rows * pitch].view(rows, pitch)[:, :cols]
        t = t[0] if rows == 1 else t
        # gradients of one model differ by decades from tensor to tensor; some are zero (nothing routed there)
        t.mul_(0.0 if r.random() < 0.02 else case.get("scale", 1.0) * 10.0 ** r.uniform(-4, -2))
        out.append(t)
    if case.get("overflow"):
        t = out[seed % len(out)]
        (t if t.dim() == 1 else t[-1])[-1:].fill_(math.inf)
    return out


def limit(case):
    """The norm allowed: well below what the list has (a global norm of about 2e-3 times the root of its size), or,
    with `slack`, far above it."""
    n = elements(case)
    if case.get("slack"):
        return 1e6
    if case.get("kind", "l2") == "max":
        return 1e-3
    return 2e-4 * math.sqrt(n / (len(shapes(case)) if case.get("scope") == "each" else 1))


def prepare(case, seed):
    grads = make_list(case, seed)
    s = dict(case=case, grads=grads, inv=1.0 / case.get("scale", 1.0), max_norm=limit(case))
    s["sizes"] = torch.tensor([g.numel() for g in grads], device="cuda")
    s["flat"] = None
    if case["op"] != "norm":
        s["flat"] = torch.zeros(elements(case), dtype=DTYPES[case["dst"]], device="cuda")
    if own:
        from zero_partitioned_mixed_reduce_amd import ZeroGrads
        s["handle"] = ZeroGrads(grads, out=s["flat"])
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import zero_partitioned_mixed_reduce_amd as zpm
    c, h = s["case"], s["handle"]
    kind = zpm.ZERO_NORM_MAX if c.get("kind") == "max" else zpm.ZERO_NORM_L2
    if c.get("moving"):
        h.zero_grads_bind(s["grads"], s["flat"])
    if c["op"] == "norm":
        h.zero_grads_norm(kind, s["inv"], per_tensor=c["each"])
        return dict(norm=h.norm, norms=h.norms) if c["each"] else dict(norm=h.norm)
    if c["op"] == "scale":
        h.zero_grads_scale(c["factor"])
        return dict(out=s["flat"])
    if c.get("scope") == "each":
        h.zero_grads_clip_norm(s["max_norm"], kind, s["inv"], zpm.ZERO_CLIP_EACH)
        return dict(norm=h.norm, norms=h.norms, out=s["flat"])
    h.zero_grads_clip_norm(s["max_norm"], kind, s["inv"])
    return dict(norm=h.norm, out=s["flat"])


def size_of(x, kind):
    """Largest magnitude, or sum of squares in 64 bits."""
    return x.abs().max().double() if kind == "max" else (x * x).sum(dtype=torch.float64)


def run_plain(s):
    c, kind = s["case"], s["case"].get("kind", "l2")
    flat = torch.cat([g.reshape(-1) for g in s["grads"]]).float()
    if c["op"] == "scale":
        return dict(out=(flat * c["factor"]).to(DTYPES[c["dst"]]))
    u = flat * s["inv"]
    each = c.get("each") or c.get("scope") == "each"
    r = {}
    if each:
        parts = torch.stack([size_of(x, kind) for x in u.split([g.numel() for g in s["grads"]])])
        total = parts.max() if kind == "max" else parts.sum()
        norms = parts if kind == "max" else parts.sqrt()
        r["norms"] = norms.float()
    else:
        total = size_of(u, kind)
    norm = total if kind == "max" else total.sqrt()
    r["norm"] = norm.float()
    if c["op"] == "norm":
        return r
    # a list with an infinity or NaN in it is carried over as it is: the step that takes it in skips
    fine = torch.isfinite(norm)
    coef = (s["max_norm"] / ((norms if each else norm) + 1e-6)).clamp(max=1.0)
    coef = torch.where(fine, coef, 1.0).float()
    if each:
        coef = torch.repeat_interleave(coef, s["sizes"], output_size=u.numel())
    r["out"] = (u * coef).to(DTYPES[c["dst"]])
    return r


def work(case):
    n, sh = elements(case), shapes(case)
    src = sum(a * b * (4 if case["src"] == "f32" or case["src"] == "mix" and i % 4 == 1 else 2)
              for i, (a, b) in enumerate(sh))
    if case["op"] == "norm":
        return dict(bytes=src + 4 + (4 * len(sh) if case["each"] else 0), flops=3 * n)
    dst = n * (4 if case["dst"] == "f32" else 2)
    return dict(bytes=src + dst, flops=n if case["op"] == "scale" else 5 * n)


def exact(case, seed):
    grads = make_list(case, seed)
    n = sum(g.numel() for g in grads)
    if case["op"] == "scale":
        out, at = torch.empty(n, dtype=torch.float64, device="cuda"), 0
        for g in grads:
            out[at:at + g.numel()] = (g.double() * case["factor"]).flatten()
            at += g.numel()
        return dict(out=out)
    scale, big = case.get("scale", 1.0), case.get("kind") == "max"
    sizes = []
    for g in grads:
        d = g.double().abs() / scale
        sizes.append(float(d.max()) if big else math.sqrt(float(torch.dot(d.flatten(), d.flatten()))))
    whole = max(sizes) if big else math.sqrt(math.fsum(x * x for x in sizes))
    r = dict(norm=torch.tensor(whole, dtype=torch.float64))
    each = case.get("scope") == "each"
    if each or case.get("each"):
        r["norms"] = torch.tensor(sizes, dtype=torch.float64)
    if case["op"] == "norm":
        return r
    top = limit(case)
    r["out"], at = torch.empty(n, dtype=torch.float64, device="cuda"), 0
    for g, x in zip(grads, sizes):
        f = min(1.0, top / ((x if each else whole) + 1e-6)) if math.isfinite(whole) else 1.0
        r["out"][at:at + g.numel()] = (g.double() * (f / scale)).flatten()
        at += g.numel()
    return r

"""The gradient-list operators on the GPU, against their formulas in 64 bits and, given the coefficient the library
reports, to the bit against torch's CPU arithmetic.

Tolerances, by counting roundings (h = 2^-24, half a step of fp32; e = finfo(destination).eps / 2):
  u = fp32(g * inv): exact for powers of two, else h
  norm: fp64 sum of n terms, at most n * 2^-53 (below h / 8 at the sizes here), then fp32: h; with u's h: 2 h (1 + 1/8)
  coefficient: fp64 from the norm (u's h, negligible otherwise), then fp32: 2 h
  result: u (h), coefficient (2 h), the product (h), then the destination (e), plus half its smallest subnormal and,
  where the fp32 product is subnormal, half of fp32's."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from synth import recipes
import zero_partitioned_mixed_reduce_amd as zpm
from tests.gpu_harness import Layout, dev16, host16
from zero_partitioned_mixed_reduce_amd import ZeroError, ZeroGrads, _abi

pytestmark = pytest.mark.gpu
H = 2.0 ** -24
L2, MAX = zpm.ZERO_NORM_L2, zpm.ZERO_NORM_MAX
GLOBAL, EACH = zpm.ZERO_CLIP_GLOBAL, zpm.ZERO_CLIP_EACH
DT = [torch.float16, torch.bfloat16, torch.float32]
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


@pytest.fixture(autouse=True)
def _gpu(need_gpu):
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rand(seed, shape, dtype, sigma=1e-3):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(dtype).cuda()


def exact_sizes(grads, kind, inv):
    out = []
    for g in grads:
        d = g.cpu().double() * inv
        out.append(0.0 if d.numel() == 0 else float(d.abs().max()) if kind == MAX else math.sqrt(math.fsum((d * d).flatten().tolist()))
                   if d.numel() < 20000 else float((d * d).sum().sqrt()))
    return out, (max(out) if kind == MAX else math.sqrt(math.fsum(x * x for x in out)))


def check_norms(h, grads, kind, inv, per_tensor=True):
    sizes, whole = exact_sizes(grads, kind, inv)
    assert abs(float(h.norm) - whole) <= 2.25 * H * whole
    if per_tensor:
        got = h.norms.cpu().double().numpy()
        assert (np.abs(got - np.array(sizes)) <= 2.25 * H * np.array(sizes)).all()
    return sizes, whole


def bits(t):
    t = t.cpu().contiguous()
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16).numpy()


def emulate(g, inv, coef, dtype):
    """fp32(fp32(g * inv) * coef) rounded into dtype, on the CPU; NaNs canonical in 16 bits."""
    x = g.cpu().float() * torch.tensor(inv, dtype=torch.float32) * torch.tensor(coef, dtype=torch.float32)
    y = x.to(dtype)
    if dtype != torch.float32:
        y = torch.where(torch.isnan(x), torch.tensor(float("nan"), dtype=dtype), y)
    return y


def check_result(got, g, inv, c64, dtype, coef32):
    want = g.cpu().double() * inv * c64
    tol = want.abs() * (4 * H + torch.finfo(dtype).eps / 2 * (1 + 4 * H)) + TINY[dtype] / 2 + 2.0 ** -150
    assert ((got.cpu().double() - want).abs() <= tol).all()
    assert (bits(got) == bits(emulate(g, inv, coef32, dtype))).all()


def c_of(norm, max_norm):
    max_norm = float(np.float32(max_norm))            # the C ABI takes it as a float
    return min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0


SIZES = [1, 2, 3, 4, 5, 63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 2047, 4099, 8191, 8192, 8193, 16384, 40003]


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("src", DT)
def test_norm_sizes_and_offsets(src, offset):
    """Every size class, at every alignment of the data; both norms; odd inverse scales."""
    store = rand(1 + offset, sum(SIZES) + 8 * len(SIZES), src)
    grads, at = [], offset
    for n in SIZES:
        grads.append(store[at:at + n])
        at += n + (8 - n % 8) % 8 if offset == 0 else n
    h = ZeroGrads(grads)
    for kind in (L2, MAX):
        for inv in (1.0, 2.0 ** -10, float(np.float32(0.3))):
            h.zero_grads_norm(kind, inv, per_tensor=True)
            check_norms(h, grads, kind, inv)
            assert int(h.found_inf) == 0
    h.close()


@pytest.mark.parametrize("dst", DT)
@pytest.mark.parametrize("src", DT)
def test_clip_types_and_offsets(src, dst):
    """Every pair of types, the destination flat and back to back (so at every alignment against its source), both
    scopes; guard elements around the destination stay."""
    grads = [rand(7 + i, n, src) for i, n in enumerate(SIZES)]
    total = sum(SIZES)
    for lead in (0, 1, 3):
        store = torch.full((total + 64,), 7.0, dtype=dst, device="cuda")
        flat = store[lead:lead + total]
        h = ZeroGrads(grads, out=flat)
        for kind, scope, inv, max_norm in ((L2, GLOBAL, 1.0, 0.05), (L2, EACH, 0.5, 0.01), (MAX, GLOBAL, float(np.float32(1.7)), 1e-3),
                                           (MAX, EACH, 1.0, 1e-3), (L2, GLOBAL, 1.0, 100.0), (L2, GLOBAL, 4.0, 0.0)):
            h.zero_grads_norm(kind, inv, per_tensor=scope == EACH)
            sizes, whole = check_norms(h, grads, kind, inv, scope == EACH)
            h.zero_grads_clip(max_norm, scope)
            q = h.query()
            assert abs(q["norm"] - whole) <= 1.25 * H * whole and not q["found_inf"]
            acc = h.tensor_acc.cpu().double()
            at = 0
            for i, g in enumerate(grads):
                if scope == EACH:
                    nrm = float(acc[i]) if kind == MAX else math.sqrt(float(acc[i]))
                    coef = float(np.float32(c_of(nrm, max_norm)))
                else:
                    coef = q["coef"]
                    assert coef == float(np.float32(c_of(q["norm"], max_norm)))
                check_result(flat[at:at + g.numel()], g, inv, c_of(sizes[i] if scope == EACH else whole, max_norm), dst, coef)
                at += g.numel()
            assert (store[:lead] == 7).all() and (store[lead + total:] == 7).all()
        h.close()


@pytest.mark.parametrize("src,dst", [(a, b) for a in DT for b in DT])
def test_ends_of_parts(src, dst):
    """Runs that end within a vector of an item's or a part's end, at every alignment of source and destination: every
    element is written once, in place too, and none beside them; each norm counts each once."""
    for extra in range(1, 10):
        sizes = [2048 + extra, 4096 + extra, 8192 + extra, 6144 - extra, 16384 + extra]
        for lead in range(8):
            total = sum(sizes)
            base = rand(extra, total + 16, src)
            out = torch.full((total + 32,), 7.0, dtype=dst, device="cuda")
            at = (3 * lead + extra) % 8
            h = ZeroGrads(list(base[lead:lead + total].split(sizes)), out=out[at:at + total])
            h.zero_grads_scale(float(np.float32(0.7)))
            assert (bits(out[at:at + total]) == bits(emulate(base[lead:lead + total], 0.7, 1.0, dst))).all()
            assert (out[:at] == 7).all() and (out[at + total:] == 7).all()
            if src == dst:
                ones = torch.full((total + 16,), 1.0, dtype=src, device="cuda")
                h = ZeroGrads(list(ones[lead:lead + total].split(sizes)))
                h.zero_grads_norm(per_tensor=True)
                assert float(h.acc) == total and h.tensor_acc.tolist() == sizes
                h.zero_grads_scale(3.0)
                assert (ones[lead:lead + total] == 3).all() and (ones[:lead] == 1).all() and (ones[lead + total:] == 1).all()


@pytest.mark.parametrize("dt", DT)
def test_in_place_and_scale(dt):
    grads = [rand(3 + i, n, dt) for i, n in enumerate(SIZES)]
    before = [g.clone() for g in grads]
    h = ZeroGrads(grads)
    h.zero_grads_clip_norm(1e9)                       # nothing to clip: nothing changes
    assert all((bits(a) == bits(b)).all() for a, b in zip(grads, before)) and h.query()["coef"] == 1.0
    h.zero_grads_clip_norm(0.01, inv_loss_scale=0.25)
    c = h.query()["coef"]
    assert c < 1.0
    assert all((bits(a) == bits(emulate(b, 0.25, c, dt))).all() for a, b in zip(grads, before))
    now = [g.clone() for g in grads]
    h.zero_grads_scale(float(np.float32(-3.3)))
    assert all((bits(a) == bits(emulate(b, -3.3, 1.0, dt))).all() for a, b in zip(grads, now))
    h.zero_grads_scale(0.0)
    assert all((a == 0).all() for a in grads)
    h.zero_grads_norm(per_tensor=True)
    assert float(h.norm) == 0.0 and (h.norms == 0).all()
    h.zero_grads_clip(1.0, EACH)                      # a zero norm does not divide by zero
    assert all((a == 0).all() for a in grads)


@pytest.mark.parametrize("src,dst", [(torch.float32, torch.float16), (torch.bfloat16, torch.float32)])
def test_scale_into(src, dst):
    grads = [rand(11 + i, n, src, 10.0) for i, n in enumerate(SIZES)]
    outs = [torch.empty_like(g, dtype=dst) for g in grads]
    h = ZeroGrads(grads, out=outs)
    for f in (1.0, 1024.0, float(np.float32(1 / 3))):
        h.zero_grads_scale(f)
        assert all((bits(o) == bits(emulate(g, f, 1.0, dst))).all() for o, g in zip(outs, grads))


@pytest.mark.parametrize("rows,cols,pitch", [(3, 1, 2), (700, 3, 7), (40, 100, 131), (300, 255, 256), (33, 256, 300),
                                             (50, 257, 301), (9, 4099, 5000), (3, 8192, 8200), (2, 20001, 20003)])
@pytest.mark.parametrize("src,dst", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16),
                                     (torch.float16, torch.float32)])
def test_strided(rows, cols, pitch, src, dst):
    """Column slices, narrow to wide: norms, into a flat buffer, and in place; the columns beside them stay."""
    wide = rand(rows + cols, (rows, pitch), src)
    keep = wide.clone()
    g = wide[:, 1:1 + cols] if pitch > cols else wide[:, :cols]
    flat = torch.empty(rows * cols, dtype=dst, device="cuda")
    h = ZeroGrads([g], out=flat)
    h.zero_grads_norm(L2, 1.0, per_tensor=True)
    _, whole = check_norms(h, [g], L2, 1.0)
    h.zero_grads_clip(whole / 3)
    q = h.query()
    check_result(flat.view(rows, cols), g, 1.0, c_of(whole, whole / 3), dst, q["coef"])
    wide_out = torch.full((rows, pitch + 5), 7.0, dtype=dst, device="cuda")
    h2 = ZeroGrads([g], out=[wide_out[:, 2:2 + cols]])
    h2.zero_grads_scale(0.5)
    assert (bits(wide_out[:, 2:2 + cols]) == bits(emulate(g, 0.5, 1.0, dst))).all()
    assert (wide_out[:, :2] == 7).all() and (wide_out[:, 2 + cols:] == 7).all()
    h3 = ZeroGrads([g])
    h3.zero_grads_clip_norm(whole / 3)
    c = h3.query()["coef"]
    full = emulate(keep, 1.0, 1.0, src).clone()
    off = 1 if pitch > cols else 0
    full[:, off:off + cols] = emulate(keep[:, off:off + cols], 1.0, c, src)
    assert (bits(wide) == bits(full)).all()


def test_in_place_slices_of_one_matrix():
    m = rand(5, (64, 120), torch.bfloat16)
    keep = m.clone()
    h = ZeroGrads([m[:, 40 * i:40 * i + 40] for i in range(3)])
    h.zero_grads_clip_norm(1e-3, scope=EACH)
    acc = h.tensor_acc.cpu()
    for i in range(3):
        c = float(np.float32(c_of(math.sqrt(float(acc[i])), 1e-3)))
        assert (bits(m[:, 40 * i:40 * i + 40]) == bits(emulate(keep[:, 40 * i:40 * i + 40], 1.0, c, torch.bfloat16))).all()
    t = ZeroGrads([m.t()])                            # memory order serves a transposed gradient in place
    t.zero_grads_norm(per_tensor=True)
    check_norms(t, [m], L2, 1.0)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", [L2, MAX])
@pytest.mark.parametrize("where", [0, 5000, 40002, -1])
def test_non_finite(value, kind, where):
    """One inf or NaN anywhere: flagged, not clipped, carried over; the other tensors' norms stand."""
    grads = [rand(21, 40003, torch.bfloat16), rand(22, 700, torch.bfloat16)]
    i = 1 if where < 0 else 0
    grads[i][where] = value
    out = torch.empty(40703, dtype=torch.float16, device="cuda")
    h = ZeroGrads(grads, out=out)
    for scope in (GLOBAL, EACH):
        h.zero_grads_norm(kind, 2.0, per_tensor=True)
        assert int(h.found_inf) == 1
        got = float(h.norm)
        assert math.isnan(got) if math.isnan(value) else got == math.inf
        h.zero_grads_clip(1e-3, scope)
        q = h.query()
        assert q["found_inf"] and q["coef"] == 1.0
        want = torch.cat([emulate(g, 2.0, 1.0, torch.float16) for g in grads])
        assert (bits(out) == bits(want)).all()
        other = exact_sizes([grads[1 - i]], kind, 2.0)[0][0]
        assert abs(float(h.norms[1 - i]) - other) <= 2.25 * H * other
    plain = [g.clone() for g in grads]
    h2 = ZeroGrads(grads)
    h2.zero_grads_clip_norm(1e-3, kind)               # in place: nothing is written
    assert all((bits(a) == bits(b)).all() for a, b in zip(grads, plain))


@pytest.mark.parametrize("src", DT)
def test_nan_encoding(src):
    """NaNs of both signs, with payloads, in vectors and at their ends: 16-bit destinations get the canonical one."""
    g = rand(8, 3001, src)
    raw = g.view(torch.int32 if src == torch.float32 else torch.int16)
    for i, v in ((0, 0x7FC00001), (1, -0x3FFFFF), (500, 0x7F812345), (1501, -1), (3000, 0x7FFFFFFF)):
        if src == torch.float16:
            v = {0: 0x7E01, 1: -0x1FF, 500: 0x7C91, 1501: -1, 3000: 0x7FFF}[i]
        elif src == torch.bfloat16:
            v = {0: 0x7FC1, 1: -0x3F, 500: 0x7F81, 1501: -1, 3000: 0x7FFF}[i]
        raw[i] = v
    assert int(torch.isnan(g).sum()) == 5
    for dst, canonical in ((torch.float16, 0x7E00), (torch.bfloat16, 0x7FC0)):
        for lead in (0, 3):
            out = torch.empty(3004, dtype=dst, device="cuda")[lead:lead + 3001]
            h = ZeroGrads([g], out=out)
            for call in (lambda: h.zero_grads_scale(2.0), lambda: h.zero_grads_clip_norm(1e-3, inv_loss_scale=2.0)):
                out.zero_()
                call()
                assert (bits(out) == bits(emulate(g, 2.0, 1.0, dst))).all()
                assert (bits(out)[[0, 1, 500, 1501, 3000]] == canonical).all()


def test_extremes_of_fp32():
    """Squares beyond fp32's range at both ends; fp16 results beyond its range become infinite."""
    big = torch.full((5000,), 3e38, device="cuda")
    h = ZeroGrads([big], out=torch.empty(5000, dtype=torch.float16, device="cuda"))
    h.zero_grads_norm()
    assert float(h.norm) == math.inf and int(h.found_inf) == 0            # finite in fp64, not in fp32
    assert abs(math.sqrt(float(h.acc)) / (float(big[0]) * math.sqrt(5000)) - 1) < 1e-12
    h.zero_grads_clip(1.0)
    q = h.query()
    # 1 / norm is 4.7e-41, a subnormal fp32 number: rounding to it is off by at most half of 2^-149
    assert abs(q["coef"] - 1.0 / (q["norm"] + 1e-6)) <= 2.0 ** -150
    h.zero_grads_scale(1.0)
    assert (h._out == math.inf).all()
    small = torch.full((3000,), 1e-40, device="cuda")                     # subnormal
    h = ZeroGrads([small])
    h.zero_grads_norm()
    assert abs(math.sqrt(float(h.acc)) / (float(small[0].double()) * math.sqrt(3000)) - 1) < 1e-12


def test_empty_tensors():
    e = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    g = rand(2, 300, torch.float32)
    out = torch.zeros(300, device="cuda")
    h = ZeroGrads([e, g, e], out=out)
    h.zero_grads_clip_norm(1e-3, scope=EACH)
    assert h.norms.cpu()[0] == 0 and h.norms.cpu()[2] == 0
    sizes, _ = exact_sizes([g], L2, 1.0)
    assert abs(float(h.norms[1]) - sizes[0]) <= 2.25 * H * sizes[0]
    only = ZeroGrads([e, e.view(0, 4)])
    for kind in (L2, MAX):
        only.zero_grads_norm(kind, per_tensor=True)
        assert float(only.norm) == 0 and int(only.found_inf) == 0 and (only.norms == 0).all()
        only.zero_grads_clip(1.0, EACH)
        assert only.query() == dict(norm=0.0, found_inf=False, coef=1.0)
    only.zero_grads_scale(2.0)


def ragged(seed, count, top, dtypes=DT):
    r = np.random.RandomState(seed)
    return [rand(seed * 1000 + i, int(r.randint(1, top)), dtypes[r.randint(len(dtypes))]) for i in range(count)]


# beside the many small ones: more than 1024 blocks, and (of one tensor of 1.4e8 elements) runs of items
@pytest.mark.parametrize("count,top", [(1, 3_000_000), (40, 60_000), (900, 3000), (5000, 40), (300, 1100),
                                       (3, 24_000_000), (1, 150_000_000)])
def test_many_tensors_and_same_bits(count, top):
    """Mixed types and sizes: against the formula; the same bits from every repetition, from the two calls and the
    one, and with other work on the GPU."""
    grads = ragged(count, count, top)
    total = sum(g.numel() for g in grads)
    out = torch.empty(total, dtype=torch.bfloat16, device="cuda")
    h = ZeroGrads(grads, out=out)
    h.zero_grads_norm(per_tensor=True)
    sizes, whole = check_norms(h, grads, L2, 1.0)
    first = (h.acc.clone(), h.norms.clone())
    h.zero_grads_clip(whole / 7)
    q = h.query()
    kept = out.clone()
    assert (bits(kept) == bits(torch.cat([emulate(g, 1.0, q["coef"], torch.bfloat16) for g in grads]))).all()
    side, noise = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for k in range(8):
        with torch.cuda.stream(side):
            for _ in range(5):
                noise = (noise @ noise).clamp(-1, 1)
        out.zero_()
        h.zero_grads_clip_norm(whole / 7, per_tensor=True)
        assert torch.equal(h.acc, first[0]) and torch.equal(h.norms, first[1])
        assert (bits(out) == bits(kept)).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", [L2, MAX])
@pytest.mark.parametrize("rows,cols,at,width,lone", [(21000, 4010, 3, 4001, 0), (2300, 30013, 5, 29999, 3), (1, 1, 0, 1, 6000)])
def test_long_lists_of_pieces(kind, rows, cols, at, width, lone):
    """Lists of more than 8192 blocks of work, whose blocks take several items: rows shorter and longer than one,
    odd starts, and tensors of one to four items that begin and end inside a block's share."""
    base = rand(rows, (rows, cols), torch.bfloat16)
    grads = ragged(rows, 40, 30_000) + [base[:, at:at + width]] + ragged(lone, lone, 30_000)
    h = ZeroGrads(grads, out=torch.empty(sum(g.numel() for g in grads), dtype=torch.float32, device="cuda"))
    for _ in range(3):
        h.zero_grads_norm(kind, per_tensor=True)
        check_norms(h, grads, kind, 1.0)
    whole, each = h.acc.clone(), h.norms.clone()
    h.zero_grads_norm(kind)
    assert torch.equal(h.acc, whole)
    grads[-1][(-1,) * grads[-1].dim()] = float("inf")
    h.zero_grads_norm(kind, per_tensor=True)
    assert int(h.found_inf) == 1 and torch.isinf(h.norms[-1]) and torch.equal(h.norms[:-1], each[:-1])


def test_order_of_calls():
    grads = [rand(1, 100, torch.float32)]
    h = ZeroGrads(grads)

    def state(f, *a, **k):
        with pytest.raises(ZeroError) as e:
            f(*a, **k)
        assert e.value.status == _abi.ZERO_ESTATE

    state(h.query)
    state(h.zero_grads_clip, 1.0)
    h.zero_grads_norm()
    state(h.zero_grads_clip, 1.0, EACH)               # no per-tensor norms
    h.zero_grads_clip(1.0)
    state(h.zero_grads_clip, 1.0)                     # the values have changed
    h.zero_grads_norm()
    h.zero_grads_scale(2.0)
    state(h.zero_grads_clip, 1.0)
    h.zero_grads_norm()
    h.zero_grads_bind([grads[0].clone()])
    state(h.zero_grads_clip, 1.0)


def test_refusals_of_calls():
    g = rand(1, 100, torch.float32)
    h = ZeroGrads([g])

    def invalid(f, *a, **k):
        with pytest.raises(ZeroError) as e:
            f(*a, **k)
        assert e.value.status == _abi.ZERO_EINVAL

    for bad in (0.0, -1.0, math.inf, math.nan):
        invalid(h.zero_grads_norm, L2, bad)
        invalid(h.zero_grads_clip_norm, 1.0, inv_loss_scale=bad)
    invalid(h.zero_grads_norm, 3)
    invalid(h.zero_grads_scale, math.inf)
    invalid(h.zero_grads_scale, math.nan)
    h.zero_grads_norm()
    invalid(h.zero_grads_clip, math.nan)
    invalid(h.zero_grads_clip, 1.0, 3)
    invalid(h.zero_grads_clip, 1.0, other_ranks_acc=-1.0)
    before = g.clone()
    twice = ZeroGrads([g, g])                         # a norm may count a tensor twice; writing it twice may not
    twice.zero_grads_norm()
    assert abs(float(twice.norm) - math.sqrt(2) * float(g.double().norm())) <= 3 * H * float(twice.norm)
    invalid(twice.zero_grads_clip, 1.0)
    invalid(twice.zero_grads_clip_norm, 1.0)
    invalid(twice.zero_grads_scale, 2.0)
    assert torch.equal(g, before)
    invalid(ZeroGrads, [g], out=[g.view(torch.int32).view(torch.float32)[:100].view(torch.float16)[:100]])
    with pytest.raises(ValueError):
        ZeroGrads([g, torch.zeros(3)])
    with pytest.raises(ValueError):
        ZeroGrads([g], out=torch.zeros(100))
    with pytest.raises(ValueError):
        ZeroGrads([g], out=torch.zeros(99, device="cuda"))
    with pytest.raises(ValueError):
        ZeroGrads([g], out=[])
    with pytest.raises(ValueError, match="tensor 1"):
        ZeroGrads([g, None])
    for bad in ([], [g, g], [g[:99]], [g.half()], [torch.zeros(100)]):
        with pytest.raises((ValueError, IndexError)):
            h.zero_grads_bind(bad)
    with pytest.raises(ValueError):
        h.zero_grads_bind([g], out=[torch.zeros(100, device="cuda")])


@pytest.mark.parametrize("count", [3, 600])
def test_bind(count):
    """New addresses with other alignments, more tensors than one bind launch carries, sources and destinations."""
    def make(seed):
        r = np.random.RandomState(seed)
        return [rand(seed + i, 30000 if i == 1 else 10 + i % 2000, DT[i % 3])[: 10 + i % 2000 if i != 1 else 30000] for i in range(count)]

    grads = make(1)
    total = sum(g.numel() for g in grads)
    out = torch.empty(total, device="cuda")
    h = ZeroGrads(grads, out=out)
    h.zero_grads_clip_norm(0.01)
    for seed in (2, 3):
        store = {d: torch.empty(sum(g.numel() for g in grads) + 16, dtype=d, device="cuda") for d in DT}
        moved, at = [], dict.fromkeys(DT, seed)
        for g in make(100 * seed):
            v = store[g.dtype][at[g.dtype]:at[g.dtype] + g.numel()]
            v.copy_(g)
            at[g.dtype] += g.numel()
            moved.append(v)
        big = torch.full((total + 9,), 7.0, device="cuda")
        h.zero_grads_bind(moved, big[seed:seed + total])
        old = out.clone()
        h.zero_grads_norm(per_tensor=True)
        check_norms(h, moved, L2, 1.0)
        h.zero_grads_clip(0.01)
        want = torch.cat([emulate(g, 1.0, h.query()["coef"], torch.float32) for g in moved])
        assert (bits(big[seed:seed + total]) == bits(want)).all()
        assert (big[:seed] == 7).all() and (big[seed + total:] == 7).all() and torch.equal(out, old)
    # refused addresses leave the old ones
    with pytest.raises(ZeroError) as e:
        h.zero_grads_bind([big[seed:seed + g.numel()] if g.dtype == torch.float32 and g.numel() > 10 else g for g in moved],
                          big[seed:seed + total])
    assert e.value.status == _abi.ZERO_EINVAL
    h.zero_grads_scale(1.0)
    assert (bits(big[seed:seed + total]) == bits(torch.cat([emulate(g, 1.0, 1.0, torch.float32) for g in moved]))).all()


def test_bind_with_empty_tensors():
    """Empty tensors have no address of their own, planned and bound: flat, per-tensor and in-place destinations."""
    def make(v):
        return [torch.full((300,), v, device="cuda"), torch.empty(0, device="cuda"), torch.full((2000,), v, device="cuda"),
                torch.empty((4, 0), device="cuda")]

    for mode in ("flat", "list", "in place"):
        def out():
            return (torch.zeros(2300, device="cuda") if mode == "flat" else None if mode == "in place"
                    else [torch.zeros_like(g) for g in make(0.0)])
        h = ZeroGrads(make(1.0), out=out())
        h.zero_grads_scale(2.0)
        grads, o = make(3.0), out()
        h.zero_grads_bind(grads, *([] if o is None else [o]))
        h.zero_grads_norm(per_tensor=True)
        assert h.tensor_acc.tolist() == [2700.0, 0.0, 18000.0, 0.0]
        h.zero_grads_scale(2.0)
        got = grads if o is None else o if isinstance(o, list) else [o]
        assert all((t == 6.0).all() for t in got)


@pytest.mark.parametrize("dst", DT)
@pytest.mark.parametrize("src", DT)
def test_all_magnitudes(src, dst):
    """Random bit patterns, subnormals, infinities and NaNs among them: every product and conversion rounds as on the
    CPU."""
    n = 70_001
    g = torch.Generator().manual_seed(5)
    if src == torch.float32:
        raw = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g).to(torch.int32)
    else:
        raw = torch.randint(-2 ** 15, 2 ** 15, (n,), generator=g).to(torch.int16)
    x = raw.view(src).cuda()
    assert int(torch.isnan(x).sum()) > 100
    out = torch.empty(n + 1, dtype=dst, device="cuda")[1:]
    h = ZeroGrads([x], out=out)
    for f in (1.0, 0.7, 2.0 ** -20, 2.0 ** 30):
        h.zero_grads_scale(f)
        want = emulate(x, f, 1.0, dst)
        nan = torch.isnan(want).numpy()
        same = bits(out) == bits(want)
        assert (same | (nan if dst == torch.float32 else False)).all() and torch.isnan(out.cpu()).numpy()[nan].all()


def test_exchange_on_the_host_and_on_the_device():
    """Two ranks' halves of a list clip like the whole list, with the statistics exchanged either way."""
    grads = ragged(4, 20, 9000, [torch.float32])
    whole = ZeroGrads(grads, out=[torch.empty_like(g) for g in grads])
    for kind, limit in ((L2, 0.02), (MAX, 1e-3)):
        whole.zero_grads_clip_norm(limit, kind)
        ref = whole.query()
        for on_device in (False, True):
            a, b = [ZeroGrads(part, out=[torch.empty_like(g) for g in part]) for part in (grads[:9], grads[9:])]
            for h in (a, b):
                h.zero_grads_norm(kind, per_tensor=True)
            if on_device:
                joint = a.acc + b.acc if kind == L2 else torch.maximum(a.acc, b.acc)
                a.acc.copy_(joint)
                b.acc.copy_(joint)
                for h in (a, b):
                    h.zero_grads_clip(limit)
            else:
                sa, sb = float(a.acc), float(b.acc)
                a.zero_grads_clip(limit, other_ranks_acc=sb)
                b.zero_grads_clip(limit, other_ranks_acc=sa)
            for h, part in ((a, grads[:9]), (b, grads[9:])):
                q = h.query()
                assert abs(q["norm"] - ref["norm"]) <= 1e-12 * ref["norm"] and not q["found_inf"]
                assert abs(float(h.norm) - ref["norm"]) <= H * ref["norm"]
                for o, g in zip(h._out, part):
                    assert (bits(o) == bits(emulate(g, 1.0, q["coef"], torch.float32))).all()
    # tensors cut across the ranks: their sums are exchanged as well, and each is clipped by its whole norm
    for kind, limit in ((L2, 5e-3), (MAX, 1e-3)):
        outs = [torch.empty_like(g) for g in grads]
        one = ZeroGrads(grads, out=outs)
        one.zero_grads_clip_norm(limit, kind, scope=EACH)
        halves = [[g[: g.numel() // 2] for g in grads], [g[g.numel() // 2:] for g in grads]]
        a, b = [ZeroGrads(part, out=[torch.empty_like(g) for g in part]) for part in halves]
        for h in (a, b):
            h.zero_grads_norm(kind, per_tensor=True)
        for x, y in ((a.acc, b.acc), (a.tensor_acc, b.tensor_acc)):
            joint = x + y if kind == L2 else torch.maximum(x, y)
            x.copy_(joint)
            y.copy_(joint)
        for h in (a, b):
            h.zero_grads_clip(limit, EACH)
        for o, x, y in zip(outs, a._out, b._out):
            # the coefficients may differ in fp64's last places and so by one step of fp32
            assert ((torch.cat([x, y]).double() - o.double()).abs() <= 4 * H * o.double().abs()).all()
        a.zero_grads_norm(kind, per_tensor=True)
        a.zero_grads_clip(1e-6, EACH, other_ranks_found_inf=True)
        assert all(torch.equal(o, g) for o, g in zip(a._out, halves[0])) and a.query()["found_inf"]
    a = ZeroGrads(grads, out=[torch.empty_like(g) for g in grads])
    # another rank's flag, or a non-finite sum of its, stops the clip here
    for kw in (dict(other_ranks_found_inf=True), dict(other_ranks_acc=math.inf), dict(other_ranks_acc=math.nan)):
        for kind in (L2, MAX):
            a.zero_grads_norm(kind)
            a.zero_grads_clip(1e-6, **kw)
            q = a.query()
            assert q["found_inf"] and q["coef"] == 1.0
            assert all(torch.equal(o, g) for o, g in zip(a._out, grads))


@pytest.mark.parametrize("scope", [GLOBAL, EACH])
def test_captured(scope):
    """Captured once, replayed with other values, eager work of the same handle and others between the replays; every
    replay equals the eager result to the bit.  Two graphs of two handles."""
    def make(seed):
        return [rand(seed + i, n, torch.bfloat16) for i, n in enumerate((5000, 70000, 3, 900, 12345))]

    grads = make(1)
    total = sum(g.numel() for g in grads)
    out, out2 = torch.empty(total, dtype=torch.float16, device="cuda"), torch.empty(total, device="cuda")
    h, h2 = ZeroGrads(grads, out=out), ZeroGrads(grads, out=out2)
    h.zero_grads_clip_norm(0.01, scope=scope)
    h2.zero_grads_clip_norm(0.02, scope=scope)
    torch.cuda.synchronize()
    graphs = []
    for hh, limit in ((h, 0.01), (h2, 0.02)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hh.zero_grads_bind(grads, out if hh is h else out2)
            hh.zero_grads_norm(per_tensor=True)
            hh.zero_grads_clip(limit, scope)
        graphs.append(g)
    check = ZeroGrads(grads, out=torch.empty(total, dtype=torch.float16, device="cuda"))
    for step in range(5):
        for g, v in zip(grads, make(100 * step)):
            g.copy_(v)
        if step == 3:
            grads[1][777] = math.inf
        out.zero_()
        out2.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert h.query()["found_inf"] == (step == 3)
        a, n = out.clone(), h.norms.clone()
        check.zero_grads_clip_norm(0.01, scope=scope)
        assert (bits(a) == bits(check._out)).all()
        assert torch.equal(check.norms, n) if scope == EACH else True
        c2 = out2.clone()
        h2.zero_grads_clip_norm(0.02, scope=scope)
        assert (bits(c2) == bits(out2)).all()


def test_other_stream():
    grads = ragged(9, 30, 20000)
    h = ZeroGrads(grads, out=[torch.zeros_like(g) for g in grads])
    h.zero_grads_clip_norm(0.01)
    ref = [o.clone() for o in h._out]
    s = torch.cuda.Stream()
    for o in h._out:
        o.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h.zero_grads_clip_norm(0.01)
        q = h.query()
    assert all((bits(a) == bits(b)).all() for a, b in zip(ref, h._out)) and not q["found_inf"]


def test_two_handles_at_once():
    """Two handles on two streams, each many times with nothing between: neither disturbs the other."""
    lists = [ragged(k, 60, 40000) for k in (31, 32)]
    hs = [ZeroGrads(g, out=torch.empty(sum(t.numel() for t in g), dtype=torch.bfloat16, device="cuda")) for g in lists]
    refs = []
    for h in hs:
        h.zero_grads_clip_norm(0.01, per_tensor=True)
        refs.append((h._out.clone(), h.acc.clone(), h.norms.clone()))
        h._out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(50):
        for h, s in zip(hs, streams):
            with torch.cuda.stream(s):
                h.zero_grads_clip_norm(0.01, per_tensor=True)
    torch.cuda.synchronize()
    for h, (o, acc, norms) in zip(hs, refs):
        assert (bits(h._out) == bits(o)).all() and torch.equal(h.acc, acc) and torch.equal(h.norms, norms)


def test_closed_handle_and_kept_tensors():
    h = ZeroGrads((torch.ones(5000, device="cuda") for _ in range(3)),   # only the handle keeps them
                  out=(torch.zeros(5000, device="cuda") for _ in range(3)))
    rest = [torch.full((5000,), 5.0, device="cuda") for _ in range(8)]
    h.zero_grads_norm()
    assert float(h.acc) == 15000.0
    h.zero_grads_scale(2.0)
    assert all((o == 2).all() for o in h._out) and all((r == 5).all() for r in rest)
    h.close()
    h.close()
    for call in (h.zero_grads_norm, h.query, lambda: h.zero_grads_scale(1.0), lambda: h.zero_grads_clip_norm(1.0)):
        with pytest.raises(ZeroError) as e:
            call()
        assert e.value.status == _abi.ZERO_EINVAL


def test_beyond_32_bits():
    """A tensor of more than 2^31 elements with its spikes beyond element 2^31, and rows more than 2^32 bytes apart."""
    n = (1 << 31) + 12_345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 31) - 1, 1 << 31, (1 << 31) + 8191, n - 1]
    for k, i in enumerate(at):
        g[i] = 2.0 ** k
    small = torch.full((3,), 2.0, device="cuda")
    out = torch.empty(n, dtype=torch.float16, device="cuda")
    h = ZeroGrads([small, g], out=[torch.empty_like(small), out])
    h.zero_grads_norm(per_tensor=True)
    want = math.fsum(4.0 ** k for k in range(5))
    assert float(h.acc) == want + 12.0 and float(h.tensor_acc[1]) == want
    h.zero_grads_clip(math.sqrt(want + 12.0) / 2)
    c = h.query()["coef"]
    assert abs(c - 0.5) < 1e-6
    for k, i in enumerate(at):
        assert float(out[i]) == float(np.float16(np.float32(2.0 ** k) * np.float32(c)))
    assert int((out != 0).sum()) == 5
    h.close()
    del out
    rows = g.as_strided((2, 9000), ((1 << 31) + 100, 1))
    rows.fill_(0.5)
    h = ZeroGrads([rows])
    h.zero_grads_clip_norm(1.0)
    assert abs(h.query()["norm"] - math.sqrt(0.25 * 18000)) < 1e-9
    assert float(rows[1, 8999]) == float(torch.tensor(0.5 * h.query()["coef"]).bfloat16())
    assert float(g[9000]) == 0.0 and float(g[(1 << 31) + 99]) == 0.0


def test_list_to_sharded_step():
    """As they are used: two ranks' lists of fp32 and strided bf16 gradients are clipped into flat 16-bit send buffers,
    the sharded step reduces them and updates; against the oracle's step on the same clipped buffers."""
    w = recipes.ragged_mini(2)
    shapes = [n for n in w.numel]
    psi, nd, dtype = w.psi, 2, oracle.BF16
    master = synth.normal_f32(psi, w.seed, synth.stream_id(synth.MASTER), 0, w.master_sigma)
    p16 = synth.normal_16(psi, dtype, w.seed, synth.stream_id(synth.MASTER), 0, w.master_sigma)
    sent, host = [], []
    for q in range(nd):
        grads = []
        for i, n in enumerate(shapes):
            if n % 256 == 0 and n > 256 and i % 2:
                grads.append(rand(q * 1000 + i, (n // 256, 300), torch.bfloat16, 1e-2)[:, :256])
            else:
                grads.append(rand(q * 1000 + i, n, torch.float32, 1e-2))
        buf = torch.empty(psi, dtype=torch.bfloat16, device="cuda")
        h = ZeroGrads(grads, out=buf)
        h.zero_grads_clip_norm(0.5, inv_loss_scale=2.0 ** -3)
        c = h.query()["coef"]
        assert c < 1.0
        expect = torch.cat([emulate(g, 2.0 ** -3, c, torch.bfloat16).flatten() for g in grads])
        assert (bits(buf) == bits(expect)).all()
        sent.append(buf)
        host.append(bits(expect).view(np.uint16))
    hp = oracle.HParams(1e-3, 0.9, 0.999, 1e-8, 0.01)
    psi_, S, b, valid = oracle.plan(w.numel, nd, 1)
    locs = [oracle.grad_stats(dtype, [g[q * S:q * S + oracle.plan(w.numel, nd, q)[3]] for g in host], 1.0) for q in range(nd)]
    glob = locs[0][2] + locs[1][2]
    st = oracle.RankState(dtype, p16[b:b + valid], master[b:b + valid])
    clip, _ = oracle.clip_coef(glob, w.max_norm)
    oracle.adam(False, locs[1][0], clip, hp, st.counters, st.w, st.m, st.v)
    oracle.cast(dtype, st.w, st.p16)
    params = dev16(p16)
    s = zpm.ZeroShard(w.numel, nd, 1, dtype, params, master_init=torch.from_numpy(master[b:b + valid]).cuda(), with_red=True)
    s.zero_reduce_grads(sent, 1.0)
    s.zero_check_overflow(False)
    s.zero_grad_norm_global(glob, w.max_norm)
    s.zero_adam_step(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    for name, exp in (("master", st.w), ("m", st.m), ("v", st.v)):
        assert (s.export(name).cpu().numpy().view(np.uint32) == exp.view(np.uint32)).all(), name
    assert (host16(params)[b:b + valid] == st.p16).all()
    # an overflow in one rank's list reaches the step, which skips
    grads[-2][5] = math.inf                           # the final norm's gradient, in rank 1's half
    h.zero_grads_clip_norm(0.5, inv_loss_scale=2.0 ** -3)
    assert h.query()["found_inf"] and int(torch.isinf(sent[1]).sum()) == 1
    s.zero_reduce_grads(sent, 1.0)
    assert s.zero_check_overflow(False, sync=True)

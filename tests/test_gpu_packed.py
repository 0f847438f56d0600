"""GPU tests of the packed-row operators against their definitions in 64 bits, and to the bit where the definition fixes
the result."""
import math

import pytest
import torch

import zero_partitioned_mixed_reduce_amd as zpm
from zero_partitioned_mixed_reduce_amd.packed import matrix

pytestmark = pytest.mark.gpu

POW2, MAX, GELU, SILU = zpm.ZERO_SCALE_POW2, zpm.ZERO_SCALE_MAX, zpm.ZERO_ACT_GELU, zpm.ZERO_ACT_SILU
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def half_step(t):
    """Most that rounding to nearest moves a value of magnitude 1."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of the type's smallest numbers."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def packed_of(x, rule):
    """(q, scale) of x by the definition, in 64 bits."""
    d = x.double()
    top = d.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    if rule == POW2:
        e = torch.ceil(torch.log2(top / 127))
        # log2 next to a whole number: settle it by the definition itself
        e = torch.where(top <= 127 * torch.exp2(e - 1), e - 1, torch.where(top > 127 * torch.exp2(e), e + 1, e))
        s = torch.exp2(e.clamp(min=-126))
    else:
        # in 64 bits and then in 32 is rounded once: a quotient by 127 that ends at 25 bits would be one of 24 times 127
        s = (top / torch.full_like(top, 127)).float().double().clamp(min=2.0 ** -126)
    q = torch.round(d / s[:, None]).clamp(-127, 127)
    q[top == 0], s[top == 0] = 0, 0
    bad = ~torch.isfinite(top)
    q[bad], s[bad] = 0, math.nan
    return q.to(torch.int8), s.float()


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0)) \
        and torch.equal(a.isnan(), b.isnan())


def strided(t, extra=24, lead=0):
    """t's values as columns of a wider matrix that is full of NaN (or 111) around them."""
    fill = 111 if t.dtype == torch.int8 else math.nan
    big = torch.full((t.shape[0], t.shape[1] + extra + lead), fill, dtype=t.dtype, device=t.device)
    v = big[:, lead:lead + t.shape[1]]
    v.copy_(t)
    return v, big


def around(v, big, lead=0):
    """What lies around v in big, to see that nothing was written there."""
    return torch.cat([big[:, :lead], big[:, lead + v.shape[1]:]], 1)


def values(p):
    return p.q.double() * p.scale.double()[:, None]


def random_packed(rows, cols, seed, rule=POW2, scales=None, nan_rows=()):
    """Packed rows with every q from -127 to 127 and scales that are powers of two (or the given ones)."""
    g = gen(seed)
    pitch = max(16, (cols + 15) // 16 * 16)
    q = torch.zeros(rows, pitch, dtype=torch.int8, device=DEV)
    q[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g, device=DEV, dtype=torch.int8)
    s = torch.exp2(torch.randint(-3, 3, (rows,), generator=g, device=DEV).float()) if scales is None else scales
    return zpm.ZeroPacked.of(q, s, cols, rule)


# --- writing and reading

ROWS_COLS = [(1, 1), (3, 7), (5, 8), (4, 15), (4, 16), (7, 17), (2, 512), (3, 513), (5, 1031), (3, 2048), (2, 2049), (3, 4104),
             (2, 8192), (1, 8193), (2, 11008), (2, 16385), (1, 32768), (2, 32769), (1, 50257), (300, 24), (1000, 100)]


@pytest.mark.parametrize("rule", [POW2, MAX])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows, cols", ROWS_COLS)
def test_write_read(rows, cols, dtype, rule):
    g = gen(rows * 1000 + cols)
    x = torch.randn(rows, cols, generator=g, device=DEV) * torch.exp(2 * torch.randn(rows, 1, generator=g, device=DEV))
    x = x.to(dtype)
    if rows > 2:
        x[1] = 0
    p = zpm.ZeroPacked(rows, cols, rule)
    p._q.fill_(99)
    p.zero_packed_write(x)
    q, s = packed_of(x, rule)
    assert same_bits(p.scale, s)
    assert torch.equal(p.q, q)
    assert not p._q[:, cols:].any()                    # zeros behind the columns
    for out in (F16, BF16, F32):
        v = p.zero_packed_read(dtype=out)
        assert same_bits(v, (q.float() * s[:, None]).to(out))     # one product in fp32, rounded once more
    if rule == POW2:
        assert torch.equal(p.zero_packed_read().double(), values(p))    # exact in bf16


@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows, cols", [(5, 7), (6, 1000), (3, 4099), (2, 33001)])
def test_write_read_strided(rows, cols, dtype, lead):
    x = torch.randn(rows, cols, generator=gen(cols), device=DEV).to(dtype)
    v, _ = strided(x, 5, lead)
    p = zpm.ZeroPacked(rows, cols).zero_packed_write(v)
    assert torch.equal(p.q, packed_of(x, POW2)[0])
    out, big = strided(torch.zeros(rows, cols, dtype=dtype, device=DEV), 5, lead)
    p.zero_packed_read(out=out)
    assert torch.equal(out, (p.q.float() * p.scale[:, None]).to(dtype))
    assert around(out, big, lead).isnan().all()


@pytest.mark.parametrize("rule", [POW2, MAX])
@pytest.mark.parametrize("cols", [40, 3000, 40000])
def test_write_extremes(cols, rule):
    """Rows next to the borders: powers of two times 127 and their neighbours, exact halves, subnormal and huge rows."""
    tops = []
    for e in (-149, -140, -130, -126, -120, -20, 0, 1, 60, 120):
        for f in (1.0, 127 / 64, 1.9844, 1.99, 63.5 / 64 * 2 - 1):
            tops.append(min(f * 2.0 ** e, 3.4e38))
    b = 127 * 2.0 ** -3
    tops += [b, b * (1 + 2.0 ** -23), b * (1 - 2.0 ** -23), 3.4028234663852886e38, 2.0 ** -149]
    x = torch.empty(len(tops), cols, device=DEV)
    g = gen(cols)
    for i, t in enumerate(tops):
        # halves of a step among other values
        x[i] = torch.randint(-254, 255, (cols,), generator=g, device=DEV) / 254 * t
        x[i, 0] = t
    p = zpm.ZeroPacked(*x.shape, rule).zero_packed_write(x)
    q, s = packed_of(x, rule)
    assert same_bits(p.scale, s)
    assert torch.equal(p.q, q)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("cols", [9, 700, 5000, 33000])
def test_rows_with_infinities(cols, bad):
    x = torch.randn(5, cols, generator=gen(cols), device=DEV).bfloat16()
    x[2, cols // 2] = bad
    x[4, -1] = bad
    for rule in (POW2, MAX):
        p = zpm.ZeroPacked(5, cols, rule).zero_packed_write(x)
        assert p.scale.isnan().tolist() == [False, False, True, False, True]
        assert not p.q[[2, 4]].any()
        v = p.zero_packed_read(dtype=F16)
        assert v[[2, 4]].isnan().all() and v[[0, 1, 3]].isfinite().all()
        assert (v[2].view(torch.int16) == 0x7E00).all()            # the canonical quiet NaN
        assert (p.zero_packed_read()[4].view(torch.int16) == 0x7FC0).all()


@pytest.mark.parametrize("rows, cols", [((1 << 22) + 9, 24), ((1 << 20) + 3, 2056), ((1 << 20) + 3, 2051)])
def test_more_rows_than_a_launch_has_blocks(rows, cols):
    """Blocks go on to further rows, where a row's threads are a wave and where they are a block."""
    x = torch.randn(rows, cols, generator=gen(cols), device=DEV, dtype=BF16)
    x[-1] = 0
    x[-2, 3] = math.inf
    p = zpm.ZeroPacked(rows, cols).zero_packed_write(x)
    blocks = 1 << 20
    at = torch.cat([torch.arange(a, a + 16, device=DEV) for a in (0, blocks - 8, rows // 2, rows - 16)])
    at = at[at < rows]
    q, s = packed_of(x[at], POW2)
    assert same_bits(p.scale[at], s) and torch.equal(p.q[at], q)
    y = p.zero_packed_read()
    assert y[-2].isnan().all() and not y[-1].any() and y[:-2].isfinite().all()
    assert torch.equal(y[at].nan_to_num(), (p.q[at].float() * p.scale[at, None]).to(BF16).nan_to_num())
    # the packed rows of the whole matrix agree with those of pieces that one launch covers
    del y
    a = rows - (1 << 18)
    r = zpm.ZeroPacked(1 << 18, cols).zero_packed_write(x[a:])
    assert torch.equal(r._q, p._q[a:]) and same_bits(r.scale, p.scale[a:])


def test_no_rows_and_no_columns():
    for rows, cols in ((0, 40), (7, 0), (0, 0)):
        p = zpm.ZeroPacked(rows, cols)
        p.scale.fill_(5)
        p.zero_packed_write(torch.empty(rows, cols, device=DEV))
        assert not p.scale.any()
        assert p.zero_packed_read().shape == (rows, cols)


# --- the linear layer

def linear_expected(x, w, bias, dtype):
    acc = x.q.double() @ w.q.double().T                # whole numbers, exact
    y = acc.float() * x.scale[:, None] * w.scale
    return (y if bias is None else y + bias.float()).to(dtype)


SHAPES = [(1, 1, 1), (1, 16, 16), (2, 33, 5), (3, 129, 257), (16, 64, 40), (17, 100, 129), (31, 1600, 70), (64, 250, 129),
          (65, 128, 128), (127, 127, 127), (128, 256, 128), (129, 384, 255), (200, 1043, 333), (257, 700, 513), (1, 4096, 1000),
          (5, 6400, 1600), (24, 11008, 300), (500, 64, 1024), (64, 20000, 64), (3, 131056, 17), (1030, 48, 2060)]


@pytest.mark.parametrize("m, k, n", SHAPES)
def test_linear(m, k, n):
    x, w = random_packed(m, k, 1), random_packed(n, k, 2, MAX, torch.rand(n, generator=gen(3), device=DEV) + 0.01)
    for dtype, bias in ((BF16, None), (F32, F32), (F16, BF16)):
        b = None if bias is None else torch.randn(n, generator=gen(4), device=DEV).to(bias) * 100
        if dtype == F16:                               # within its range
            x.scale.mul_(2.0 ** -12)
        y = x.zero_packed_linear(w, bias=b, dtype=dtype)
        assert same_bits(y, linear_expected(x, w, b, dtype)), (dtype, bias)


@pytest.mark.parametrize("m, k, n", [(1, 70, 9), (40, 333, 131), (300, 200, 270)])
def test_linear_strided(m, k, n):
    """x and w as columns of wider packed rows (on 16-byte boundaries), y as columns of a wider matrix."""
    def inside(p):
        wide = torch.full((p.rows, p._q.shape[1] + 48), 77, dtype=torch.int8, device=DEV)
        wide[:, 16:16 + p._q.shape[1]] = p._q
        return zpm.ZeroPacked.of(wide[:, 16:16 + p._q.shape[1]], p.scale, p.cols, p.rule)
    x, w = random_packed(m, k, 1), random_packed(n, k, 2)
    for lead in (0, 1, 4):
        y, big = strided(torch.zeros(m, n, dtype=BF16, device=DEV), 7, lead)
        inside(x).zero_packed_linear(inside(w), out=y)
        assert torch.equal(y, linear_expected(x, w, None, BF16))
        assert around(y, big, lead).isnan().all()


@pytest.mark.parametrize("m", [1, 20, 130])
def test_linear_nan_and_empty_rows(m):
    x, w = random_packed(m, 90, 1), random_packed(50, 90, 2)
    x.scale[m - 1] = math.nan
    w.scale[7] = math.nan
    w.scale[9] = 0
    w._q[9] = 0
    y = x.zero_packed_linear(w, dtype=F32)
    assert same_bits(y, linear_expected(x, w, None, F32))
    assert y[m - 1].isnan().all() and y[:, 7].isnan().all() and (m == 1 or not y[:m - 1, 9].any())


def test_linear_without_input_features():
    x, w, b = zpm.ZeroPacked(5, 0), zpm.ZeroPacked(9, 0), torch.arange(9, device=DEV, dtype=F32)
    x.scale.fill_(1), w.scale.fill_(1)
    assert torch.equal(x.zero_packed_linear(w, bias=b, dtype=F32), b.expand(5, 9))
    assert not x.zero_packed_linear(w).any()
    x = zpm.ZeroPacked(300, 0)
    x.scale.fill_(1)
    assert torch.equal(x.zero_packed_linear(w, bias=b, dtype=F32), b.expand(300, 9))


def test_linear_far_offsets():
    """Weights of more than 2^31 bytes, and a result whose elements pass 2^31."""
    n, k = 70016, 32768
    w = random_packed(n, k, 2)
    for m in (2, 70):
        x = random_packed(m, k, 1)
        y = x.zero_packed_linear(w, dtype=F32)
        at = torch.tensor([0, 1, 40000, 65535, 65536, 65537, n - 2, n - 1], device=DEV)
        few = zpm.ZeroPacked.of(w._q[at].contiguous(), w.scale[at].contiguous(), k)
        assert same_bits(y[:, at].contiguous(), linear_expected(x, few, None, F32))
    del w, y
    m, n, k = 50000, 50000, 16
    x, w = random_packed(m, k, 1), random_packed(n, k, 2)
    y = x.zero_packed_linear(w)
    for r in (0, 42949, 42950, m - 1):                 # around element 2^31
        assert torch.equal(y[r:r + 1], linear_expected(x[r:r + 1], w, None, BF16))


@pytest.mark.parametrize("m", [1, 16, 17, 33, 64])
@pytest.mark.parametrize("k, n", [(33, 2050), (1100, 2048), (4096, 8191), (700, 8192), (1024, 9001)])
def test_linear_of_few_tokens_into_many_channels(m, k, n):
    x, w = random_packed(m, k, 1), random_packed(n, k, 2, MAX, torch.rand(n, generator=gen(3), device=DEV) + 0.01)
    assert same_bits(x.zero_packed_linear(w, bias=w.scale, dtype=F32), linear_expected(x, w, w.scale, F32))
    y, big = strided(torch.zeros(m, n, dtype=BF16, device=DEV), 7, 1)
    x.zero_packed_linear(w, out=y)
    assert torch.equal(y, linear_expected(x, w, None, BF16)) and around(y, big, 1).isnan().all()


@pytest.mark.parametrize("m, n", [(3, 17), (64, 40), (130, 129)])
def test_linear_of_the_largest_sums(m, n):
    """131056 products of the largest bytes there are, of one sign and of both: sums next to 2^31."""
    k = 131056
    x, w = random_packed(m, k, 1), random_packed(n, k, 2)
    x._q.fill_(-128), w._q.fill_(-128)
    w._q[n // 2:].fill_(127)
    w._q[:, k:], x._q[:, k:] = 0, 0
    y = x.zero_packed_linear(w, dtype=F32)
    assert same_bits(y, linear_expected(x, w, None, F32))
    assert (y[:, 0] == (2.0 ** 31 - 2.0 ** 18) * x.scale * w.scale[0]).all()


# --- gradients

def whole_dy(m, n, dtype, seed, top=3):
    return torch.randint(-top, top + 1, (m, n), generator=gen(seed), device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rule", [POW2, MAX])
@pytest.mark.parametrize("m, k, n", [s for s in SHAPES if s[1] < 20000])
def test_gradients_to_the_bit(m, k, n, rule, dtype):
    """Whole numbers times powers of two: every sum of these sizes is exact in fp32, in any order and in either split."""
    dy = whole_dy(m, n, dtype, 5)
    x = random_packed(m, k, 1, rule, torch.exp2(torch.randint(-1, 2, (m,), generator=gen(6), device=DEV).float()))
    w = random_packed(n, k, 2, rule, torch.exp2(torch.randint(-1, 2, (n,), generator=gen(7), device=DEV).float()))
    dw, dx = dy.double().T @ values(x), dy.double() @ values(w)
    assert max(m, n) * 3 * 127 * 4 < 2 ** 24            # in units of half a step
    for out in (F32, BF16):
        db = torch.empty(n, dtype=out, device=DEV)
        assert torch.equal(x.zero_packed_weight_grad(dy, dtype=out, bias_grad=db), dw.to(out))
        assert torch.equal(db, dy.double().sum(0).to(out))
        assert torch.equal(w.zero_packed_input_grad(dy, dtype=out), dx.to(out))
    old, old_b = torch.full((n, k), 3.0, device=DEV), torch.full((n,), -2.0, device=DEV)
    x.zero_packed_weight_grad(dy, out=old, accumulate=True, bias_grad=old_b)
    assert torch.equal(old, (dw + 3).float()) and torch.equal(old_b, (dy.double().sum(0) - 2).float())
    old = torch.full((m, k), 3.0, device=DEV, dtype=BF16)
    w.zero_packed_input_grad(dy, out=old, accumulate=True)
    assert torch.equal(old, (dx + 3).float().to(BF16))


@pytest.mark.parametrize("dtype, rule", [(BF16, POW2), (F16, POW2), (BF16, MAX)])
@pytest.mark.parametrize("long", [1, 24, 31, 32, 33, 130, 200, 227, 264, 300])
def test_gradients_in_large_tiles(long, dtype, rule):
    """Results of so many tiles that they are the large ones, with ragged edges, and sums that end anywhere in a step:
    lengths and widths that are multiples of eight and that are not (loaded straight into LDS, and through registers)."""
    one = lambda rows, seed: torch.exp2(torch.randint(-1, 2, (rows,), generator=gen(seed), device=DEV).float())
    for k, wide in ((2856, 3080), (2851, 3077)):
        x, dy = random_packed(long, k, 1, rule, one(long, 6)), whole_dy(long, wide, dtype, 5)
        assert torch.equal(x.zero_packed_weight_grad(dy, dtype=BF16), (dy.double().T @ values(x)).to(BF16))
        old = torch.full((wide, k), 3.0, device=DEV)
        x.zero_packed_weight_grad(dy, out=old, accumulate=True)
        assert torch.equal(old, (dy.double().T @ values(x) + 3).float())
        w, dz = random_packed(long, k, 2, rule, one(long, 7)), whole_dy(wide, long, dtype, 8)
        assert torch.equal(w.zero_packed_input_grad(dz, dtype=F32), (dz.double() @ values(w)).float())
        v, _ = strided(dz, 8)                           # NaN behind each row
        assert torch.equal(w.zero_packed_input_grad(v, dtype=F32), (dz.double() @ values(w)).float())
        v, _ = strided(dy, 8)
        assert torch.equal(x.zero_packed_weight_grad(v), (dy.double().T @ values(x)).float())


@pytest.mark.parametrize("k", [1, 16, 48, 63, 64, 65, 130, 256, 300, 333])
def test_linear_in_large_tiles(k):
    x, w = random_packed(4100, k, 1), random_packed(4150, k, 2, MAX, torch.rand(4150, generator=gen(3), device=DEV) + 0.01)
    y = x.zero_packed_linear(w, bias=w.scale, dtype=F32)
    assert same_bits(y, linear_expected(x, w, w.scale, F32))
    out, big = strided(torch.zeros(4100, 4150, dtype=BF16, device=DEV), 7, 1)
    x.zero_packed_linear(w, out=out)
    assert torch.equal(out, linear_expected(x, w, None, BF16)) and around(out, big, 1).isnan().all()


ALL_FEEDS = [(BF16, POW2), (F16, POW2), (BF16, MAX), (F16, MAX)]


def halves(rows, seed):
    """Scales a half, one and two."""
    return torch.exp2(torch.randint(-1, 2, (rows,), generator=gen(seed), device=DEV).float())


@pytest.mark.parametrize("dtype, rule", ALL_FEEDS)
@pytest.mark.parametrize("long", [2050, 4093, 4104])
def test_gradients_of_long_sums_in_large_tiles(long, dtype, rule):
    """Dense sums of up to 129 steps of large tiles, not split: the steps' places in LDS go round many times."""
    for k, wide in ((2856, 3080), (2851, 3077)):
        assert zpm.zero_packed_workspace(zpm.ZERO_PACKED_INPUT_GRAD, wide, k, long) == 0
        assert long * 3 * 127 * 4 < 2 ** 24             # in units of half a step: every sum is exact
        x, dy = random_packed(long, k, 1, rule, halves(long, 6)), whole_dy(long, wide, dtype, 5)
        assert torch.equal(x.zero_packed_weight_grad(dy), (dy.double().T @ values(x)).float())
        dz = whole_dy(wide, long, dtype, 8)
        assert torch.equal(x.zero_packed_input_grad(dz, dtype=F32), (dz.double() @ values(x)).float())


@pytest.mark.parametrize("dtype, rule", ALL_FEEDS)
@pytest.mark.parametrize("long", [5401, 8192])
@pytest.mark.parametrize("wide, k", [(2048, 4096), (4096, 2048), (2041, 4090)])
def test_gradients_of_split_sums_in_large_tiles(wide, k, long, dtype, rule):
    """Results of exactly 128 large tiles, half of what the chip takes at once: long sums are split and joined."""
    call = zpm.zero_packed_workspace
    assert call(zpm.ZERO_PACKED_INPUT_GRAD, wide, k, long) == (2 * wide * ((k + 3) // 4 * 4) * 4 + 255) // 256 * 256
    assert long * 3 * 127 * 4 < 2 ** 24
    x, dy, db = random_packed(long, k, 1, rule, halves(long, 6)), whole_dy(long, wide, dtype, 5), torch.empty(wide, device=DEV)
    want = dy.double().T @ values(x)
    assert torch.equal(x.zero_packed_weight_grad(dy, bias_grad=db), want.float())
    assert torch.equal(db, dy.double().sum(0).float())
    old, big = strided(torch.full((wide, k), 3.0, device=DEV), 5, 3)
    x.zero_packed_weight_grad(dy, out=old, accumulate=True)
    assert torch.equal(old, (want + 3).float()) and around(old, big, 3).isnan().all()
    assert torch.equal(x.zero_packed_weight_grad(dy, dtype=BF16), want.to(BF16))
    dz = whole_dy(wide, long, dtype, 8)
    want = dz.double() @ values(x)
    assert torch.equal(x.zero_packed_input_grad(dz, dtype=F32), want.float())
    old = torch.full((wide, k), 3.0, device=DEV, dtype=BF16)
    x.zero_packed_input_grad(dz, out=old, accumulate=True)
    assert torch.equal(old, (want + 3).float().to(BF16))


@pytest.mark.parametrize("k", [4096, 4091, 1040])
def test_linear_of_long_sums_in_large_tiles(k):
    x, w = random_packed(4100, k, 1), random_packed(4150, k, 2, MAX, torch.rand(4150, generator=gen(3), device=DEV) + 0.01)
    assert zpm.zero_packed_workspace(zpm.ZERO_PACKED_LINEAR, 4100, k, 4150) == 0
    assert same_bits(x.zero_packed_linear(w, bias=w.scale, dtype=F32), linear_expected(x, w, w.scale, F32))
    assert torch.equal(x.zero_packed_linear(w), linear_expected(x, w, None, BF16))


@pytest.mark.parametrize("rule, dtype", [(POW2, BF16), (POW2, F16), (MAX, BF16), (MAX, F16)])
@pytest.mark.parametrize("m, k, n", [(40, 50, 60), (1003, 333, 143), (2048, 256, 688), (70, 640, 1600)])
def test_gradients(m, k, n, rule, dtype):
    g = gen(m)
    dy = (torch.randn(m, n, generator=g, device=DEV) * torch.exp(torch.randn(m, 1, generator=g, device=DEV)) * 0.01).to(dtype)
    x = zpm.ZeroPacked(m, k, rule).zero_packed_write(torch.randn(m, k, generator=g, device=DEV) * torch.exp(torch.randn(m, 1, generator=g, device=DEV)))
    w = zpm.ZeroPacked(n, k, rule).zero_packed_write(torch.randn(n, k, generator=g, device=DEV) * 0.02)
    # every product passes at most as many fp32 additions as there are, each off by half a step of a partial sum, which
    # the sum of magnitudes bounds; for ZERO_SCALE_MAX dy * scale is off by 2^-17 of itself (2^-24 more for its product
    # in fp32), and where it is less than a normal bf16 its second term ends at 2^-134
    for got, a, b in ((x.zero_packed_weight_grad(dy), dy.double().T, values(x)), (w.zero_packed_input_grad(dy, dtype=F32), dy.double(), values(w))):
        terms = a.shape[1]
        most = a.abs() @ b.abs() * ((terms + 16) * 2.0 ** -24 + (2.0 ** -17 + 2.0 ** -24 if rule == MAX else 0)) + terms * 127 * 2.0 ** -134
        want = a @ b
        assert ((got.double() - want).abs() <= most + want.abs() * half_step(F32)).all()
    # 16-bit results are the fp32 ones rounded once
    for out in (F16, BF16):
        assert torch.equal(x.zero_packed_weight_grad(dy, dtype=out), x.zero_packed_weight_grad(dy).to(out))
        assert torch.equal(w.zero_packed_input_grad(dy, dtype=out), w.zero_packed_input_grad(dy, dtype=F32).to(out))


@pytest.mark.parametrize("lead", [0, 1, 8])
@pytest.mark.parametrize("m, k, n", [(37, 45, 51), (200, 300, 136), (130, 256, 264)])
def test_gradients_strided(m, k, n, lead):
    x, w, dy = random_packed(m, k, 1), random_packed(n, k, 2), whole_dy(m, n, BF16, 5)
    v, _ = strided(dy, 5 if lead == 1 else 8, lead)    # NaN around it
    for call, shape in ((x.zero_packed_weight_grad, (n, k)), (w.zero_packed_input_grad, (m, k))):
        out, big = strided(torch.zeros(shape, dtype=F32, device=DEV), 5, lead)
        call(v, out=out)
        assert torch.equal(out, call(dy, dtype=F32))
        assert around(out, big, lead).isnan().all()


@pytest.mark.parametrize("dtype, rule", [(BF16, POW2), (F16, POW2), (BF16, MAX)])
def test_gradients_of_infinities(dtype, rule):
    """An infinity in dy, and a row of NaN, reach the gradients that they enter, and no others."""
    m, k, n = 70, 90, 50
    one = torch.ones
    x, w = random_packed(m, k, 1, rule, one(m, device=DEV)), random_packed(n, k, 2, rule, one(n, device=DEV))
    dy = whole_dy(m, n, dtype, 5)
    dy[3, 7] = math.inf
    x._q[3, :k // 2] = 5                               # elsewhere the sign varies and zeros make NaN
    want = dy.double().T @ values(x)
    got = x.zero_packed_weight_grad(dy)
    assert same_bits(got, want.float())
    assert not got[7].isfinite().any() and got[:7].isfinite().all() and got[8:].isfinite().all()
    assert same_bits(w.zero_packed_input_grad(dy, dtype=F32), (dy.double() @ values(w)).float())
    dy[3, 7] = 1
    x.scale[11] = math.nan
    assert x.zero_packed_weight_grad(dy).isnan().all()
    w.scale[13] = math.nan
    assert w.zero_packed_input_grad(dy).isnan().all()


@pytest.mark.parametrize("e", [-126, -100, 104, 112, 121, 122])
def test_gradients_of_extreme_scales(e):
    """Scales from the smallest to the largest there are: the products q * scale are finite, and exact."""
    m, k, n = 45, 70, 33
    top = 63 if e == 122 else 127                       # 127 * 2^122 is no float
    x = random_packed(m, k, 1, POW2, torch.full((m,), 2.0 ** e, device=DEV))
    x._q.clamp_(-top, top)
    assert torch.equal(x.zero_packed_read(dtype=F32).double(), values(x)) and values(x).abs().max() < 3.4e38
    dy = whole_dy(m, n, BF16, 5) * 2.0 ** (-e // 2)
    assert torch.equal(x.zero_packed_weight_grad(dy).double(), dy.double().T @ values(x))
    w = x
    dz = whole_dy(n, m, BF16, 6) * 2.0 ** (-e // 2)
    assert torch.equal(w.zero_packed_input_grad(dz, dtype=F32).double(), dz.double() @ values(w))


@pytest.mark.parametrize("m", [45, 48, 300])
@pytest.mark.parametrize("rule, dtype", [(POW2, BF16), (POW2, F16), (MAX, BF16), (MAX, F16)])
@pytest.mark.parametrize("e", [-126, -119, -100, 100, 121])
def test_gradients_at_the_ends_of_the_range(e, rule, dtype, m):
    """Scales at both ends, dy from the type's usual smallest to beyond what dy * scale could hold: products that are
    multiples of 2^-149 are exact, and columns of zeros are zeros wherever dy is finite."""
    k = 72
    x = random_packed(m, k, 1, rule, torch.full((m,), 2.0 ** e, device=DEV))
    x._q[:, 5], x._q[:, 64] = 0, 0
    for d in (-24, -14, -3) if e < 0 else (-24, -20):
        for wide in (33, 40):                           # through registers, and bf16 with powers of two straight into LDS
            unit = max(e + d, -149)
            dy = whole_dy(m, wide, dtype, 5, 15) * 2.0 ** (unit - e)
            got = x.zero_packed_weight_grad(dy)
            assert torch.equal(got.double(), dy.double().T @ values(x)) and got.any()
            dz = whole_dy(wide, m, dtype, 6, 15) * 2.0 ** (unit - e)
            assert torch.equal(x.zero_packed_input_grad(dz, dtype=F32).double(), dz.double() @ values(x))
    x._q.abs_().clamp_(max=63)
    for dy in (torch.full((m, 40), 6e4, device=DEV).to(dtype), torch.full((m, 33), 2.0 ** 15, device=DEV).to(dtype)):
        for got, want in ((x.zero_packed_weight_grad(dy), (dy.double().T @ values(x)).float()),
                          (x.zero_packed_input_grad(dy.T.contiguous(), dtype=F32), (dy.double().T @ values(x)).float())):
            assert not got[:, 5].any() and not got[:, 64].any() and not got.isnan().any()
            # all terms but second ones are positive, fp16 dy has two: each addition is off by half a step of the sum
            assert torch.equal(got.isinf(), want.isinf()) and (e > 0 or ((got - want).abs() <= want * (2 * m + 16) * 2.0 ** -24).all())


@pytest.mark.parametrize("m", [45, 48, 300])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("e", [-126, -100, 0, 120])
def test_gradients_by_the_maximum_at_the_ends_of_the_range(e, dtype, m):
    """Scales that are no powers of two: dy times a scale's significand is off by 2^-17 of itself (2^-24 more for its product
    in fp32), whatever the scale's exponent."""
    x = random_packed(m, 72, 1, MAX, (1 + torch.rand(m, generator=gen(2), device=DEV)) * 2.0 ** e)
    x._q[:, 5] = 0
    small = 2.0 ** -20 if e > 0 else 2.0 ** -3          # dy of at most 4 to 5 times this: finite sums
    dy = (torch.randn(m, 40, generator=gen(3), device=DEV) * small).to(dtype)
    a, v = dy.double().T, values(x)
    want, mag = a @ v, a.abs() @ v.abs()
    # two terms a product; a sum below the normal numbers is off by half of 2^-149 an addition
    most = mag * ((2 * m + 16) * 2.0 ** -24 + 2.0 ** -17 + 2.0 ** -24) + (2 * m + 16) * 2.0 ** -150
    for got in (x.zero_packed_weight_grad(dy), x.zero_packed_input_grad(dy.T.contiguous(), dtype=F32)):
        assert ((got.double() - want).abs() <= most).all() and not got[:, 5].any()
    # dy beyond what dy * scale could hold
    dy.fill_(6e4)
    got = x.zero_packed_weight_grad(dy)
    assert not got[:, 5].any() and (e < 0 or torch.equal(got.isfinite(), (dy.double().T @ v).float().isfinite()))
    x.scale[7] = math.nan
    assert x.zero_packed_weight_grad(dy).isnan().all() and x.zero_packed_input_grad(dy.T.contiguous()).isnan().all()


@pytest.mark.parametrize("m", [45, 300])
@pytest.mark.parametrize("rule", [POW2, MAX])
def test_gradients_of_rows_of_all_scales(rule, m):
    """Rows next to each other whose scales lie hundreds of binades apart, and dy the other way round: products are whole
    numbers, and so every sum is exact.  Then the smallest rows by themselves, whose sums no other row joins."""
    g = gen(m)
    e = torch.randint(-94, 84, (m,), generator=g, device=DEV).float()
    e[:8] = torch.tensor([-94, -33, -32, -31, 31, 32, 33, 84], device=DEV)
    x = random_packed(m, 72, 1, rule, torch.exp2(e))
    dy = (whole_dy(m, 40, BF16, 5).float() * torch.exp2(-e)[:, None]).to(BF16)
    want = dy.double().T @ values(x)
    assert torch.equal(x.zero_packed_weight_grad(dy).double(), want)
    assert torch.equal(x.zero_packed_input_grad(dy.T.contiguous(), dtype=F32).double(), want)
    small = e < -32
    x._q[~small, :9] = 0
    for dtype in (BF16, F16):
        dz = whole_dy(m, 40, dtype, 6)
        want = dz.double().T @ values(x)
        most = (dz.double().abs().T @ values(x).abs()) * (2 * m + 16) * 2.0 ** -24
        for got in (x.zero_packed_weight_grad(dz), x.zero_packed_input_grad(dz.T.contiguous(), dtype=F32)):
            assert ((got.double() - want).abs() <= most).all() and got[:, :9].abs().max() < 2.0 ** -15


def test_gradients_of_nothing():
    x, dy = zpm.ZeroPacked(0, 40), torch.empty(0, 30, dtype=BF16, device=DEV)
    db = torch.full((30,), 7.0, device=DEV)
    assert not x.zero_packed_weight_grad(dy, bias_grad=db).any() and not db.any()
    dw, db = torch.full((30, 40), 2.0, device=DEV), torch.full((30,), 7.0, device=DEV)
    x.zero_packed_weight_grad(dy, out=dw, accumulate=True, bias_grad=db)
    assert (dw == 2).all() and (db == 7).all()
    w = zpm.ZeroPacked(0, 40)
    assert not w.zero_packed_input_grad(torch.empty(6, 0, dtype=BF16, device=DEV)).any()
    x = zpm.ZeroPacked(5, 0)
    db = torch.empty(30, device=DEV)
    assert x.zero_packed_weight_grad(torch.ones(5, 30, dtype=BF16, device=DEV), bias_grad=db).shape == (30, 0)
    assert (db == 5).all()


def test_products_of_the_largest_pitches():
    """Rows as far apart as the calls allow: tiles' rows then lie up to 2^31 bytes apart."""
    m, k, n, far = 300, 72, 40, 1 << 22

    def apart(p):
        wide = torch.empty(p.rows, far, dtype=torch.int8, device=DEV)
        wide[:, :p._q.shape[1]] = p._q
        return zpm.ZeroPacked.of(wide, p.scale, p.cols, p.rule)
    x, w = random_packed(m, k, 1), random_packed(n, k, 2)
    xf = apart(x)
    assert torch.equal(xf.zero_packed_linear(w), linear_expected(x, w, None, BF16))
    assert torch.equal(w.zero_packed_linear(xf), linear_expected(w, x, None, BF16))
    wf = apart(random_packed(300, k, 3))
    assert torch.equal(xf.zero_packed_linear(wf), linear_expected(x, wf, None, BF16))
    del wf
    assert torch.equal(xf.zero_packed_read(), x.zero_packed_read())
    dy, dz = whole_dy(m, n, BF16, 5), whole_dy(n, m, BF16, 6)
    want, want_x = (dy.double().T @ values(x)).float(), (dz.double() @ values(x)).float()
    for dtype in (BF16, F16):
        assert torch.equal(xf.zero_packed_weight_grad(dy.to(dtype)), want)
        assert torch.equal(xf.zero_packed_input_grad(dz.to(dtype), dtype=F32), want_x)
    del xf
    # dy's rows: the farthest that go straight into LDS, and beyond
    for pitch in (far, far + 8):
        wide = torch.empty(m, pitch, dtype=BF16, device=DEV)
        wide[:, :n] = dy
        assert torch.equal(x.zero_packed_weight_grad(wide[:, :n]), want)
        tall = torch.empty(m, pitch, dtype=BF16, device=DEV)
        tall[:, :n] = dy
        assert torch.equal(w.zero_packed_input_grad(tall[:, :n], dtype=F32), (dy.double() @ values(w)).float())
        del wide, tall
    wide = torch.empty(5, 1 << 30, dtype=BF16, device=DEV)
    wide[:, :n] = dy[:5]
    assert torch.equal(x[:5].zero_packed_weight_grad(wide[:, :n]), (dy[:5].double().T @ values(x[:5])).float())
    out = wide[:, 64:64 + k]
    w.zero_packed_input_grad(dy[:5], out=out)
    assert torch.equal(out, (dy[:5].double() @ values(w)).to(BF16))


def test_gradient_far_offsets():
    """dy of more than 2^31 elements (both orders), and a weight gradient of more than 2^31 bytes."""
    m, n, k = 65600, 32800, 40
    dy = torch.zeros(m, n, dtype=BF16, device=DEV)
    x, w = random_packed(m, k, 1), random_packed(n, k, 2)
    rows, cols = [0, 1, 32767, 65470, 65598, m - 1], [0, 5, 17000, n - 1]
    for r in rows:
        for c in cols:
            dy[r, c] = r % 3 + 1 + c % 2
    sub = dy[rows][:, cols].double()
    dw = x.zero_packed_weight_grad(dy)
    assert torch.equal(dw[cols].double(), sub.T @ values(x)[rows]) and int(dw.any(1).sum()) <= len(cols)
    dx = w.zero_packed_input_grad(dy, dtype=F32)
    assert torch.equal(dx[rows].double(), sub @ values(w)[cols]) and int(dx.any(1).sum()) <= len(rows)
    del dy, dw, dx
    n, k, m = 40000, 30000, 5
    dy, x = whole_dy(m, n, BF16, 5), random_packed(m, k, 1)
    dw = x.zero_packed_weight_grad(dy)
    for r in (0, 17895, 17896, 35791, 35792, n - 1):
        assert torch.equal(dw[r].double(), dy[:, r].double() @ values(x))


# --- activation functions

def f64(x, kind, want_slope):
    """f, f' and the h whose logistic function f goes by."""
    if kind == GELU:
        a = 2 * math.sqrt(2 / math.pi)
        h, dh = a * (x + 0.044715 * x ** 3), a * (1 + 3 * 0.044715 * x ** 2)
    else:
        h, dh = x, torch.ones_like(x)
    s, t = torch.sigmoid(h), torch.sigmoid(-h)
    return (s + x * s * t * dh if want_slope else x * s), h, s, t, dh


def act_bound(x, kind):
    """How far fp32 arithmetic may be off: h by four roundings, which the exponential turns into a relative error of e^-h
    of as many times |h|; a few more roundings for the exponential, sum, reciprocal and products."""
    f, h, s, t, dh = f64(x, kind, False)
    rel = (6 * h.abs() + 16) * 2.0 ** -24
    # tails below the smallest normal number may become zero
    ef = f.abs() * (rel * t + 4 * 2.0 ** -24) + (x.abs() + 1) * 2.0 ** -126
    es = (s + (x * s * t * dh).abs()) * rel * 2 + (1 + (x * dh).abs()) * 2.0 ** -126
    return ef, es


ACT_SHAPES = [(1, 1), (3, 7), (4, 16), (5, 33), (2, 520), (3, 1031), (7, 2048), (2, 4100), (1, 8191), (2, 11008), (2, 20001),
              (1, 32769), (600, 40)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", [GELU, SILU])
@pytest.mark.parametrize("rows, n", ACT_SHAPES)
def test_act(rows, n, kind, gated):
    for src, rule in ((BF16, POW2), (F16, MAX), (F32, POW2)):
        x = (3 * torch.randn(rows, 2 * n if gated else n, generator=gen(n), device=DEV)).to(src)
        x.view(-1)[:: max(1, x.numel() // 7)] *= 8
        xp, yp = zpm.ZeroPacked(*x.shape, rule), zpm.ZeroPacked(rows, n, rule)
        for p in (xp, yp):
            p._q.fill_(99)
        y = xp.zero_packed_act(x, kind, gated, packed=yp, dtype=F32)
        want_q, want_s = packed_of(x, rule)
        assert torch.equal(xp.q, want_q) and same_bits(xp.scale, want_s) and not xp._q[:, xp.cols:].any()
        d = x.double()
        f, ef = f64(d[:, :n], kind, False)[0], act_bound(d[:, :n], kind)[0]
        u = d[:, n:] if gated else torch.ones_like(f)
        want, most = f * u, (ef * u.abs() + (f * u).abs() * 2.0 ** -23)
        assert ((y.double() - want).abs() <= most).all()
        # the packed result is that of these very fp32 values
        want_q, want_s = packed_of(y, rule)
        assert torch.equal(yp.q, want_q) and same_bits(yp.scale, want_s) and not yp._q[:, n:].any()
        # 16-bit results are the fp32 ones rounded; any of the three may be left out
        for out in (F16, BF16):
            assert torch.equal(xp.zero_packed_act(x, kind, gated, dtype=out), y.to(out))
        alone = zpm.ZeroPacked(rows, n, rule)
        assert zpm.ZeroPacked(*x.shape).zero_packed_act(x, kind, gated, packed=alone) is alone
        assert torch.equal(alone._q, yp._q)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows, n", [(5, 33), (3, 1031), (2, 4100), (2, 20001), (2, 20008)])
def test_act_results_one_by_one(rows, n, gated):
    """Each result by itself, by the C names, is the one of the call that asks for all; the packed two by rules of their own."""
    stream = torch.cuda.current_stream().cuda_stream
    x = (3 * torch.randn(rows, 2 * n if gated else n, generator=gen(n), device=DEV)).to(BF16)
    new = lambda cols, rule: zpm.ZeroPacked(rows, cols, rule)
    xp, yp, y = new(x.shape[1], MAX), new(n, POW2), torch.empty(rows, n, device=DEV)
    for t in (xp, yp):
        t._q.fill_(99)
    zpm.zero_packed_act(SILU, gated, matrix(x, "x"), xp._desc, matrix(y, "y"), yp._desc, stream)
    for p, want in ((xp, packed_of(x, MAX)), (yp, packed_of(y, POW2))):
        assert torch.equal(p.q, want[0]) and same_bits(p.scale, want[1]) and not p._q[:, p.cols:].any()
    y1, xp1, yp1 = torch.empty_like(y), new(x.shape[1], MAX), new(n, POW2)
    zpm.zero_packed_act(SILU, gated, matrix(x, "x"), None, matrix(y1, "y"), None, stream)
    zpm.zero_packed_act(SILU, gated, matrix(x, "x"), xp1._desc, None, None, stream)
    zpm.zero_packed_act(SILU, gated, matrix(x, "x"), None, None, yp1._desc, stream)
    assert torch.equal(y1, y)
    assert torch.equal(xp1.q, xp.q) and torch.equal(xp1.scale, xp.scale) and torch.equal(yp1.q, yp.q) and torch.equal(yp1.scale, yp.scale)


@pytest.mark.parametrize("gated", [False, True])
def test_act_of_more_rows_than_a_launch_has_blocks(gated):
    rows, n = (1 << 20) + 3, 1032
    x = torch.randn(rows, 2 * n if gated else n, generator=gen(n), device=DEV, dtype=BF16)
    xp, yp = zpm.ZeroPacked(*x.shape), zpm.ZeroPacked(rows, n)
    y = xp.zero_packed_act(x, GELU, gated, packed=yp, dtype=BF16)
    dx = xp.zero_packed_act_grad(y, GELU, gated)
    for a in (0, rows - 128):
        b = slice(a, a + 128)
        xq, yq = zpm.ZeroPacked(128, x.shape[1]), zpm.ZeroPacked(128, n)
        assert torch.equal(xq.zero_packed_act(x[b], GELU, gated, packed=yq, dtype=BF16), y[b])
        for got, want in ((xp[b], xq), (yp[b], yq)):
            assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)
        assert torch.equal(xq.zero_packed_act_grad(y[b], GELU, gated), dx[b])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", [GELU, SILU])
@pytest.mark.parametrize("rows, n", ACT_SHAPES)
def test_act_grad(rows, n, kind, gated):
    g = gen(n)
    xp = random_packed(rows, 2 * n if gated else n, 1, POW2, torch.exp2(torch.randint(-7, -3, (rows,), generator=g, device=DEV).float()))
    v = values(xp)
    slope, es = f64(v[:, :n], kind, True)[0], act_bound(v[:, :n], kind)[1]
    for dtype, out in ((BF16, F32), (F32, F32), (F16, BF16)):
        dy = torch.randn(rows, n, generator=g, device=DEV).to(dtype)
        d = dy.double()
        got = xp.zero_packed_act_grad(dy, kind, gated, dtype=out).double()
        if gated:
            f, ef = f64(v[:, :n], kind, False)[0], act_bound(v[:, :n], kind)[0]
            want = torch.cat([d * v[:, n:] * slope, d * f], 1)
            most = torch.cat([(d * v[:, n:]).abs() * (es + slope.abs() * 2.0 ** -23), d.abs() * (ef + f.abs() * 2.0 ** -23)], 1)
        else:
            want, most = d * slope, d.abs() * (es + slope.abs() * 2.0 ** -23)
        assert ((got - want).abs() <= most + (want.abs() + most) * half_step(out) + tiny(out)).all()


@pytest.mark.parametrize("kind", [GELU, SILU])
def test_act_slope_against_differences(kind):
    """The gradient is that of the function: central differences of the forward formula in 64 bits."""
    x = torch.linspace(-8, 8, 2001, dtype=torch.float64)
    h = 1e-5
    diff = (f64(x + h, kind, False)[0] - f64(x - h, kind, False)[0]) / (2 * h)
    # third derivatives of both functions are below 4: h^2 / 6 * 4, and the differences' own rounding
    assert ((diff - f64(x, kind, True)[0]).abs() <= 4 * h * h / 6 + 8 * 2.0 ** -53 / h * 2).all()
    p = zpm.ZeroPacked(1, 255)
    q = torch.zeros(1, 256, dtype=torch.int8, device=DEV)
    q[0, :255] = torch.arange(-127, 128, device=DEV).to(torch.int8)
    p = zpm.ZeroPacked.of(q, torch.full((1,), 2.0 ** -4, device=DEV), 255)
    v = values(p).cpu()
    diff = (f64(v + h, kind, False)[0] - f64(v - h, kind, False)[0]) / (2 * h)
    got = p.zero_packed_act_grad(torch.ones(1, 255, device=DEV), kind).double().cpu()
    assert ((got - diff).abs() <= 4 * h * h / 6 + 16 * 2.0 ** -53 / h + act_bound(v, kind)[1]).all()


@pytest.mark.parametrize("kind", [GELU, SILU])
def test_act_of_huge_values_and_infinities(kind):
    x = torch.tensor([[1e30, -1e30, 3e38, -3e38, 60.0, -60.0, 0.0, -200.0], [1.0, math.inf, 2, 3, 4, 5, 6, 7],
                      [1.0, -math.inf, 2, 3, 4, 5, 6, 7], [1.0, math.nan, 2, 3, 4, 5, 6, 7]], device=DEV)
    xp = zpm.ZeroPacked(4, 8)
    y = xp.zero_packed_act(x, kind)
    assert torch.equal(y[0].abs(), torch.tensor([1e30, 0, 3e38, 0, 60.0, 0, 0, 0], device=DEV)) or \
        (y[0, 5].abs() < 1e-20 and torch.equal(y[0, [0, 1, 2, 3, 4, 6]].abs(), torch.tensor([1e30, 0, 3e38, 0, 60.0, 0], device=DEV)))
    assert y[1:, 0].isfinite().all() and y[3, 1].isnan() and y[1, 1] == math.inf and y[2, 1].isnan()
    # beside 3e38 the packed 1e30 is 0, where both slopes are a half
    dx = xp.zero_packed_act_grad(torch.ones(4, 8, device=DEV), kind)
    assert torch.equal(dx[0, :4], torch.tensor([0.5, 0.5, 1, 0], device=DEV)) and dx[1:].isnan().all()


def test_act_grad_in_place_and_strided():
    n = 1003
    xp = random_packed(9, n, 1, POW2, torch.full((9,), 2.0 ** -5, device=DEV))
    dy = torch.randn(9, n, generator=gen(2), device=DEV).bfloat16()
    want = xp.zero_packed_act_grad(dy, GELU)
    v, big = strided(dy, 5, 3)
    xp.zero_packed_act_grad(v, GELU, out=v)
    assert torch.equal(v, want) and around(v, big, 3).isnan().all()
    gp = random_packed(9, 2 * n, 1, POW2, torch.full((9,), 2.0 ** -5, device=DEV))
    out, big = strided(torch.zeros(9, 2 * n, dtype=BF16, device=DEV), 5, 3)
    gp.zero_packed_act_grad(dy, SILU, True, out=out)
    assert torch.equal(out, gp.zero_packed_act_grad(dy, SILU, True)) and around(out, big, 3).isnan().all()
    x, _ = strided(torch.randn(9, 2 * n, generator=gen(3), device=DEV).half(), 5, 1)
    y, big = strided(torch.zeros(9, n, dtype=F16, device=DEV), 5, 1)
    p, r = zpm.ZeroPacked(9, 2 * n), zpm.ZeroPacked(9, 2 * n)
    p.zero_packed_act(x, SILU, True, out=y)
    assert torch.equal(y, r.zero_packed_act(x.contiguous(), SILU, True)) and torch.equal(p._q, r._q)
    assert around(y, big, 1).isnan().all()

"""The packed-row operators as they are used together: a gated and a plain layer's forward and backward pass, into the
sharded step; captured calls, streams, rows of one buffer, tensors on leaves of an autograd graph."""
import math

import numpy as np
import pytest
import torch

import oracle
import zero_partitioned_mixed_reduce_amd as zpm
from tests.gpu_harness import dev16
from tests.test_gpu_packed import BF16, DEV, F16, F32, GELU, POW2, SILU, f64, gen, packed_of, random_packed, values, whole_dy
from zero_partitioned_mixed_reduce_amd import ZeroGrads, ZeroPacked, _abi
from zero_partitioned_mixed_reduce_amd.packed import matrix

pytestmark = pytest.mark.gpu


class Block:
    """x -> x + W2 f(W1 x + b1), f a gated or plain activation: parameters are views of one flat 16-bit buffer, gradients
    of one flat buffer in the same order; what the backward pass needs is kept in packed rows."""

    def __init__(self, flat, grads, d, f, kind, gated):
        self.kind, self.gated, self.d, self.f = kind, gated, d, f
        wide = 2 * f if gated else f
        sizes = [(wide, d), (wide,), (d, f)]
        self.numel = [math.prod(s) for s in sizes]
        cut = lambda t: [v.view(s) for v, s in zip(t[:sum(self.numel)].split(self.numel), sizes)]
        self.w1, self.b1, self.w2 = cut(flat)
        self.dw1, self.db1, self.dw2 = cut(grads)
        self.p1, self.p2 = ZeroPacked(wide, d), ZeroPacked(d, f)

    def pack_weights(self):
        self.p1.zero_packed_write(self.w1)
        self.p2.zero_packed_write(self.w2)

    def forward(self, x):
        m = x.shape[0]
        self.xp, self.hp, self.ap = ZeroPacked(m, self.d), ZeroPacked(m, self.p1.rows), ZeroPacked(m, self.f)
        h = self.xp.zero_packed_write(x).zero_packed_linear(self.p1, bias=self.b1)
        self.hp.zero_packed_act(h, self.kind, self.gated, packed=self.ap)
        return x + self.ap.zero_packed_linear(self.p2)

    def backward(self, dy, accumulate):
        self.ap.zero_packed_weight_grad(dy, out=self.dw2, accumulate=accumulate)
        da = self.p2.zero_packed_input_grad(dy)
        dh = self.hp.zero_packed_act_grad(da, self.kind, self.gated)
        self.xp.zero_packed_weight_grad(dh, out=self.dw1, accumulate=accumulate, bias_grad=self.db1)
        return self.p1.zero_packed_input_grad(dh) + dy


@pytest.mark.parametrize("kind, gated", [(SILU, True), (GELU, False)])
def test_block_into_sharded_step(kind, gated):
    """Two micro-steps of a block, its gradients clipped into the send buffer and taken in by the sharded step."""
    d, f, m = 136, 200, 333
    g = gen(1)
    psi = (2 * f if gated else f) * (d + 1) + d * f
    flat = (torch.randn(psi, generator=g, device=DEV) * 0.1).to(BF16)
    grads = torch.full((psi,), math.nan, device=DEV)
    b = Block(flat, grads, d, f, kind, gated)
    assert sum(b.numel) == psi
    b.pack_weights()
    exact = [torch.zeros_like(t, dtype=torch.float64) for t in (b.dw1, b.db1, b.dw2)]
    for step in range(2):
        x = torch.randn(m, d, generator=g, device=DEV).to(BF16)
        dy = (torch.randn(m, d, generator=g, device=DEV) * 1e-3).to(BF16)
        y, dx = b.forward(x), b.backward(dy, accumulate=step > 0)
        # the same block in 64 bits, on the values that the packed rows stand for
        X, W1, W2, H, A = (values(p) for p in (b.xp, b.p1, b.p2, b.hp, b.ap))
        h = X @ W1.T + b.b1.double()
        # h in 16 bits and then in 8: off by half a step of each of its row's packed values and 2^-8 of itself
        assert ((H - h).abs() <= b.hp.scale.double()[:, None] / 2 + h.abs() * 2.0 ** -7).all()
        a = f64(H[:, :f], kind, False)[0] * (H[:, f:] if gated else 1)
        assert ((A - a).norm() / a.norm()) < 0.03       # A is of h, not of H: a step of 8 bits apart
        want_y = x.double() + A @ W2.T
        assert ((y.double() - want_y).abs() <= 2.0 ** -8 * (want_y.abs() + (A @ W2.T).abs()) + 2.0 ** -20).all()
        DY = dy.double()
        da = (DY @ W2).to(BF16).double()
        slope = f64(H[:, :f], kind, True)[0]
        dh = torch.cat([da * H[:, f:] * slope, da * f64(H[:, :f], kind, False)[0]], 1) if gated else da * slope
        # dh is rounded to 16 bits, and so is da, within a rounding of the one here
        exact[0] += dh.T @ X
        exact[1] += dh.sum(0)
        exact[2] += DY.T @ A
        for got, want, mag in zip((b.dw1, b.db1, b.dw2), exact, (dh.abs().T @ X.abs(), dh.abs().sum(0), DY.abs().T @ A.abs())):
            assert ((got.double() - want).abs() <= (step + 1) * mag.max() * 2.0 ** -6).all()
            assert (got.double() - want).norm() <= 2.0 ** -7 * want.norm()
        assert (dx.double() - DY - dh @ W1).norm() <= 2.0 ** -6 * (dh @ W1 + DY).norm()

    # into the step: clipped into the 16-bit send buffer, one rank's shard is the model
    send = torch.empty(psi, dtype=BF16, device=DEV)
    clip = ZeroGrads([b.dw1, b.db1, b.dw2], out=send)
    clip.zero_grads_clip_norm(0.05)
    assert clip.query()["coef"] < 1.0 and abs(clip.query()["norm"] - float(grads.double().norm())) <= 1e-6 * clip.query()["norm"]
    host = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    p16, master = host(flat).copy(), flat.float().cpu().numpy()
    hp = oracle.HParams(1e-3, 0.9, 0.999, 1e-8, 0.01)
    st = oracle.RankState(oracle.BF16, p16.copy(), master.copy())
    loc = oracle.grad_stats(oracle.BF16, [host(send)], 1.0)
    coef, _ = oracle.clip_coef(loc[2], 1.0)
    oracle.adam(False, loc[0], coef, hp, st.counters, st.w, st.m, st.v)
    oracle.cast(oracle.BF16, st.w, st.p16)
    s = zpm.ZeroShard(b.numel, 1, 0, oracle.BF16, flat.view(torch.int16), with_red=True)
    s.zero_reduce_grads([send], 1.0)
    s.zero_check_overflow(False)
    s.zero_grad_norm(0.0, 1.0)
    s.zero_adam_step(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    assert (host(flat) == st.p16).all() and (host(flat) != p16).any()
    # the updated parameters are packed again
    b.pack_weights()
    assert torch.equal(b.p1.q, packed_of(b.w1, POW2)[0])
    # an infinity in an activation reaches the step, which skips
    x[5, 3] = math.inf
    b.forward(x), b.backward(dy, accumulate=False)
    clip.zero_grads_clip_norm(0.05)
    assert clip.query()["found_inf"]
    s.zero_reduce_grads([send], 1.0)
    assert s.zero_check_overflow(False, sync=True)


def test_captured_block():
    """A step captured and replayed with other inputs, eager work and synchronisations between the replays; the first graph
    shares its pool's memory with nothing of the second."""
    d, f, m = 128, 300, 260
    psi = 2 * f * (d + 1) + d * f
    flat = (torch.randn(psi, generator=gen(1), device=DEV) * 0.1).to(BF16)
    eager, graphed = torch.zeros(psi, device=DEV), torch.zeros(psi, device=DEV)
    one, two = Block(flat, eager, d, f, SILU, True), Block(flat, graphed, d, f, SILU, True)
    x, dy = torch.zeros(m, d, dtype=BF16, device=DEV), torch.zeros(m, d, dtype=BF16, device=DEV)
    res = {}

    def step(b):
        b.pack_weights()
        return b.forward(x), b.backward(dy, accumulate=False)
    step(two)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res[k] = step(two)
        graphs.append(g)
    for turn in range(4):
        x.copy_(torch.randn(m, d, generator=gen(10 + turn), device=DEV))
        dy.copy_(torch.randn(m, d, generator=gen(20 + turn), device=DEV) * 1e-3)
        want = step(one)
        for k, g in enumerate(graphs):
            graphed.fill_(5)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(res[k][0], want[0]) and torch.equal(res[k][1], want[1]) and torch.equal(graphed, eager), (turn, k)
        flat.mul_(0.99)


def test_split_products_in_graphs_and_on_streams():
    """Products whose sums are split and joined through a workspace: captured twice, replayed in turn with eager calls of
    other sizes between; and on two streams at once."""
    x, dy = random_packed(30000, 96, 1), whole_dy(30000, 80, BF16, 2, 1)
    xs, w = random_packed(3, 20000, 3), random_packed(130, 20000, 4)
    assert zpm.zero_packed_workspace(zpm.ZERO_PACKED_WEIGHT_GRAD, 30000, 96, 80) > 0
    want, want_y = x.zero_packed_weight_grad(dy), xs.zero_packed_linear(w, dtype=F32)
    assert torch.equal(want_y, ((xs.q.double() @ w.q.double().T).float() * xs.scale[:, None] * w.scale))
    torch.cuda.synchronize()
    outs, graphs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((x.zero_packed_weight_grad(dy), xs.zero_packed_linear(w, dtype=F32)))
        graphs.append(g)
    for turn in range(3):
        for k, g in enumerate(graphs):
            outs[k][0].zero_(), outs[k][1].zero_()
            g.replay()
            x[:4000].zero_packed_weight_grad(dy[:4000])
            torch.cuda.synchronize()
            assert torch.equal(outs[k][0], want) and torch.equal(outs[k][1], want_y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((x.zero_packed_weight_grad(dy), xs.zero_packed_linear(w, dtype=F32)))
    torch.cuda.synchronize()
    for a, b in got[0] + got[1]:
        assert torch.equal(a, want) and torch.equal(b, want_y)


def test_split_linear_and_column_sums_in_graphs_and_on_streams():
    """A linear layer of so many tokens that its sums are split and joined, and a weight gradient whose bias gradient is
    joined through the same workspace: captured twice, replayed in turn with eager calls of other sizes between; and on two
    streams at once."""
    m, k, n = 130, 20000, 131
    assert zpm.zero_packed_workspace(zpm.ZERO_PACKED_LINEAR, m, k, n) >= 2 * m * 132 * 4
    x, w, dy, z = random_packed(m, k, 3), random_packed(n, k, 4), whole_dy(30000, 80, F16, 2, 1), random_packed(30000, 96, 1)
    assert zpm.zero_packed_workspace(zpm.ZERO_PACKED_WEIGHT_GRAD, 30000, 96, 80) > 2 * 96 * 80 * 4

    def step(into):
        into[0].copy_(x.zero_packed_linear(w, bias=w.scale, dtype=F32))
        z.zero_packed_weight_grad(dy, out=into[1], bias_grad=into[2])
        z.zero_packed_weight_grad(dy, out=into[1], bias_grad=into[2], accumulate=True)
        return into

    fresh = lambda: [torch.full(s, math.nan, device=DEV) for s in ((m, n), (80, 96), (80,))]
    want = [(x.q.double() @ w.q.double().T).float() * x.scale[:, None] * w.scale + w.scale,
            (2 * (dy.double().T @ values(z))).float(), (2 * dy.double().sum(0)).float()]
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))
    assert same(step(fresh()))
    torch.cuda.synchronize()
    outs, graphs = [fresh(), fresh()], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append(g)
    for turn in range(3):
        for o, g in zip(outs, graphs):
            for t in o:
                t.fill_(5)
            g.replay()
            x[:70].zero_packed_linear(w)
            z[:4000].zero_packed_weight_grad(dy[:4000], bias_grad=torch.empty(80, device=DEV))
            torch.cuda.synchronize()
            assert same(o), turn
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step(fresh()))
    torch.cuda.synchronize()
    assert all(same(o) for o in got)


def test_same_bits_every_time():
    """Whatever runs beside it, and in whatever order blocks end."""
    g = gen(3)
    x = ZeroPacked(5000, 700).zero_packed_write(torch.randn(5000, 700, generator=g, device=DEV))
    dy = torch.randn(5000, 300, generator=g, device=DEV).half()
    db = torch.empty(300, device=DEV)
    want, want_b = x.zero_packed_weight_grad(dy, bias_grad=db).clone(), db.clone()
    other = torch.cuda.Stream()
    noise = torch.randn(2048, 2048, device=DEV)
    for _ in range(10):
        with torch.cuda.stream(other):
            noise @ noise
        got = x.zero_packed_weight_grad(dy, bias_grad=db)
        assert torch.equal(got, want) and torch.equal(db, want_b)
    torch.cuda.synchronize()


def test_rows_of_one_buffer():
    """Slices of packed rows (sequences behind each other) are packed rows: written, read and multiplied by themselves, the
    rows beside them left as they were."""
    p = ZeroPacked(100, 50)
    p._q.fill_(7), p.scale.fill_(3)
    x = torch.randn(100, 50, generator=gen(1), device=DEV)
    p[20:61].zero_packed_write(x[20:61])
    assert (p._q[:20] == 7).all() and (p._q[61:] == 7).all() and (p.scale[:20] == 3).all() and (p.scale[61:] == 3).all()
    p.zero_packed_write(x)
    w, dy = random_packed(30, 50, 2), whole_dy(41, 30, BF16, 3)
    y = p.zero_packed_linear(w)
    assert torch.equal(p[20:61].zero_packed_linear(w), y[20:61])
    assert torch.equal(p[60:61].zero_packed_linear(w), y[60:61])
    alone = ZeroPacked(41, 50).zero_packed_write(x[20:61])
    assert torch.equal(p[20:61].zero_packed_weight_grad(dy), alone.zero_packed_weight_grad(dy))
    assert p[5:5].zero_packed_linear(w).shape == (0, 30) and p[:].nbytes == p.nbytes
    for bad in (3, slice(0, 10, 2), [1, 2]):
        with pytest.raises(ValueError):
            p[bad]


def test_binding_checks():
    p, q = ZeroPacked(4, 40), torch.zeros(4, 48, dtype=torch.int8, device=DEV)
    s = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError, match="bytes"):
        ZeroPacked.of(q, s, 49)
    with pytest.raises(ValueError, match="bytes"):
        ZeroPacked.of(q[:, :40], s, 40)
    with pytest.raises(ValueError, match="rule"):
        ZeroPacked(4, 40, 3)
    with pytest.raises(zpm.ZeroError, match="16-byte"):
        ZeroPacked.of(q[:, 8:24], s).zero_packed_read()
    with pytest.raises(ValueError, match="not ZeroPacked"):
        p.zero_packed_linear(q)
    with pytest.raises(ValueError, match="accumulate"):
        p.zero_packed_weight_grad(torch.zeros(4, 8, dtype=BF16, device=DEV), accumulate=True)
    with pytest.raises(ValueError, match="accumulate"):
        p.zero_packed_input_grad(torch.zeros(4, 4, dtype=BF16, device=DEV), accumulate=True)
    with pytest.raises(ValueError, match="dtype"):
        p.zero_packed_read(dtype=torch.float64)
    with pytest.raises(ValueError, match="is on cpu"):
        p.zero_packed_write(torch.zeros(4, 40))
    with pytest.raises(zpm.ZeroError, match="dy must be"):
        p.zero_packed_weight_grad(torch.zeros(4, 8, device=DEV))
    with pytest.raises(zpm.ZeroError, match="same size"):
        p.zero_packed_write(torch.zeros(5, 40, device=DEV))


def test_leaves_of_an_autograd_graph():
    """Parameters that an eager autograd graph holds are read as they are; a backward pass captured while that graph lives
    works on its own buffers."""
    w = torch.randn(64, 96, generator=gen(1), device=DEV).to(BF16).requires_grad_()
    x = torch.randn(50, 96, generator=gen(2), device=DEV).to(BF16)
    loss = (x @ w.t()).float().square().mean()          # alive during the capture
    wp, xp = ZeroPacked(64, 96).zero_packed_write(w), ZeroPacked(50, 96).zero_packed_write(x)
    dy = torch.randn(50, 64, generator=gen(3), device=DEV).to(BF16)
    want, want_x = xp.zero_packed_weight_grad(dy), wp.zero_packed_input_grad(dy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dw, dx = xp.zero_packed_weight_grad(dy), wp.zero_packed_input_grad(dy)
    for _ in range(3):
        dw.zero_(), dx.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want) and torch.equal(dx, want_x)
    loss.backward()
    assert w.grad.isfinite().all()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [1, 9, 700])
def test_act_without_columns(rows, gated):
    """Packed results without columns, whose q may be NULL, get the scales of rows of zeros, as zero_packed_write gives them."""
    stream = torch.cuda.current_stream().cuda_stream
    x = _abi.zero_matrix_t(None, rows, 0, 0, _abi.ZERO_BF16)
    sx, sy, sw = (torch.full((rows,), math.nan, device=DEV) for _ in range(3))
    none = lambda s: _abi.zero_packed_t(None, s.data_ptr(), rows, 0, 16, POW2)
    zpm.zero_packed_write(x, none(sw), stream)
    zpm.zero_packed_act(SILU, gated, x, none(sx), None, none(sy), stream)
    assert not sw.any() and not sx.any() and not sy.any()
    sx.fill_(math.nan)
    zpm.zero_packed_act(GELU, gated, x, none(sx), x, None, stream)
    assert not sx.any()
    sy.fill_(math.nan)
    zpm.zero_packed_act(GELU, gated, x, None, None, none(sy), stream)
    assert not sy.any()
    # and what follows is the bias, not NaN
    w, b = ZeroPacked(6, 0), torch.arange(6, device=DEV, dtype=F32)
    w.scale.fill_(1)
    y = torch.empty(rows, 6, device=DEV)
    zpm.zero_packed_linear(none(sy), w._desc, matrix(b, "b"), matrix(y, "y"), None, 0, stream)
    assert torch.equal(y, b.expand(rows, 6))

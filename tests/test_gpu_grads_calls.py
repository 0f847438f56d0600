"""The gradient-list operators over several steps of one handle: what one call leaves for the next, calls captured into
graphs beside eager ones, and other streams.  Tolerances are those of tests/test_gpu_grads.py."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_grads import EACH, GLOBAL, H, L2, MAX, _gpu, bits, c_of, check_norms, emulate, rand  # noqa: F401
from zero_partitioned_mixed_reduce_amd import ZeroError, ZeroGrads, _abi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [L2, MAX])
def test_empty_tensors_norms_are_of_this_call(kind):
    """An empty tensor's results are 0 in every call, whatever an exchange has put there since the last one."""
    e = torch.empty(0, device="cuda")
    for grads in ([rand(1, 700, torch.float32), e, rand(2, 20_000, torch.float32), e.view(3, 0)], [e, e.view(0, 4)], [e] * 700,
                  [rand(3, 5, torch.float32)] + [e] * 700):
        h = ZeroGrads(grads, out=[torch.empty_like(g) for g in grads])
        none = torch.tensor([g.numel() == 0 for g in grads], device="cuda")
        for _ in range(2):
            h.zero_grads_norm(kind, per_tensor=True)
            assert (h.tensor_acc[none] == 0).all() and (h.norms[none] == 0).all()
            check_norms(h, grads, kind, 1.0)
            h.tensor_acc.add_(9.0)                    # what other ranks hold of these tensors
            h.zero_grads_clip(1.0, EACH)
            h.norms.fill_(7.0)
        h.zero_grads_clip_norm(1.0, kind, scope=EACH)
        assert (h.tensor_acc[none] == 0).all() and (h.norms[none] == 0).all()


@pytest.mark.parametrize("kind", [L2, MAX])
def test_exchanges_step_after_step(kind):
    """Two ranks' lists in one order, some tensors held by one rank alone: every step clips by that step's norms."""
    cuts = [(9000, 0), (0, 300), (500, 700), (0, 0), (2049, 1)]
    limit = 1e-3
    grads = [[torch.zeros(n[r], device="cuda") for n in cuts] for r in (0, 1)]
    hs = [ZeroGrads(g, out=[torch.empty_like(x) for x in g]) for g in grads]
    for step in range(3):
        for r, g in enumerate(grads):
            for i, x in enumerate(g):
                x.copy_(rand(100 * step + 10 * i + r, x.numel(), torch.float32, 1e-3 * 2.0 ** (2 - step)))
        for h in hs:
            h.zero_grads_norm(kind, per_tensor=True)
        for a, b in ((hs[0].acc, hs[1].acc), (hs[0].tensor_acc, hs[1].tensor_acc)):
            joint = a + b if kind == L2 else torch.maximum(a, b)
            a.copy_(joint)
            b.copy_(joint)
        for h in hs:
            h.zero_grads_clip(limit, EACH)
        for i in range(len(cuts)):
            d = torch.cat([grads[0][i], grads[1][i]]).cpu().double()
            norm = 0.0 if d.numel() == 0 else float(d.abs().max()) if kind == MAX else math.sqrt(math.fsum((d * d).tolist()))
            for h, g in zip(hs, grads):
                want = g[i].cpu().double() * c_of(norm, limit)
                assert ((h._out[i].cpu().double() - want).abs() <= 4 * H * want.abs() + 2.0 ** -149).all(), (step, i)


def test_bind_refuses_negated_views():
    """Sources and destinations whose memory holds the opposite sign, as the constructor refuses them."""
    z = torch.complex(torch.ones(300), torch.full((300,), 2.0)).cuda()
    x, y = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
    for plain, neg in ((z.imag, z.conj().imag), (y, torch._neg_view(y))):
        into = torch.zeros(4 + plain.numel(), device="cuda")
        for out, bad in ((None, ([x, neg], None)), (into, ([x, neg], into)), ([into[:4], into[4:]], ([x, neg], [into[:4], into[4:]]))):
            with pytest.raises(ValueError, match="negated"):
                ZeroGrads([x, neg], out=out)
            h = ZeroGrads([x, plain], out=out)
            with pytest.raises(ValueError, match="negated"):
                h.zero_grads_bind(*bad)
            h.zero_grads_norm()                       # the plan's own addresses stand
            assert float(h.acc) == 4.0 + float((plain.cpu().double() ** 2).sum())
    flat = torch.zeros(4, device="cuda")
    h = ZeroGrads([x], out=flat)
    with pytest.raises(ValueError, match="negated"):
        h.zero_grads_bind([x], torch._neg_view(flat))
    h = ZeroGrads([x], out=[flat])
    with pytest.raises(ValueError, match="negated"):
        h.zero_grads_bind([x], [torch._neg_view(flat)])
    for bad in ([None], [3], [x.to_sparse()], [x.cpu()]):
        with pytest.raises(ValueError):
            h.zero_grads_bind(bad, [flat])


def refused_by_the_device(h, out):
    """A clip that finds no norm of the values on the device: nothing written, and the query says so."""
    assert all((o == 7).all() for o in out)
    with pytest.raises(ZeroError) as e:
        h.query()
    assert e.value.status == _abi.ZERO_ESTATE


def captured(*calls):
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f in calls:
            f()
    return g


def two_lists(seed=1):
    grads = [rand(seed + i, n, torch.bfloat16) for i, n in enumerate((5000, 70_000, 3, 900))]
    out = [torch.full((g.numel(),), 7.0, device="cuda") for g in grads]
    return grads, out, ZeroGrads(grads, out=out)


def renew(grads, out, seed):
    for i, (g, o) in enumerate(zip(grads, out)):
        g.copy_(rand(seed + i, g.numel(), torch.bfloat16))
        o.fill_(7.0)


def check_clipped(h, grads, out, kind, inv, max_norm, scope=GLOBAL):
    """The list as this norm, inverse scale and limit clip it, by the formula and, given the coefficient, to the bit."""
    sizes, whole = check_norms(h, grads, kind, inv, scope == EACH)
    q = h.query()
    assert abs(q["norm"] - whole) <= 1.25 * H * whole and not q["found_inf"]
    for i, (g, o) in enumerate(zip(grads, out)):
        acc = float(h.tensor_acc[i])
        coef = (float(np.float32(c_of(acc if kind == MAX else math.sqrt(acc), max_norm))) if scope == EACH else
                float(np.float32(c_of(q["norm"], max_norm))))
        assert (bits(o) == bits(emulate(g, inv, coef, torch.float32))).all()
    return q


def test_captured_norm_and_clip_beside_it():
    """The norm in a graph and the clip at once or in another graph, step after step, as around an exchange that is not
    captured: the clip goes by the norm that ran last, its kind and inverse scale."""
    for kind, inv, scope in ((L2, 0.5, GLOBAL), (MAX, 0.25, EACH)):
        grads, out, h = two_lists()
        norm = captured(lambda: h.zero_grads_norm(kind, inv, per_tensor=True))
        h.zero_grads_clip(1e-3, scope)                # the graph has not run: there is no norm
        refused_by_the_device(h, out)
        clip = captured(lambda: h.zero_grads_clip(1e-3, scope))
        with pytest.raises(ZeroError):                # nor has this one
            h.query()
        for step in range(4):
            renew(grads, out, 100 * step)
            norm.replay()
            if step % 2:
                clip.replay()
            else:
                h.zero_grads_clip(1e-3, scope)
            check_clipped(h, grads, out, kind, inv, 1e-3, scope)
            for o in out:
                o.fill_(7.0)
            if step % 2:
                h.zero_grads_clip(1e-3, scope)        # a second clip of the same norm
            else:
                clip.replay()
            refused_by_the_device(h, out)
        # an eager norm of another kind and scale, then the captured clip, and the other way round
        for first, k, i in ((lambda: h.zero_grads_norm(3 - kind, 2.0, per_tensor=True), 3 - kind, 2.0), (norm.replay, kind, inv)):
            for then in (clip.replay, lambda: h.zero_grads_clip(1e-3, scope)):
                renew(grads, out, 7)
                h.zero_grads_norm(kind, inv, per_tensor=True)
                norm.replay()
                first()
                then()
                check_clipped(h, grads, out, k, i, 1e-3, scope)


def test_replays_between_a_norm_and_its_clip():
    """Replayed calls count as calls: one that takes another norm replaces the first, one that writes ends it."""
    grads, out, h = two_lists()
    other = captured(lambda: h.zero_grads_norm(MAX, 0.25))
    write = captured(lambda: h.zero_grads_scale(3.0))
    renew(grads, out, 5)
    h.zero_grads_norm(L2, 0.5, per_tensor=True)
    other.replay()
    h.zero_grads_clip(1e-3)
    check_clipped(h, grads, out, MAX, 0.25, 1e-3)
    renew(grads, out, 6)
    h.zero_grads_norm(L2, 0.5, per_tensor=True)
    other.replay()
    h.zero_grads_clip(1e-3, EACH)                     # the norm that ran last has no per-tensor norms
    refused_by_the_device(h, out)
    h.zero_grads_norm(L2, 0.5, per_tensor=True)
    write.replay()
    for o in out:
        o.fill_(7.0)
    h.zero_grads_clip(1e-3)
    refused_by_the_device(h, out)
    h.zero_grads_clip_norm(1e-3, L2, 0.5)             # both in one call are never apart
    check_clipped(h, grads, out, L2, 0.5, 1e-3)
    both = captured(lambda: h.zero_grads_norm(L2, 2.0, per_tensor=True), lambda: h.zero_grads_clip(1e-3, EACH))
    for step in range(3):
        renew(grads, out, 50 + step)
        both.replay()
        check_clipped(h, grads, out, L2, 2.0, 1e-3, EACH)
        h.zero_grads_norm(MAX)
    # without any norm in a graph the host knows, and says so at once
    grads, out, h = two_lists()
    captured(lambda: h.zero_grads_scale(1.0))
    with pytest.raises(ZeroError) as e:
        h.zero_grads_clip(1.0)
    assert e.value.status == _abi.ZERO_ESTATE
    h.zero_grads_norm()
    captured(lambda: h.zero_grads_scale(1.0))         # has not run: the norm stands
    h.zero_grads_clip(1e-3)
    check_clipped(h, grads, out, L2, 1.0, 1e-3)


def test_bind_in_a_graph_binds_when_replayed():
    """Eager calls work on the list bound last by what has run; the handle keeps every list that its table may name."""
    import weakref

    def make(v):
        return [torch.full((n,), v, device="cuda") for n in (5000, 7)], [torch.zeros(n, device="cuda") for n in (5000, 7)]

    def holds(out, v):
        return all((o == v).all() for o in out)

    def kept(refs):
        return [r() is not None for r in refs]

    (a, oa), (b, ob) = make(1.0), make(10.0)
    h = ZeroGrads(a, out=oa)
    ra, rb = [[weakref.ref(t) for t in x] for x in (a + oa, b + ob)]
    g = captured(lambda: h.zero_grads_bind(b, ob), lambda: h.zero_grads_scale(2.0))
    late = captured(lambda: h.zero_grads_scale(7.0))  # has no bind of its own
    watch = [t.view(-1) for t in oa], [t.view(-1) for t in ob]
    del a, b, oa, ob
    assert all(kept(ra)) and all(kept(rb))
    h.zero_grads_scale(3.0)                           # the graph has not run
    assert holds(watch[0], 3.0) and holds(watch[1], 0.0)
    g.replay()
    assert holds(watch[0], 3.0) and holds(watch[1], 20.0)
    h.zero_grads_scale(5.0)
    assert holds(watch[0], 3.0) and holds(watch[1], 50.0)
    c, oc = make(100.0)
    h.zero_grads_bind(c, oc)
    assert not any(kept(ra[:2])) and all(kept(rb))    # oa are held by their views here
    for _ in range(3):
        h.zero_grads_scale(2.0)
        assert holds(oc, 200.0) and holds(watch[0], 3.0)
        late.replay()                                 # works on what is bound now
        assert holds(oc, 700.0)
        g.replay()
        assert holds(watch[1], 20.0) and holds(oc, 700.0)
        late.replay()
        assert holds(watch[1], 70.0) and holds(oc, 700.0)
        h.zero_grads_norm(per_tensor=True)
        assert float(h.acc) == 5007 * 100.0
        h.zero_grads_bind(c, oc)
    torch.cuda.synchronize()
    h.close()
    assert not any(kept(rb[:2]))


def test_graphs_and_lists_that_overlap():
    """A list with overlapping tensors takes norms only, and neither a replay nor a later bind brings it to a call that
    writes."""
    x, y = torch.ones(3000, device="cuda"), torch.ones(3000, device="cuda")

    def invalid(f, *a):
        with pytest.raises(ZeroError) as e:
            f(*a)
        assert e.value.status == _abi.ZERO_EINVAL

    h = ZeroGrads([x, y])
    g = captured(lambda: h.zero_grads_scale(2.0))
    invalid(h.zero_grads_bind, [x, x])                # the graph would write x twice
    captured(h.zero_grads_norm, lambda: invalid(h.zero_grads_bind, [y, y]))
    g.replay()
    assert (x == 2).all() and (y == 2).all()
    h = ZeroGrads([x, y])
    g = captured(lambda: h.zero_grads_bind([x, x]), lambda: h.zero_grads_norm())
    h.zero_grads_norm()
    invalid(h.zero_grads_clip, 1.0)                   # a replay may have come before
    invalid(h.zero_grads_scale, 3.0)
    h.zero_grads_bind([x, y])
    invalid(h.zero_grads_scale, 3.0)
    g.replay()
    assert float(h.acc) == 2 * 4.0 * 3000 and (x == 2).all() and (y == 2).all()
    h = ZeroGrads([x, x])                             # bound apart at once, it writes
    h.zero_grads_bind([x, y])
    h.zero_grads_scale(0.5)
    assert (x == 1).all() and (y == 1).all()


def test_workspace_of_a_handle_closed_while_another_stream_works():
    """The workspace's memory is not given to others before every stream that the handle used is done with it."""
    grads = [rand(i, 5000 + i, torch.float32) for i in range(40)]
    side = torch.cuda.Stream()
    h = ZeroGrads(grads, out=[torch.empty_like(g) for g in grads])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                 # some milliseconds of work in front of the handle's
        h.zero_grads_clip_norm(1e-3, per_tensor=True)
    keep, at, size = h._out, h.workspace.data_ptr(), h.workspace.numel()
    h.close()
    del h
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query() and all(t.data_ptr() != at for t in others)
    side.synchronize()
    norm = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))
    coef = c_of(norm, 1e-3)
    for o, g in zip(keep, grads):
        want = g.double() * coef
        assert ((o.double() - want).abs() <= 4 * H * want.abs() + 2.0 ** -149).all()


@pytest.mark.parametrize("sizes", [(5000, 0, 700), (0, 0)])
def test_a_captured_clip_has_not_run(sizes):
    """There is nothing to query before the first replay; afterwards every replay gives what the eager call gives."""
    grads = [rand(i, n, torch.float32) for i, n in enumerate(sizes)]
    h = ZeroGrads(grads, out=[torch.empty_like(g) for g in grads])
    g = captured(lambda: h.zero_grads_clip_norm(1e-3, scope=EACH))
    with pytest.raises(ZeroError) as e:
        h.query()
    assert e.value.status == _abi.ZERO_ESTATE
    for step in range(3):
        for i, x in enumerate(grads):
            x.copy_(rand(10 * step + i, x.numel(), torch.float32))
        h.tensor_acc.fill_(9.0)
        g.replay()
        q, each, out = h.query(), h.tensor_acc.clone(), [o.clone() for o in h._out]
        check_norms(h, grads, L2, 1.0)
        h.zero_grads_clip_norm(1e-3, scope=EACH)
        assert h.query() == q and torch.equal(h.tensor_acc, each)
        assert all((bits(a) == bits(b)).all() for a, b in zip(out, h._out))

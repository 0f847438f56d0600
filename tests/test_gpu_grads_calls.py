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

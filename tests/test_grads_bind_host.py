"""What a bound list is checked for by the Python binding of the gradient lists, on the CPU: it has to be what the plan
was made of, and nothing that the plan would have refused."""
import pytest
import torch

from zero_partitioned_mixed_reduce_amd.grads import _Layout, describe


def negated(n):
    """A lazily negated view of n elements beside the same storage seen plainly."""
    z = torch.complex(torch.ones(n), torch.full((n,), 2.0))
    return z.imag, z.conj().imag


def test_bound_lists_are_not_negated_views():
    one, two = torch.ones(4), torch.ones(4)
    for plain, neg in ((negated(4)), (negated(1)), (one, torch._neg_view(two))):
        assert neg.is_neg() and plain.stride() == neg.stride() and plain.shape == neg.shape
        with pytest.raises(ValueError, match="negated"):
            describe(0, neg, None)
        layout = _Layout([one, plain])
        assert layout.addresses([two, plain], "tensors") == [two.data_ptr(), plain.data_ptr()]
        with pytest.raises(ValueError, match="resolve_neg"):
            layout.addresses([two, neg], "tensors")


def test_bound_lists_are_those_of_the_plan():
    a, wide = torch.zeros(6, dtype=torch.bfloat16), torch.zeros(4, 10)
    layout = _Layout([a, wide[:, :5]])
    assert layout.addresses([a.view(2, 3), wide[:, 5:]], "tensors") == [a.data_ptr(), wide[:, 5:].data_ptr()]
    for x, y in ((a.half(), wide[:, :5]), (a[:5], wide[:, :5]), (a, wide[:, :6]), (a, wide[:, :5].contiguous()),
                 (a, wide.t()[:5]), (a, wide.view(20, 2)[::2]), (a.float(), wide[:, :5]), 
                 (None, wide[:, :5]), (a, 3), (a.to_sparse(), wide[:, :5]), (a, torch.eye(4, 10).to_sparse_csr()),
                 (a, torch.eye(4, 10).to_sparse())):
        with pytest.raises(ValueError):
            layout.addresses([x, y], "tensors")
    with pytest.raises(ValueError, match="2 tensors"):
        layout.addresses([a], "tensors")

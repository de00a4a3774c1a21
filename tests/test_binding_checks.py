"""Checks of tensors in the binding that need no GPU."""
import pytest
import torch

from gaussian_mixture_sequence_gb300 import gma


class _Cuda(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = True


def test_an_empty_tensor_is_not_an_absent_one():
    none = torch.empty(0, dtype=torch.int32).as_subclass(_Cuda)
    with pytest.raises(ValueError, match=r"lengths has shape \(0,\), expected \(2,\)"):
        gma._p(none, "lengths", (2,), torch.int32, 0, optional=True)
    with pytest.raises(ValueError, match="state_in has shape"):
        gma._p(none.view(0, 3), "state_in", (2, 3), torch.float32, 0, optional=True)
    assert gma._p(None, "lengths", (2,), torch.int32, 0, optional=True) is None
    # sequences of no rows have empty buffers
    assert gma._p(torch.empty(2, 0, 4).as_subclass(_Cuda), "x", (2, 0, 4), torch.float32, 0) is None

"""What clipping and reordering write in place is known to autograd: a backward pass that saved such a
tensor is refused, as after torch's own in-place operations."""
import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def saved(n=12):
    """A leaf, a tensor made from it, and a result whose backward pass needs that tensor."""
    leaf = torch.randn(n, 5, device=DEV, requires_grad=True)
    mid = leaf * 2.0
    return leaf, mid, mid.square().sum()


def test_clipped_gradients(gpu_lib):
    for out in (None, "other"):
        leaf, mid, end = saved()
        if out is None:
            flce.clip_grad_norm([mid], 0.1)
        else:
            flce.clip_grad_norm([torch.ones_like(leaf)], 0.1, out=[mid.detach()])
        with pytest.raises(RuntimeError, match="inplace"):
            end.backward()
    # what is only read keeps its version
    leaf, mid, end = saved()
    flce.grad_norm([mid])
    flce.clip_grad_norm([mid], 0.1, out=[torch.empty(12, 5, device=DEV)])
    end.backward()
    assert torch.equal(leaf.grad, 8 * leaf.detach())
    with torch.inference_mode():  # (tensors without a version)
        assert flce.clip_grad_norm([torch.ones(7, device=DEV)], 1.0).item() > 2.6


def test_clipped_parameters(gpu_lib):
    p = torch.nn.Parameter(torch.randn(12, 5, device=DEV))
    (p * p).sum().backward()
    end = (p.grad.requires_grad_(False) * torch.ones(12, 5, device=DEV, requires_grad=True)).sum()  # saves the gradient
    flce.clip_grad_norm_([p], 0.1)
    with pytest.raises(RuntimeError, match="inplace"):
        end.backward()

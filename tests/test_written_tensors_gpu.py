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


def test_reordered_states(gpu_lib):
    parents = torch.tensor([[1, 0, 2], [2, 2, 1]], dtype=torch.int32, device=DEV)
    leaf, mid, end = saved(6)
    with torch.no_grad():
        flce.beam_reorder([mid], parents)
    with pytest.raises(RuntimeError, match="inplace"):
        end.backward()
    leaf, mid, end = saved(6)
    flce.beam_reorder([torch.zeros(6, 5, device=DEV)], parents, out=[mid.detach()])
    with pytest.raises(RuntimeError, match="inplace"):
        end.backward()
    leaf, mid, end = saved(6)
    out = flce.beam_reorder([mid], parents, out=[torch.empty(6, 5, device=DEV)])[0]  # what is only read
    end.backward()
    assert torch.equal(leaf.grad, 8 * leaf.detach()) and not out.requires_grad
    with torch.inference_mode():
        s = torch.arange(6.0, device=DEV)[:, None]
        assert flce.beam_reorder([s], parents)[0].flatten().tolist() == [1, 0, 2, 5, 5, 4]


def test_reordering_what_needs_a_gradient_is_refused(gpu_lib):
    """Its gradient would not know of the new order."""
    parents = torch.tensor([[1, 0, 2], [2, 2, 1]], dtype=torch.int32, device=DEV)
    leaf, mid, _ = saved(6)
    before = mid.detach().clone()
    for states, out in (([mid], None), ([leaf], None), ([torch.zeros(6, 5, device=DEV)], [mid])):
        with pytest.raises(RuntimeError, match="no_grad"):
            flce.beam_reorder(states, parents, out=out)
    assert torch.equal(mid, before)

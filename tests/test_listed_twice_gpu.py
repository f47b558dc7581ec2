"""Tensors that are listed twice, or written for one entry while another reads them: two blocks would work on
the same elements in no order, so such lists are refused before any launch."""
import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_tied_parameters_count_once(gpu_lib):
    """A weight that two modules share is one parameter, however often it is listed."""
    p, q = (torch.nn.Parameter(torch.zeros(300, 7, device=DEV)) for _ in range(2))
    p.grad, q.grad = torch.randn(300, 7, device=DEV), torch.randn(300, 7, device=DEV)
    want = [p.grad.double(), q.grad.double()]
    norm = torch.cat([w.flatten() for w in want]).norm()
    total = flce.clip_grad_norm_([p, q, p, p], 0.5)
    # (the bounds of the other clipping tests: 20 and 24 steps of 2^-24)
    assert abs(total.item() - norm.item()) <= 20 * 2.0 ** -24 * norm.item()
    f = 0.5 / (norm + 1e-6)
    for t, w in zip((p, q), want):
        assert bool(((t.grad.double() - w * f).abs() <= 25 * 2.0 ** -24 * (w * f).abs()).all())


def test_clipping_refuses(gpu_lib):
    a, b, c = (torch.ones(50, device=DEV) for _ in range(3))
    before = flce.flce_kernel_launches()
    for grads, out in [([a, a], None), ([a, b, a.view(5, 10)], None), ([a, b], [c, c]), ([a, b], [b, a]), ([a, b], [b, c]),
                       ([a, a], [a, b]), ([a, a], [b, a])]:
        with pytest.raises(ValueError):
            flce.clip_grad_norm(grads, 1.0, out=out)
    assert flce.flce_kernel_launches() == before
    # what is only read may be listed twice, and tensors without elements may have one address
    assert abs(flce.grad_norm([a, a]).item() - 10.0) <= 20 * 2.0 ** -24 * 10.0
    flce.clip_grad_norm([a, a], 1.0, out=[b, c])
    assert torch.equal(b, c)
    flce.clip_grad_norm([a, a[:0], a[:0]], 1.0)
    flce.clip_grad_norm([a, b], 0.1, out=[a, c])


def test_reordering_refuses(gpu_lib):
    parents = torch.tensor([[1, 0], [0, 1]], dtype=torch.int32, device=DEV)
    a, b, c = (torch.arange(12.0, device=DEV).view(4, 3).clone() for _ in range(3))
    before = flce.flce_kernel_launches()
    for states, out in [([a, a], None), ([a, b, a[:]], None), ([a, b], [c, c]), ([a, b], [b, a]), ([a, b], [b, c]), ([a, a], [a, b])]:
        with pytest.raises(ValueError):
            flce.beam_reorder(states, parents, out=out)
    assert flce.flce_kernel_launches() == before
    # one state into two others, parts of one buffer, states without elements at one address
    flce.beam_reorder([a, a], parents, out=[b, c])
    assert torch.equal(b, c) and b[:, 0].tolist() == [3.0, 0.0, 6.0, 9.0]
    flce.beam_reorder([a[:, :1], a[:, 1:], a[:, :0], a[:, :0]], parents)
    assert torch.equal(a, b)
    flce.beam_reorder([a, b], parents, out=[a, c])
    assert torch.equal(a, c) and a[:, 0].tolist() == [0.0, 3.0, 6.0, 9.0]

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

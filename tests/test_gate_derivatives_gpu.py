"""Gradients of saturated gates. With e = exp(-k |g|) (k = 1 for the sigmoid, 2 for tanh) the
activation's derivative is k^2 e / (1 + e)^2: it keeps its relative precision where the value itself is
1 to all its bits.

The bound: the gate's gradient is that of a linear gate times the derivative, so it has the bound of
that one, plus the derivative's own rounding, 2 steps for the exponential (and k |g| rounded: exact for
k = 1 and 2), and one each for 1 + e, its reciprocal and two products: 16 steps with room."""
import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce
from tests import block_norm_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
GATES = [0.0, 0.5, -1.0, 3.0, -6.0, 8.0, 12.0, -12.0, 17.0, 25.0, 40.0, -40.0, 60.0, -80.0]


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("rows", [1, 4, 24])
@pytest.mark.parametrize("post,norm,D", [(False, "rms", 512), (True, "rms", 512), (True, "layer", 512), (False, "layer", 77),
                                         (True, "layer", 5120)])
@pytest.mark.parametrize("x", [torch.float32, torch.bfloat16])
def test_saturated_gates(gpu_lib, act, rows, post, norm, D, x):
    g = torch.Generator(device=DEV).manual_seed(rows)
    n = lambda s, t=torch.float32, m=0.0: torch.empty(s, device=DEV, dtype=t).normal_(m, 0.5, generator=g)  # noqa: E731
    N = 24
    gate = torch.tensor(GATES, device=DEV).repeat(rows * D // len(GATES) + 1)[:rows * D].view(rows, D).contiguous()
    w1 = n((D,), m=1.0) if post else None
    b1 = n((D,)) if post and norm == "layer" else None
    t = [n((N, D), x, 0.2), n((N, D)), n((D,), m=1.0)]
    gate.requires_grad_()
    h, y = flce.block_norm(*t, gate=gate, post_weight=w1, post_bias=b1, gate_activation=act, norm=norm, scale=0.6, eps=1e-5)
    stats = h.grad_fn.saved_tensors[-1]
    dh, dy = n((N, D)), n((N, D), x)
    got, = torch.autograd.grad((h, y), gate, (dh, dy))
    gate = gate.detach()
    lin, bound = ref.backward(t[0], h.detach(), gate, w1, b1, t[2], None, stats, dh, dy, norm, 0.6, "none", 0.0)["dgate"]
    k = 2.0 if act == "tanh" else 1.0
    e = torch.exp(-k * gate.double().abs())
    da = k * k * e / (1 + e) ** 2
    # below fp32's normal range a result is exact to half its smallest number, of up to 24 terms
    ref.close(got, lin * da, bound * da + 16 * ref.U * (lin * da).abs() + 64 * 2.0 ** -149, "dgate")

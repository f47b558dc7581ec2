"""Factors of clipping that fp32 holds with few bits or not at all: gradients near the end of its range,
clipped to a small norm. Bounds as in test_grad_clip_gpu.py: the norm's error, the factor's and two
products' rounding, half a step of the output's type."""
import math

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p", [2.0, math.inf])
@pytest.mark.parametrize("std,max_norm,scale", [(1e36, 1e-3, 1.0), (1e36, 1e-9, 1.0), (3e35, 1e-6, -0.5), (1e30, 1e-10, 1.0),
                                                (1e-30, 1e-3, 1.0), (1e-36, 1e-3, 1e30)])
def test_small_factors(gpu_lib, dtype, p, std, max_norm, scale):
    g = torch.Generator(device=DEV).manual_seed(1)
    grads = [torch.empty(n, device=DEV).normal_(0, std, generator=g).to(dtype) for n in (40, 3000, 1)]
    t = torch.cat([v.double() for v in grads])
    norm = abs(scale) * float(t.square().sum().sqrt() if p == 2.0 else t.abs().max())
    f = scale * min(1.0, max_norm / (norm + 1e-6))
    want = [v.double() * f for v in grads]
    outs = [torch.empty_like(v) for v in grads], [torch.empty(v.shape, device=DEV) for v in grads], None
    for out in outs:
        total = flce.clip_grad_norm(grads, max_norm, norm_type=p, grad_scale=scale, out=out)
        assert abs(total.item() - norm) <= 20 * U * norm
        for o, w in zip(out or grads, want):
            info = torch.finfo(o.dtype)
            assert bool(((o.double() - w).abs() <= 24 * U * w.abs() + w.abs() * (info.eps / 2) + info.tiny * info.eps).all())

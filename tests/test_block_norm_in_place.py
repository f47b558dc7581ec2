"""h in the residual's own buffer: refused where its rows would fall on residual rows that are still to be
read (on the CPU), right at unaligned widths (on the GPU)."""
import ctypes

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce


def _forward(N, ld_residual, h):
    d = flce.FlceBlockNormDesc(N=N, D=64, x=0x10000, residual=0x20000, weight=0x30000, ld_x=64, ld_residual=ld_residual,
                               eps=1e-6, scale=1.0)
    return flce.load_library().flce_block_norm_forward(ctypes.byref(d), h, 0x50000, 0x60000, None)


def test_wider_residual_rows_are_refused():
    assert _forward(4, 65, 0x20000) == _forward(2, 128, 0x20000) == 1
    assert flce.flce_last_error_detail().startswith("h: ")


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none")
def test_what_is_not_refused():
    """These go on to the check of the device."""
    assert _forward(4, 64, 0x20000) == _forward(1, 65, 0x20000) == _forward(4, 65, 0x40000) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("D", [77, 264, 5121])
@pytest.mark.parametrize("r", [torch.bfloat16, torch.float32])
def test_unaligned_widths_in_place(gpu_lib, D, r):
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.empty(700, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    res = torch.empty(700, D, device="cuda", dtype=r).normal_(generator=g)
    w = torch.empty(D, device="cuda").normal_(1.0, 0.2, generator=g)
    h, y = flce.block_norm(x, res, w, norm="layer", scale=0.5)
    y2 = torch.empty_like(x)
    d = flce.FlceBlockNormDesc(N=700, D=D, x=x.data_ptr(), residual=res.data_ptr(), weight=w.data_ptr(), ld_x=D, ld_residual=D,
                               x_dtype=0, residual_dtype=0 if r == torch.bfloat16 else 2, weight_dtype=2, norm=1, eps=1e-6, scale=0.5)
    flce.flce_block_norm_forward(d, res, y2)
    assert torch.equal(res, h) and torch.equal(y2, y)

"""Host-side checks of the block norm: refusals of the C ABI and of the Python call (nothing is
launched), workspace sizes, and the reference's own gradient against differences."""
import ctypes

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce
from tests import block_norm_ref as ref


def _desc(**kw):
    d = flce.FlceBlockNormDesc()
    base = dict(N=4, D=64, x=0x10000, residual=0x20000, weight=0x30000, ld_x=64, ld_residual=64, eps=1e-6, scale=1.0)
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def _fwd(h=0x40000, y=0x50000, stats=0x60000, **kw):
    return flce.load_library().flce_block_norm_forward(ctypes.byref(_desc(**kw)), h, y, stats, None)


def _bwd(h=0x40000, stats=0x60000, dh=0x70000, ld_dh=64, dy=0x80000, ld_dy=64, ws=0x90000, ws_bytes=1 << 30, grads=None,
         **kw):
    g = flce.FlceBlockNormGrads(dx=0xa0000, **(grads or {}))
    return flce.load_library().flce_block_norm_backward(ctypes.byref(_desc(**kw)), h, stats, dh, ld_dh, dy, ld_dy,
                                                        ctypes.byref(g), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), 1), (dict(D=0), 1), (dict(D=16385, ld_x=16385, ld_residual=16385), 9), (dict(N=1 << 30), 9),
    (dict(x=None), 1), (dict(h=None), 1), (dict(y=None), 1), (dict(weight=None), 1), (dict(ld_x=63), 1),
    (dict(ld_residual=1), 1), (dict(x_dtype=3), 1), (dict(residual_dtype=1), 1), (dict(norm=2), 1),
    (dict(gate_activation=3), 1), (dict(gate_rows=1), 1), (dict(gate=0x11000, ld_gate=64), 1),
    (dict(gate=0x11000, ld_gate=64, gate_rows=3), 1), (dict(gate=0x11000, ld_gate=64, gate_rows=8), 1),
    (dict(gate=0x11000, ld_gate=64, gate_rows=2, gate_dtype=1), 1), (dict(gate=0x11000, ld_gate=8, gate_rows=2), 1),
    (dict(bias=0x12000, weight=None, y=None), 1), (dict(post_bias=0x12000), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(weight_offset=float("nan")), 1),
    (dict(x=0x10001), 2), (dict(weight=0x30002, weight_dtype=2), 2), (dict(h=0x40001), 2), (dict(stats=0x60002), 2)])
def test_forward_refuses(kw, status):
    assert _fwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), 1), (dict(stats=None), 1), (dict(dh=None, dy=None), 1), (dict(weight=None), 1), (dict(ld_dy=8), 1),
    (dict(ld_dh=63), 1), (dict(grads=dict(dgate=0xb0000)), 1), (dict(grads=dict(dpost_weight=0xb0000)), 1),
    (dict(grads=dict(dbias=0xb0000)), 1), (dict(ws=None), 1), (dict(ws=0x90010), 2), (dict(ws_bytes=16), 4),
    (dict(dy=0x80001), 2), (dict(grads=dict(dweight=0xb0001)), 2)])
def test_backward_refuses(kw, status):
    assert _bwd(**kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the refusal on a machine without a GB300")
def test_good_arguments_reach_the_device_check():
    assert _fwd() == 3 and _bwd() == 3


def test_workspace_size():
    size = flce.flce_block_norm_workspace_size
    assert size(0, 64) == size(4, 0) == size(4, 16385) == size(4, 64, 3) == size(4, 64, 5) == size(4, 64, -1) == 0
    for N, D in [(1, 1), (1, 4096), (65536, 4096), (100000, 64), (77, 16384)]:
        # four parameter sums for each of at most 152 * 16 blocks
        assert 4 * D * 4 <= size(N, D) <= 4 * 152 * 16 * (D * 4 + 256)
        # a gate for every row needs no sums; groups need at most a few for each worker
        assert size(N, D, N) == size(N, D)
    assert size(65536, 4096, 16) <= size(65536, 4096) + 8 * 152 * 16 * 4096 * 4


@pytest.mark.parametrize("kw,exc", [
    (dict(x=torch.zeros(4, 8)), ValueError), (dict(x=torch.zeros(4, 8, dtype=torch.float64)), TypeError),
    (dict(x=torch.zeros(4, 8, dtype=torch.int32)), TypeError)])
def test_python_refuses(kw, exc):
    with pytest.raises(exc):
        flce.block_norm(**kw)


def test_python_gate_rows():
    from linear_cross_entropy_tcgen05_gb300.norm_ops import _gate_rows
    x2, x3 = torch.zeros(12, 8), torch.zeros(3, 4, 8)
    assert _gate_rows(torch.zeros(8), x3) == 1 and _gate_rows(torch.zeros(3, 1, 8), x3) == 3
    assert _gate_rows(x3, x3) == 12 and _gate_rows(torch.zeros(1, 1, 8), x3) == 1
    assert [_gate_rows(torch.zeros(g, 8), x2) for g in (1, 3, 4, 12)] == [1, 3, 4, 12]
    for gate, x in [(torch.zeros(7), x2), (torch.zeros(5, 8), x2), (torch.zeros(24, 8), x2), (torch.zeros(1, 4, 8), x3),
                    (torch.zeros(2, 1, 8), x3), (torch.zeros(3, 8), x3), (torch.zeros(()), x2)]:
        with pytest.raises(ValueError):
            _gate_rows(gate, x)


def test_packed_descriptors():
    """The packed forms have the layout of the structures."""
    from linear_cross_entropy_tcgen05_gb300 import norm_ops as ops
    assert ops._PACK.size == ctypes.sizeof(flce.FlceBlockNormDesc) == 152
    assert ops._GRADS.size == ctypes.sizeof(flce.FlceBlockNormGrads)
    values = list(range(1, 23)) + [0.5, 0.25, 0.125]
    d = flce.FlceBlockNormDesc.from_buffer_copy(ops._PACK.pack(*values))
    assert [getattr(d, n) for n, _ in d._fields_] == values


def test_module_refuses():
    with pytest.raises(ValueError):
        flce.BlockNorm(8, norm="batch")
    with pytest.raises(ValueError):
        flce.BlockNorm(8, gate_activation="relu")


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "tanh"])
@pytest.mark.parametrize("rows", [0, 1, 3, 6])
def test_reference_gradient_against_differences(norm, act, rows):
    """The formulas' gradients agree with central differences of the formulas' forward."""
    g = torch.Generator().manual_seed(7 + rows)
    N, D, eps, scale, off = 6, 5, 1e-5, 0.6, 0.25
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    t = {"x": r(N, D), "residual": r(N, D), "gate": r(rows, D) if rows else None, "post_weight": r(D), "post_bias": r(D),
         "weight": r(D), "bias": r(D)}
    dh, dy = r(N, D), r(N, D)

    def loss():
        out, _ = ref.forward(**t, norm=norm, eps=eps, scale=scale, act=act, off=off)
        return float((out["h"][0] * dh).sum() + (out["y"][0] * dy).sum())

    out, s = ref.forward(**t, norm=norm, eps=eps, scale=scale, act=act, off=off)
    stats = torch.cat([s["m1"], s["r1"], s["m2"], s["r2"]], 1)
    grads = ref.backward(t["x"], out["h"][0], t["gate"], t["post_weight"], t["post_bias"], t["weight"], t["bias"], stats,
                         dh, dy, norm, scale, act, off)
    for name, v in t.items():
        if v is None:
            continue
        for i in range(0, v.numel(), 3):
            keep, step = v.flatten()[i].item(), 1e-6
            v.view(-1)[i] = keep + step
            up = loss()
            v.view(-1)[i] = keep - step
            down = loss()
            v.view(-1)[i] = keep
            want = grads["d" + name][0].reshape(-1)[i].item()
            # central differences of step 1e-6 in 64 bits: about 1e-9 from rounding, 1e-11 from the cut
            assert abs((up - down) / (2 * step) - want) <= 1e-6 * (1 + abs(want)), (name, i)

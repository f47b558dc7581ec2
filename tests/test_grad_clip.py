"""Host-side checks of gradient clipping: refusals of the C ABI and of the Python call, workspace
sizes. Nothing is launched."""
import ctypes
import math

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce


def _call(grad=0x10000, out=0x10000, n=100, dt=2, odt=2, count=1, max_norm=1.0, p=2.0, eps=1e-6, scale=1.0,
          total=0x20000, ws=0x30000, ws_bytes=1 << 24, table=True):
    words = [grad, out, n, dt | odt << 32]
    t = (ctypes.c_int64 * 4)(*words) if table else None
    return flce.load_library().flce_clip_grad_norm(t, count, max_norm, p, eps, scale, total, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), 1), (dict(table=False), 1), (dict(count=(1 << 24) + 1), 9), (dict(p=1.0), 1), (dict(p=-math.inf), 1),
    (dict(p=math.nan), 1), (dict(max_norm=-1.0), 1), (dict(max_norm=math.nan), 1), (dict(eps=-1.0), 1), (dict(eps=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(total=None), 1), (dict(ws=None), 1), (dict(total=0x20002), 2),
    (dict(ws=0x30010), 2), (dict(n=-1), 1), (dict(n=1 << 40), 9), (dict(dt=3), 1), (dict(odt=3), 1), (dict(grad=0), 1),
    (dict(odt=0), 1), (dict(grad=0x10002, out=0), 2), (dict(out=0x20001, odt=1), 2), (dict(ws_bytes=8), 4)])
def test_refuses(kw, status):
    assert _call(**kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the refusal on a machine without a GB300")
def test_good_arguments_reach_the_device_check():
    assert _call() == 3 and _call(out=0) == 3 and _call(n=0, grad=0) == 3


def test_workspace_size():
    size = flce.flce_clip_grad_norm_workspace_size
    assert size(-1) == size((1 << 24) + 1) == 0
    assert 0 < size(0) <= size(1) <= size(1000) and size(1 << 24) > 0


def test_python_refuses():
    with pytest.raises(ValueError):
        flce.clip_grad_norm([torch.zeros(3)], 1.0)
    with pytest.raises(ValueError):
        flce.clip_grad_norm([torch.zeros(3)], 1.0, out=[])


def test_no_gradients():
    assert flce.clip_grad_norm([], 1.0).item() == 0.0 and flce.grad_norm([]).item() == 0.0
    assert flce.clip_grad_norm_([torch.nn.Parameter(torch.zeros(3))], 1.0).item() == 0.0


def test_dense():
    from linear_cross_entropy_tcgen05_gb300.grad_ops import _dense
    a = torch.zeros(4, 5, 6)
    assert _dense(a) and _dense(a.permute(2, 0, 1)) and _dense(a[1]) and _dense(a[:, :1, :1].contiguous())
    assert not _dense(a[:, 1]) and not _dense(a[..., :3]) and not _dense(torch.zeros(1).expand(4))

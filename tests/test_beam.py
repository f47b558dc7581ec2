"""Host-side checks of the beam-search step: refusals of the C ABI and of the Python calls, state
descriptors, workspace sizes. Nothing is launched."""
import ctypes

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce


def _select(logits=0x10000, dtype=2, B=2, K=3, V=100, ld_batch=300, ld_beam=100, scores=0x20000, finished=None, pad=0, M=3,
            s=0x30000, p=0x40000, t=0x50000, ws=0x60000, ws_bytes=1 << 30):
    return flce.load_library().flce_beam_select(logits, dtype, B, K, V, ld_batch, ld_beam, scores, finished, pad, M, s, p, t,
                                                ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(s=None), 1), (dict(p=None), 1), (dict(t=None), 1), (dict(ws=None), 1),
    (dict(B=0), 1), (dict(K=0), 1), (dict(V=0), 1), (dict(M=0), 1), (dict(K=33), 9), (dict(M=65), 9), (dict(B=65536), 9),
    (dict(B=30000, K=3), 9), (dict(V=1 << 30), 9), (dict(V=1, M=4, ld_beam=1), 1), (dict(dtype=3), 1), (dict(ld_beam=99), 1),
    (dict(ld_batch=99), 1), (dict(finished=0x70000, pad=-1), 1), (dict(finished=0x70000, pad=100), 1), (dict(logits=0x10002), 2),
    (dict(scores=0x20001), 2), (dict(t=0x50002), 2), (dict(ws=0x60010), 2), (dict(ws_bytes=64), 4)])
def test_select_refuses(kw, status):
    assert _select(**kw) == status


def _reorder(src=0x10000, dst=0x20000, inner=64, sizes=(1, 1, 1, 1), ss=64, sd=64, os=(0,) * 4, od=(0,) * 4, count=1,
             parents=0x30000, ld=2, B=3, K=2, table=True):
    a = ctypes.c_int64 * 4
    st = flce.FlceBeamState(src, dst, ss, sd, inner, a(*sizes), a(*os), a(*od))
    t = (flce.FlceBeamState * 1)(st) if table else None
    return flce.load_library().flce_beam_reorder(t and ctypes.addressof(t), count, parents, ld, B, K, None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), 1), (dict(table=False), 1), (dict(parents=None), 1), (dict(B=0), 1), (dict(K=0), 1), (dict(K=33, ld=33), 9),
    (dict(ld=1), 1), (dict(parents=0x30002), 2), (dict(inner=-1), 1), (dict(sizes=(1, -1, 1, 1)), 1), (dict(src=None), 1),
    (dict(dst=None), 1), (dict(dst=0x10000, sd=128), 1), (dict(dst=0x10000, sizes=(2, 1, 1, 1), os=(4096, 0, 0, 0)), 1)])
def test_reorder_refuses(kw, status):
    assert _reorder(**kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the refusal on a machine without a GB300")
def test_good_arguments_reach_the_device_check():
    assert _select() == 3 and _select(finished=0x70000) == 3 and _reorder() == 3 and _reorder(dst=0x10000) == 3


def test_workspace_size():
    size = flce.flce_beam_select_workspace_size
    assert size(0, 1, 10, 1) == size(1, 33, 10, 1) == size(1, 1, 0, 1) == size(1, 1, 10, 65) == 0
    for B, K, V, M in [(1, 1, 1, 1), (1, 4, 128256, 8), (64, 8, 32000, 16), (16, 16, 256000, 32), (2000, 32, 256000, 64)]:
        segments = -(-V // 2048) + 1
        assert 0 < size(B, K, V, M) <= B * K * segments * (8 + 8 * M) + 512


def test_state_descriptors():
    from linear_cross_entropy_tcgen05_gb300.beam_ops import _state as words

    def _state(src, dst, dim):
        w = words(src, dst, dim)
        assert len(w) * 8 == ctypes.sizeof(flce.FlceBeamState)
        return flce.FlceBeamState.from_buffer_copy((ctypes.c_int64 * 17)(*w))

    a = torch.zeros(3, 8, 5, 16, 4)  # layers, beams, heads, positions, columns
    s = _state(a, a, 1)
    assert s.inner_bytes == 5 * 16 * 4 * 4 and list(s.outer_size) == [3, 1, 1, 1] and s.beam_stride_src == 5 * 16 * 4 * 4
    assert s.outer_stride_src[0] == s.outer_stride_dst[0] == 8 * 5 * 16 * 4 * 4
    s = _state(a[:, :, :, :7], a[:, :, :, :7], 1)  # the first positions alone
    assert s.inner_bytes == 7 * 4 * 4 and list(s.outer_size) == [5, 3, 1, 1]
    assert list(s.outer_stride_src)[:2] == [16 * 4 * 4, 8 * 5 * 16 * 4 * 4]
    s = _state(a.permute(4, 3, 2, 1, 0), a.permute(4, 3, 2, 1, 0), 3)
    assert s.inner_bytes == 5 * 16 * 4 * 4 and list(s.outer_size) == [3, 1, 1, 1]
    b = torch.zeros(3, 8, 5, 16, 4).permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4)  # another layout for out
    s = _state(a, b, 1)
    assert s.inner_bytes == 4 * 4 and sorted(s.outer_size) == [1, 3, 5, 16]
    f = torch.zeros(8, dtype=torch.bool)
    s = _state(f, f, 0)
    assert s.inner_bytes == 1 and list(s.outer_size) == [1, 1, 1, 1] and s.beam_stride_src == 1


def test_python_refuses():
    z, s = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    for args, kw, exc in [((z.double(), s), {}, TypeError), ((z[0], s), {}, ValueError), ((z, s[:1]), {}, ValueError),
                          ((z, s.double()), {}, TypeError), ((z, s), {}, ValueError)]:
        with pytest.raises(exc):
            flce.beam_select(*args, **kw)
    with pytest.raises(TypeError):
        flce.beam_reorder([z], torch.zeros(2, 3))
    with pytest.raises(ValueError):
        flce.beam_reorder([z], torch.zeros(2, 3, dtype=torch.int32))

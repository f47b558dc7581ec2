"""The global gradient norm over many tensors, and clipping. ``clip_grad_norm`` takes gradient
tensors, ``clip_grad_norm_`` parameters; ``flce_clip_grad_norm`` marshals to the C ABI
(include/flce.h), which has the formulas."""
from __future__ import annotations

import array
import collections
import ctypes
import math

import torch
from torch.autograd.graph import increment_version

__all__ = ["clip_grad_norm", "clip_grad_norm_", "grad_norm", "flce_clip_grad_norm", "flce_clip_grad_norm_workspace_size"]


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    vp, i64, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.flce_clip_grad_norm_workspace_size.argtypes, lib.flce_clip_grad_norm_workspace_size.restype = [i64], sz
    lib.flce_clip_grad_norm.argtypes = [vp, i64, f32, f32, f32, f32, vp, vp, sz, vp]
    lib.flce_clip_grad_norm.restype = ctypes.c_int


from . import _call_on, _check, _nbytes, _ptr, _stream, load_library  # noqa: E402  (defined before this module is imported)
from .norm_ops import DTYPES  # noqa: E402


def flce_clip_grad_norm_workspace_size(count: int) -> int:
    """Workspace bytes of flce_clip_grad_norm for this number of tensors."""
    return int(load_library().flce_clip_grad_norm_workspace_size(count))


def flce_clip_grad_norm(tensors, total_norm, workspace, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6,
                        grad_scale: float = 1.0, stream=None, raise_on_error: bool = True) -> int:
    """Call flce_clip_grad_norm; ``tensors`` is a list of (gradient address, output address or 0,
    elements, dtype, output dtype) with dtypes as in flce_dtype. Returns the status."""
    table = _table([w for g, o, n, dt, odt in tensors for w in (g, o, n, dt | odt << 32)])
    st = load_library().flce_clip_grad_norm(table.buffer_info()[0], len(tensors), max_norm, norm_type, eps, grad_scale,
                                            _ptr(total_norm), _ptr(workspace), _nbytes(workspace), _stream(stream))
    if raise_on_error:
        _check(st, "flce_clip_grad_norm")
    return st


def _table(words) -> array.array:
    """An array of flce_grad_tensor: two addresses, a size and two 32-bit types, four 64-bit words."""
    return array.array("q", words)


def _dense(t) -> bool:
    """Whether t's elements fill one run of memory, in whatever order of its dimensions."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != step:
            return False
        step *= size
    return True


def check_written(read, write) -> None:
    """Refuses lists of addresses in which an entry writes what another one reads or writes: the kernels work
    on all entries at once, in no order."""
    written = set(write)
    if len(written) != len(write):
        raise ValueError("a tensor may not be listed twice")
    if read != write and not written.isdisjoint(read):
        readers = collections.Counter(read)
        if any(readers[w] != (w == r) for r, w in zip(read, write)):
            raise ValueError("a tensor of out may not be another entry's input")


def _run(grads, max_norm, norm_type, eps, grad_scale, out):
    first = grads[0]
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("gradients must be CUDA tensors")
    words = []
    for i, g in enumerate(grads):
        dt = DTYPES.get(g.dtype)
        if dt is None:
            raise TypeError(f"gradients must be bfloat16, float16 or float32, got {g.dtype}")
        if g.device != dev:
            raise ValueError("gradients must be on one device")
        if not g.is_contiguous() and not _dense(g):
            raise ValueError("a gradient must fill one run of memory (no gaps, nothing expanded)")
        p = g.data_ptr()
        if out is None:
            words += (p, 0, g.numel(), dt)
        elif out is grads:
            words += (p, p, g.numel(), dt | dt << 32)
        else:
            o = out[i]
            odt = DTYPES.get(o.dtype)
            if odt is None:
                raise TypeError(f"out must be bfloat16, float16 or float32, got {o.dtype}")
            if o.device != dev or o.shape != g.shape or (o.stride() != g.stride() and not
                                                         (g.is_contiguous() and o.is_contiguous())):
                raise ValueError("out must have the gradients' shapes, strides and device")
            words += (p, o.data_ptr(), g.numel(), dt | odt << 32)
    if out is not None:
        sizes, read, write = words[2::4], words[0::4], words[1::4]
        if 0 in sizes:  # (tensors without elements may have one address)
            read, write = ([a for a, n in zip(t, sizes) if n] for t in (read, write))
        check_written(read, write)
    lib, table = load_library(), _table(words)
    total = torch.empty((), dtype=torch.float32, device=dev)
    need = lib.flce_clip_grad_norm_workspace_size(len(grads))
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call_on(dev, "flce_clip_grad_norm", lib.flce_clip_grad_norm, table.buffer_info()[0], len(grads), max_norm, norm_type,
             eps, grad_scale, total.data_ptr(), ws.data_ptr(), need)
    if out is not None:
        increment_version(out)  # a backward pass that saved one of them is refused
    return total


def clip_grad_norm(grads, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, grad_scale: float = 1.0, out=None):
    """Scales all ``grads`` (a list of tensors) by ``grad_scale * min(1, max_norm / (total + eps))``
    and returns ``total``, the norm of all of them together after ``grad_scale``, as a 0-dim
    float32 tensor on their device. Nothing waits for the GPU.

    ``norm_type`` is 2 or infinity, ``grad_scale`` what every gradient is multiplied with first
    (one over the loss scale or the number of micro-batches), ``out`` a list of tensors of the
    gradients' shapes that get the result, of any of the three types (None: in place). Squares
    are added in 32 bits by sixteens, and their sums in 64; nothing overflows or underflows where the norm
    does not. As in
    torch, a NaN norm makes every gradient NaN, and an infinite one makes them 0 or NaN. A
    tensor may not be listed twice. Runs as under ``no_grad``: the norm and the results carry no gradient.
    """
    grads = list(grads)
    if out is not None and len(out) != len(grads):
        raise ValueError("out must have one tensor for each gradient")
    if not grads:
        return torch.zeros((), dtype=torch.float32)
    return _run(grads, max_norm, norm_type, eps, grad_scale, grads if out is None else out)


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, grad_scale: float = 1.0):
    """``clip_grad_norm`` in place on the ``.grad`` of ``parameters`` (a tensor or an iterable);
    those without one are passed over, and one that is listed again (tied weights) counts once."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    unique = {id(p): p for p in parameters}.values()
    return clip_grad_norm([p.grad for p in unique if p.grad is not None], max_norm, norm_type, eps, grad_scale)


def grad_norm(grads, norm_type: float = 2.0, grad_scale: float = 1.0):
    """The norm of all ``grads`` together, which stay as they are. It carries no gradient."""
    grads = list(grads)
    if not grads:
        return torch.zeros((), dtype=torch.float32)
    return _run(grads, math.inf, norm_type, 0.0, grad_scale, None)

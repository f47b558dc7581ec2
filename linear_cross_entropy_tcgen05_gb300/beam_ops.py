"""A beam-search step: ``beam_select`` chooses the best continuations over beams and vocabulary,
``beam_reorder`` moves the states (caches, token histories, flags) to the beams that go on.
``flce_beam_select`` and ``flce_beam_reorder`` marshal to the C ABI (include/flce.h)."""
from __future__ import annotations

import array
import ctypes
import math

import torch
from torch.autograd.graph import increment_version

__all__ = ["beam_select", "beam_reorder", "flce_beam_select", "flce_beam_select_workspace_size", "flce_beam_reorder",
           "FlceBeamState"]


class FlceBeamState(ctypes.Structure):
    """Mirror of ``flce_beam_state`` in include/flce.h."""

    _fields_ = ([("src", ctypes.c_void_p), ("dst", ctypes.c_void_p)]
                + [(n, ctypes.c_int64) for n in ("beam_stride_src", "beam_stride_dst", "inner_bytes")]
                + [(n, ctypes.c_int64 * 4) for n in ("outer_size", "outer_stride_src", "outer_stride_dst")])


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    lib.flce_beam_select_workspace_size.argtypes, lib.flce_beam_select_workspace_size.restype = [i64] * 4, sz
    lib.flce_beam_select.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, vp, i32, i64, vp, vp, vp, vp, sz, vp]
    lib.flce_beam_select.restype = ctypes.c_int
    lib.flce_beam_reorder.argtypes = [vp, i64, vp, i64, i64, i64, vp]
    lib.flce_beam_reorder.restype = ctypes.c_int


from . import _call_on, _check, _nbytes, _ptr, _stream, load_library  # noqa: E402  (defined before this module is imported)
from .grad_ops import check_written  # noqa: E402
from .norm_ops import DTYPES  # noqa: E402


def flce_beam_select_workspace_size(B: int, K: int, V: int, M: int) -> int:
    """Workspace bytes of flce_beam_select."""
    return int(load_library().flce_beam_select_workspace_size(B, K, V, M))


def _select_args(logits, scores, finished, pad_token, M, out_scores, out_parents, out_tokens, workspace, ws_bytes):
    B, K, V = logits.shape
    sb, sk, _ = logits.stride()
    return (logits.data_ptr(), DTYPES[logits.dtype], B, K, V, max(sb, V) if B == 1 else sb, max(sk, V) if K == 1 else sk,
            scores.data_ptr(), None if finished is None else finished.data_ptr(), int(pad_token), int(M), _ptr(out_scores),
            _ptr(out_parents), _ptr(out_tokens), _ptr(workspace), ws_bytes)


def flce_beam_select(logits, scores, finished, pad_token: int, M: int, out_scores, out_parents, out_tokens, workspace,
                     stream=None, raise_on_error: bool = True) -> int:
    """Call flce_beam_select on logits [B, K, V] with unit stride along V; returns the status."""
    st = load_library().flce_beam_select(*_select_args(logits, scores, finished, pad_token, M, out_scores, out_parents,
                                                       out_tokens, workspace, _nbytes(workspace)), _stream(stream))
    if raise_on_error:
        _check(st, "flce_beam_select")
    return st


def flce_beam_reorder(states, parents, B: int, K: int, ld_parents: int | None = None, stream=None,
                      raise_on_error: bool = True) -> int:
    """Call flce_beam_reorder on a list of FlceBeamState; returns the status."""
    table = (FlceBeamState * len(states))(*states)
    st = load_library().flce_beam_reorder(ctypes.addressof(table), len(states), _ptr(parents), K if ld_parents is None else ld_parents, B, K,
                                          _stream(stream))
    if raise_on_error:
        _check(st, "flce_beam_reorder")
    return st


def beam_select(logits, scores, num: int | None = None, finished=None, pad_token: int = 0):
    """The ``num`` best continuations (K unless given) of each request: ``(scores, parents, tokens)``,
    float32 and int32 [B, num], best first.

    ``logits`` [B, K, V] (bf16, f16 or f32, unit stride along V) and the beams' ``scores`` [B, K]
    (float32, sums of log-probabilities) give every candidate ``scores[b, k] + log_softmax(logits[b,
    k])[v]``; of equal ones the lowest ``k * V + v`` comes first (equal rows at equal scores are exact ties; the
    log of a row's sum of exponentials is right to about 1e-7). A beam marked in ``finished`` [B,
    K] (bool) goes on with ``pad_token`` alone, at its score. Masked tokens have a logit of -inf and
    so a score of -inf; a beam whose score or logsumexp is not finite (all tokens masked, a NaN) has
    no candidate. Candidates at -inf are returned, lowest index first, only where there are no
    others. Unused beams (all but the first at the first step) have a score of -inf. K is at most
    32, num 64. The scores carry no gradient.
    """
    if logits.dtype not in DTYPES:
        raise TypeError(f"logits must be bfloat16, float16 or float32, got {logits.dtype}")
    if logits.dim() != 3 or scores.shape != logits.shape[:2]:
        raise ValueError(f"expected logits [B, K, V] and scores [B, K], got {tuple(logits.shape)} and {tuple(scores.shape)}")
    if scores.dtype != torch.float32:
        raise TypeError("scores must be float32")
    dev = logits.device
    if dev.type != "cuda" or scores.device != dev or (finished is not None and finished.device != dev):
        raise ValueError("logits, scores and finished must be CUDA tensors on one device")
    if logits.shape[2] > 1 and logits.stride(2) != 1:
        raise ValueError("logits must have unit stride along the vocabulary")
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8):
            raise TypeError("finished must be bool")
        if finished.shape != scores.shape:
            raise ValueError("finished must have the scores' shape")
        finished = finished.contiguous()
    scores = scores.contiguous()
    B, K, V = logits.shape
    num = K if num is None else int(num)
    if K < 1 or V < 1 or not 1 <= num <= K * V:
        raise ValueError(f"num must be between 1 and the {K * V} candidates, got {num}")
    out = torch.empty((B, num), dtype=torch.float32, device=dev)
    parents = torch.empty((B, num), dtype=torch.int32, device=dev)
    tokens = torch.empty_like(parents)
    if B > 0:
        lib = load_library()
        need = lib.flce_beam_select_workspace_size(B, K, V, num)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _call_on(dev, "flce_beam_select", lib.flce_beam_select,
                 *_select_args(logits, scores, finished, pad_token, num, out, parents, tokens, ws, need))
    return out, parents, tokens


def _state(src, dst, dim: int):
    """A state's flce_beam_state as its 17 words: the dimensions but the beams' joined into one
    inner run of bytes and at most four outer ones."""
    size, shape = src.element_size(), src.shape
    if src.is_contiguous() and dst.is_contiguous():
        inner = math.prod(shape[dim + 1:]) * size
        step = inner * shape[dim]
        return (src.data_ptr(), dst.data_ptr(), inner, inner, inner, math.prod(shape[:dim]), 1, 1, 1, step, 0, 0, 0, step, 0, 0, 0)
    dims = [(n, a * size, b * size) for i, (n, a, b) in enumerate(zip(shape, src.stride(), dst.stride()))
            if i != dim and n != 1]
    dims.sort(key=lambda t: (t[1], t[2]))  # innermost first
    inner, outer = size, []
    for n, a, b in dims:
        if not outer and a == inner and b == inner:
            inner *= n
        elif outer and a == outer[-1][0] * outer[-1][1] and b == outer[-1][0] * outer[-1][2]:
            outer[-1] = (outer[-1][0] * n, outer[-1][1], outer[-1][2])
        else:
            outer.append((n, a, b))
    if len(outer) > 4:
        raise ValueError("a state has too many separate strides")
    outer += [(1, 0, 0)] * (4 - len(outer))
    return (src.data_ptr(), dst.data_ptr(), src.stride(dim) * size, dst.stride(dim) * size, inner,
            *[t[i] for i in range(3) for t in outer])


def beam_reorder(states, parents, dims=0, out=None):
    """Moves the beams of every tensor in ``states``: along its dimension ``dims`` (a number, or one for
    each state), of size B * K, beam j of request b becomes what beam ``parents[b, j]`` of that
    request was. ``parents`` is int32 [B, K] with unit stride along K (the first K columns of
    ``beam_select``'s, say). In place, without a second buffer, or into ``out`` (a list of tensors of the
    same shapes and types, which share no memory with the states). None may be written twice. Returns the reordered tensors.

    States have any type and any strides that leave at most four outer dimensions: a cache's
    first ``length`` positions are reordered alone as ``cache[:, :, :length]``. A parent
    outside [0, K) leaves the beam what it was. K is at most 32. Not differentiable: what is written may not
    require a gradient (but under ``no_grad``).
    """
    states = list(states)
    dst = states if out is None else list(out)
    if len(dst) != len(states):
        raise ValueError("out must have one tensor for each state")
    if parents.dtype != torch.int32 or parents.dim() != 2:
        raise TypeError("parents must be int32 [B, K]")
    B, K = parents.shape
    if K < 1 or (K > 1 and parents.stride(1) != 1):
        raise ValueError("parents must have at least one beam and unit stride along the beams")
    dev = parents.device
    if dev.type != "cuda":
        raise ValueError("parents must be a CUDA tensor")
    dims = [dims] * len(states) if isinstance(dims, int) else list(dims)
    if len(dims) != len(states):
        raise ValueError("dims must have one number for each state")
    table = []
    for s, d, dim in zip(states, dst, dims):
        if not -s.dim() <= dim < s.dim() or s.shape[dim] != B * K:
            raise ValueError(f"a state of shape {tuple(s.shape)} has no {B * K} beams along dimension {dim}")
        if d.shape != s.shape or d.dtype != s.dtype or s.device != dev or d.device != dev:
            raise ValueError("out must have the states' shapes and types, and all be on the parents' device")
        if not d.is_contiguous() and any(n > 1 and st == 0 for n, st in zip(d.shape, d.stride())):
            raise ValueError("an expanded tensor cannot be reordered into")
        if s.numel():
            table += _state(s, d, dim % s.dim())
    if torch.is_grad_enabled() and any([d.requires_grad for d in dst]):
        raise RuntimeError("a tensor that requires a gradient cannot be reordered into: its gradient would not know of the "
                           "new order. Decode under torch.no_grad(), or detach the states")
    if table:
        words = array.array("q", table)
        check_written(words[0::17], words[1::17])
        _call_on(dev, "flce_beam_reorder", load_library().flce_beam_reorder, words.buffer_info()[0], len(words) // 17,
                 parents.data_ptr(), parents.stride(0) if B > 1 else K, B, K)
        increment_version(dst)  # a backward pass that saved one of them is refused
    return dst

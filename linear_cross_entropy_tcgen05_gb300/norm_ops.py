"""The block norm: norms after and before a transformer block, fused with the block's gate and
residual scale. ``block_norm`` is the differentiable call; ``flce_block_norm_forward`` and
``flce_block_norm_backward`` marshal device tensors to the C ABI (include/flce.h), which has
the formulas."""
from __future__ import annotations

import ctypes
import struct

import torch
from torch.autograd import forward_ad

__all__ = ["block_norm", "BlockNormFunction", "BlockNorm", "FlceBlockNormDesc", "FlceBlockNormGrads",
           "flce_block_norm_forward", "flce_block_norm_backward", "flce_block_norm_workspace_size", "DTYPES", "NORMS",
           "GATE_ACTIVATIONS"]

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # flce_dtype
NORMS = {"rms": 0, "layer": 1}  # flce_norm
GATE_ACTIVATIONS = {"none": 0, "sigmoid": 1, "tanh": 2}  # flce_gate_activation

_VP, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class FlceBlockNormDesc(ctypes.Structure):
    """Mirror of ``flce_block_norm_desc`` in include/flce.h."""

    _fields_ = ([(n, _I64) for n in ("N", "D", "gate_rows")]
                + [(n, _VP) for n in ("x", "residual", "gate", "post_weight", "post_bias", "weight", "bias")]
                + [(n, _I64) for n in ("ld_x", "ld_residual", "ld_gate")]
                + [(n, _I32) for n in ("x_dtype", "residual_dtype", "gate_dtype", "post_weight_dtype",
                                       "post_bias_dtype", "weight_dtype", "bias_dtype", "norm", "gate_activation")]
                + [(n, _F32) for n in ("eps", "scale", "weight_offset")])


class FlceBlockNormGrads(ctypes.Structure):
    """Mirror of ``flce_block_norm_grads`` in include/flce.h."""

    _fields_ = [(n, _VP) for n in ("dx", "dresidual", "dgate", "dpost_weight", "dpost_bias", "dweight", "dbias")]


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    sz, i = ctypes.c_size_t, ctypes.c_int  # (the descriptors go as addresses: of a structure, or of packed bytes)
    lib.flce_block_norm_forward.argtypes, lib.flce_block_norm_forward.restype = [_VP] * 5, i
    lib.flce_block_norm_workspace_size.argtypes, lib.flce_block_norm_workspace_size.restype = [_I64, _I64, _I64], sz
    lib.flce_block_norm_backward.argtypes = [_VP, _VP, _VP, _VP, _I64, _VP, _I64, _VP, _VP, sz, _VP]
    lib.flce_block_norm_backward.restype = i


from . import _call_on, _check, _nbytes, _ptr, _stream, load_library  # noqa: E402  (defined before this module is imported)


def flce_block_norm_workspace_size(N: int, D: int, gate_rows: int = 0) -> int:
    """Workspace bytes of flce_block_norm_backward."""
    return int(load_library().flce_block_norm_workspace_size(N, D, gate_rows))


def flce_block_norm_forward(desc: FlceBlockNormDesc, h, y, stats=None, stream=None, raise_on_error: bool = True) -> int:
    """Call flce_block_norm_forward; returns the status."""
    st = load_library().flce_block_norm_forward(ctypes.byref(desc), _ptr(h), _ptr(y), _ptr(stats), _stream(stream))
    if raise_on_error:
        _check(st, "flce_block_norm_forward")
    return st


def flce_block_norm_backward(desc: FlceBlockNormDesc, h, stats, dh, dy, grads: FlceBlockNormGrads, workspace,
                             stream=None, raise_on_error: bool = True) -> int:
    """Call flce_block_norm_backward (dh and dy [N, D] with unit column stride, or None)."""
    st = load_library().flce_block_norm_backward(
        ctypes.byref(desc), _ptr(h), _ptr(stats), _ptr(dh), 0 if dh is None else _row_stride(dh), _ptr(dy),
        0 if dy is None else _row_stride(dy), ctypes.byref(grads), _ptr(workspace), _nbytes(workspace), _stream(stream))
    if raise_on_error:
        _check(st, "flce_block_norm_backward")
    return st


def _row_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _rows(t, D: int, name: str):
    """t as [rows, D] without a copy."""
    if t.dim() == 2 and (t.stride(1) == 1 or D == 1):
        return t
    if t.dim() != 2 and (t.stride(-1) == 1 or D == 1):
        try:
            return t.view(-1, D)
        except RuntimeError:
            pass
    raise ValueError(f"{name} must have unit stride along its last dimension and one stride between its rows")


def _has_rows(t, D: int) -> bool:
    """Whether the kernels can read t as it is."""
    try:
        return _row_stride(_rows(t if t.dim() > 1 else t.unsqueeze(0), D, "")) >= D
    except ValueError:
        return False


def _joined(t):
    """t, or a copy of one whose rows have more than one stride between them (x[:, 1:] of three dimensions)."""
    if t is None or t.is_contiguous() or t.stride(-1) != 1 or _has_rows(t, t.shape[-1]):
        return t
    return t.contiguous()


def _gate_rows(gate, x) -> int:
    """Rows of the gate: it is shared by all rows ([D]), by equal runs of rows ([G, D], or x's
    shape with ones between the leading dimensions and the last), or has one for each."""
    D = x.shape[-1]
    if gate.dim() == 0 or gate.shape[-1] != D:
        raise ValueError(f"gate must end with {D} columns, got {tuple(gate.shape)}")
    rows = gate.numel() // D if D else 0
    if gate.dim() == 1 or gate.shape == x.shape:
        return rows
    if x.dim() == 2 and gate.dim() == 2:
        if rows > 0 and x.shape[0] % rows == 0:
            return rows
    elif gate.dim() == x.dim():
        k = gate.dim() - 1
        while k > 0 and gate.shape[k - 1] == 1:
            k -= 1
        if gate.shape[:k] == x.shape[:k]:
            return rows
    raise ValueError(f"gate {tuple(gate.shape)} does not group the rows of x {tuple(x.shape)}")


_PACK = struct.Struct("3q7q3q9i3f")  # flce_block_norm_desc
_GRADS = struct.Struct("7q")  # flce_block_norm_grads: dx, dresidual, dgate, dpost_weight, dpost_bias, dweight, dbias


def _describe(x, residual, weight, bias, post_weight, post_bias, gate, norm, eps, scale, gate_activation,
              weight_offset):
    """A call's flce_block_norm_desc as bytes, its rows and gate rows; raises on what the library
    cannot take."""
    xd, dev = DTYPES.get(x.dtype), x.device
    if xd is None:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have at least one column")
    if dev.type != "cuda":
        raise ValueError("x must be a CUDA tensor")
    D = x.shape[-1]
    rows = _rows(x, D, "x")
    N, px, ld_x = rows.shape[0], x.data_ptr(), _row_stride(rows)
    pr = pg = ld_r = ld_g = gate_rows = gd = 0
    rd = xd
    if residual is not None:
        if residual.shape != x.shape or residual.device != dev:
            raise ValueError(f"residual must have x's shape {tuple(x.shape)} and device, got {tuple(residual.shape)}")
        if residual.dtype != x.dtype and residual.dtype != torch.float32:
            raise TypeError(f"residual must have x's type or float32, got {residual.dtype}")
        pr, ld_r, rd = residual.data_ptr(), _row_stride(_rows(residual, D, "residual")), DTYPES[residual.dtype]
    if gate is not None:
        if gate.device != dev:
            raise ValueError("gate must be on x's device")
        gate_rows, gd = _gate_rows(gate, x), DTYPES.get(gate.dtype)
        if gd != xd and gd != rd:
            raise TypeError(f"gate must have x's or the residual's type, got {gate.dtype}")
        pg, ld_g = gate.data_ptr(), _row_stride(_rows(gate if gate.dim() > 1 else gate.unsqueeze(0), D, "gate"))
    if (bias is not None and weight is None) or (post_bias is not None and post_weight is None):
        raise ValueError("a bias needs its weight")
    pw, wd = _param("post_weight", post_weight, D, dev)
    pb, bd = _param("post_bias", post_bias, D, dev)
    qw, vd = _param("weight", weight, D, dev)
    qb, cd = _param("bias", bias, D, dev)
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}")
    if gate_activation not in GATE_ACTIVATIONS:
        raise ValueError(f"gate_activation must be one of {sorted(GATE_ACTIVATIONS)}")
    words = _PACK.pack(N, D, gate_rows, px, pr, pg, pw, pb, qw, qb, ld_x, ld_r, ld_g, xd, rd, gd, wd, bd, vd, cd,
                       NORMS[norm], GATE_ACTIVATIONS[gate_activation], eps, scale, weight_offset)
    return words, N, gate_rows


def _param(name: str, t, D: int, dev):
    """Address and type of a parameter [D], or zeros."""
    if t is None:
        return 0, 0
    if t.dim() != 1 or t.shape[0] != D or t.device != dev:
        raise ValueError(f"{name} must be [{D}] on x's device, got {tuple(t.shape)}")
    dt = DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    if D > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), dt


def _forward(desc, x, h_dtype, want_y: bool, want_stats: bool):
    words, N, _ = desc
    dev = x.device
    plain = x.is_contiguous()
    h = torch.empty_like(x) if plain and h_dtype == x.dtype else torch.empty(x.shape, dtype=h_dtype, device=dev)
    y = None
    if want_y:
        y = torch.empty_like(x) if plain else torch.empty(x.shape, dtype=x.dtype, device=dev)
    stats = torch.empty((N, 4), dtype=torch.float32, device=dev) if want_stats else None
    if N > 0:
        _call_on(dev, "flce_block_norm_forward", load_library().flce_block_norm_forward, words, h.data_ptr(),
                 None if y is None else y.data_ptr(), None if stats is None else stats.data_ptr())
    return h, y, stats


class BlockNormFunction(torch.autograd.Function):
    """(h, y) of the block norm with fused gradients; see ``block_norm``."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, post_weight, post_bias, gate, norm, eps, scale, gate_activation,
                weight_offset):
        opts = (norm, eps, scale, gate_activation, weight_offset)
        desc = _describe(x, residual, weight, bias, post_weight, post_bias, gate, *opts)
        h, y, stats = _forward(desc, x, x.dtype if residual is None else residual.dtype, weight is not None, True)
        # the residual's values are not needed again, only its type (h has it)
        ctx.save_for_backward(x, weight, bias, post_weight, post_bias, gate, h, stats)
        ctx.opts = opts
        ctx.set_materialize_grads(False)
        return h, y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dy):
        if dh is None and dy is None:
            return (None,) * 12
        # a saved-tensor hook may have brought them back elsewhere or with other strides: described anew
        # (the residual may be gone, h stands in for its type), and copied where the kernels need it
        saved = ctx.saved_tensors
        if not all([t is None or t.is_contiguous() for t in saved]):
            rows = saved[0], saved[5]  # x and the gate are read with strides between their rows
            saved = [t if t is None or any(t is r for r in rows) and _has_rows(t, t.shape[-1]) else t.contiguous() for t in saved]
        x, weight, bias, post_weight, post_bias, gate, h, stats = saved
        want, dev, D = ctx.needs_input_grad, x.device, x.shape[-1]
        words, N, gate_rows = _describe(x, h, weight, bias, post_weight, post_bias, gate, *ctx.opts)
        out = [None] * 12
        at = [0] * 7
        for i, t in enumerate((x, h, weight, bias, post_weight, post_bias, gate)):
            if want[i]:
                out[i] = torch.empty(t.shape, dtype=t.dtype, device=dev)
                at[i] = out[i].data_ptr()
        if N == 0:
            for t in out:
                if t is not None:
                    t.zero_()
            return tuple(out)
        dh, ld_dh, _dh = _upstream(dh, D, h.dtype)
        dy, ld_dy, _dy = _upstream(dy, D, x.dtype)
        lib = load_library()
        need = lib.flce_block_norm_workspace_size(N, D, gate_rows)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _call_on(dev, "flce_block_norm_backward", lib.flce_block_norm_backward, words, h.data_ptr(),
                 stats.data_ptr(), dh, ld_dh, dy, ld_dy,
                 _GRADS.pack(at[0], at[1], at[6], at[4], at[5], at[2], at[3]), ws.data_ptr(), need)
        return tuple(out)


def _upstream(t, D: int, dtype):
    """Address, row stride and tensor of an upstream gradient as rows of D columns; one that is
    expanded, or of another type, is copied."""
    if t is None:
        return None, 0, None
    if t.dtype != dtype:
        t = t.to(dtype)
    if t.dim() != 2:
        t = t.reshape(-1, D)
    if (t.stride(1) != 1 and D > 1) or _row_stride(t) < D:
        t = t.contiguous()
    return t.data_ptr(), _row_stride(t), t


def block_norm(x, residual=None, weight=None, *, bias=None, post_weight=None, post_bias=None, gate=None,
               gate_activation: str = "none", scale: float = 1.0, norm: str = "rms", eps: float = 1e-6,
               weight_offset: float = 0.0):
    """``(h, y)`` with ``h = residual + scale * act(gate) * u`` and ``y = Norm(h; weight, bias)``,
    ``u = Norm(x; post_weight, post_bias)`` or ``x`` without a post_weight.

    ``x`` [..., D] (bf16, f16 or f32) is a block's output, ``residual`` the stream it is added
    to (x's type or f32; None: nothing is added), ``y`` the next block's or the head's input in
    x's type (None without a ``weight``), ``h`` the new stream in the residual's type. ``gate``
    (x's or the residual's type) has one row for all rows ([D]), one for each equal run of rows
    ([G, D] for x [N, D], [B, 1, D] for x [B, T, D]) or x's shape, and goes through
    ``gate_activation`` ("none", "sigmoid", "tanh"). ``norm`` is "rms" or "layer"; weights are
    used as ``weight + weight_offset``. D is at most 16384. x, residual and gate have unit stride along
    D; rows with one stride between them are read in place, others are copied first.

    Differentiable in every tensor (by backward passes; forward-mode inputs raise); a gradient has its
    input's type. With a 16-bit residual stream the backward pass reads the h that was rounded to it, so that
    the weight's gradient has that rounding too (2.4e-3 of it off in bf16, 1.7e-3 by its own); with an fp32
    stream nothing is rounded between the passes.
    """
    if x.dim() > 2:
        x, residual, gate = _joined(x), _joined(residual), _joined(gate)
    args = (x, residual, weight, bias, post_weight, post_bias, gate)
    if torch.is_grad_enabled() and any([t is not None and t.requires_grad for t in args]) or _forward_mode(args):
        return BlockNormFunction.apply(*args, norm, eps, scale, gate_activation, weight_offset)
    desc = _describe(*args, norm, eps, scale, gate_activation, weight_offset)
    h, y, _ = _forward(desc, x, x.dtype if residual is None else residual.dtype, weight is not None, False)
    return h, y


def _forward_mode(args) -> bool:
    """Whether a tensor has a forward-mode tangent. BlockNormFunction refuses it; a call that does not go
    through autograd would lose it."""
    return forward_ad._current_level >= 0 and any([t is not None and forward_ad.unpack_dual(t).tangent is not None
                                                   for t in args])


class BlockNorm(torch.nn.Module):
    """``block_norm`` with parameters of its own: a pre-norm (``weight``), and as asked a post-norm
    (``post_weight``), a gate for each channel (``gate``, starting at ``gate_init``) and biases. Parameters may
    have another type than the activations (fp32 ones, say, by default)."""

    def __init__(self, dim: int, norm: str = "rms", eps: float = 1e-6, scale: float = 1.0, post_norm: bool = False,
                 gate_init: float | None = None, gate_activation: str = "none", bias: bool = False, device=None,
                 dtype=None):
        super().__init__()
        if norm not in NORMS:
            raise ValueError(f"norm must be one of {sorted(NORMS)}")
        if gate_activation not in GATE_ACTIVATIONS:
            raise ValueError(f"gate_activation must be one of {sorted(GATE_ACTIVATIONS)}")
        kw = dict(device=device, dtype=dtype)
        par = torch.nn.Parameter
        self.norm, self.eps, self.scale, self.gate_activation = norm, float(eps), float(scale), gate_activation
        self.weight = par(torch.ones(dim, **kw))
        self.bias = par(torch.zeros(dim, **kw)) if bias else None
        self.post_weight = par(torch.ones(dim, **kw)) if post_norm else None
        self.post_bias = par(torch.zeros(dim, **kw)) if post_norm and bias else None
        self.gate = par(torch.full((dim,), float(gate_init), **kw)) if gate_init is not None else None

    def forward(self, x, residual=None):
        gate = self.gate
        if gate is not None and gate.dtype != x.dtype and (residual is None or gate.dtype != residual.dtype):
            # the kernels read a gate with the rows, in x's or the residual's type: rounded to x's, half a step
            # of what its product with x has anyway
            gate = gate.to(x.dtype)
        return block_norm(x, residual, self.weight, bias=self.bias, post_weight=self.post_weight,
                          post_bias=self.post_bias, gate=gate, gate_activation=self.gate_activation,
                          scale=self.scale, norm=self.norm, eps=self.eps)

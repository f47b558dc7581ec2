"""The block norm on the GPU against its formulas in 64 bits: forward values, gradients, types,
layouts, odd sizes, rows shared by clusters, streams, graphs and non-finite rows."""
import math

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce
from tests import block_norm_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# N, D, x type, residual type (None: no residual), norm, post, gate rows (0 none, -1 one a row), activation, biases
CASES = [
    (1, 1, "f32", "f32", "rms", False, 0, "none", False),
    (1, 4096, "bf16", "bf16", "rms", True, 0, "none", False),
    (2, 7, "bf16", "bf16", "layer", True, 1, "none", True),
    (3, 8, "f16", "f32", "rms", True, -1, "sigmoid", False),
    (5, 64, "bf16", "f32", "layer", True, 5, "tanh", True),
    (64, 129, "f16", "f16", "rms", True, 4, "tanh", True),
    (300, 256, "f32", "f32", "layer", False, 3, "sigmoid", True),
    (17, 250, "bf16", "bf16", "rms", False, 0, "none", False),
    (100, 1001, "f32", "f32", "layer", True, -1, "sigmoid", True),
    (333, 1000, "bf16", "bf16", "rms", True, 0, "none", False),
    (1200, 2304, "bf16", "f32", "layer", True, 16, "tanh", True),
    (77, 4096, "f16", "f16", "layer", False, 1, "none", False),
    (2000, 4096, "bf16", "bf16", "rms", True, 1, "sigmoid", False),
    (9, 5120, "f32", "f32", "rms", True, 0, "none", True),
    (7, 5128, "bf16", "bf16", "layer", True, 1, "tanh", True),
    (33, 5121, "f16", "f32", "rms", True, 3, "sigmoid", False),
    (350, 8192, "bf16", "bf16", "rms", True, -1, "none", False),
    (11, 16384, "bf16", "f32", "layer", True, 11, "sigmoid", True),
    (3, 16384, "f32", "f32", "layer", True, 1, "tanh", True),
    (30, 4096, "f32", "f32", "layer", True, -1, "tanh", True),
    (30, 3456, "f32", "f32", "layer", True, 2, "sigmoid", True),
    (19, 4096, "bf16", "f32", "rms", True, 19, "sigmoid", False),
    (1500, 2560, "f16", "f16", "layer", True, 6, "sigmoid", True),
    (2, 16383, "bf16", "bf16", "rms", False, 0, "none", False),
    (40, 512, "bf16", None, "rms", False, 0, "none", False),
    (41, 640, "f16", None, "layer", True, 1, "sigmoid", True),
    (700, 96, "bf16", "bf16", "rms", True, 350, "sigmoid", False),
]


def make(case, seed=0, offset=0.0):
    N, D, x, res, norm, post, rows, act, bias = case
    g = torch.Generator(device=DEV).manual_seed(1000 + seed)
    n = lambda s, t, std=1.0, mean=0.0: torch.empty(s, device=DEV, dtype=t).normal_(mean, std, generator=g)  # noqa: E731
    tr = T[res or x]
    t = {"x": n((N, D), T[x], 1.3, offset), "residual": n((N, D), tr, 2.0, offset) if res else None,
         "gate": n((N if rows < 0 else rows, D), tr, 0.8, 0.2) if rows else None,
         "post_weight": n((D,), tr, 0.3, 1.0) if post else None, "post_bias": n((D,), tr, 0.3) if post and bias else None,
         "weight": n((D,), T[x], 0.3, 1.0), "bias": n((D,), tr, 0.3) if bias else None}
    return t, n((N, D), tr, 0.1), n((N, D), T[x], 0.1)


def options(case):
    return dict(norm=case[4], eps=1e-5, scale=0.75, gate_activation=case[7], weight_offset=0.125)


def check(case, t, h, y, stats, dh, dy, grads):
    o = options(case)
    out, _ = ref.forward(**t, norm=o["norm"], eps=o["eps"], scale=o["scale"], act=o["gate_activation"],
                         off=o["weight_offset"])
    ref.close(h, *out["h"], "h")
    if t["weight"] is not None:
        ref.close(y, *out["y"], "y")
    want = ref.backward(t["x"], h, t["gate"], t["post_weight"], t["post_bias"], t["weight"], t["bias"], stats, dh, dy,
                        o["norm"], o["scale"], o["gate_activation"], o["weight_offset"])
    for name, got in grads.items():
        if got is not None:
            ref.close(got.reshape(want["d" + name][0].shape), *want["d" + name], "d" + name)


def leaves(t):
    return {k: v for k, v in t.items() if v is not None}


def run(case, t, dh, dy):
    """Forward and backward through autograd, with the statistics that were saved."""
    l = leaves(t)
    for v in l.values():
        v.requires_grad_()
    h, y = flce.block_norm(**t, **options(case))
    stats = h.grad_fn.saved_tensors[-1]
    got = torch.autograd.grad([v for v in (h, y) if v is not None], list(l.values()), [v for v in (dh, dy) if v is not None])
    for v in l.values():
        v.requires_grad_(False)
    return h.detach(), None if y is None else y.detach(), stats, dict(zip(l, got))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_formulas(gpu_lib, case):
    t, dh, dy = make(case)
    h, y, stats, grads = run(case, t, dh, dy)
    check(case, t, h, y, stats, dh, dy, grads)
    for k, v in grads.items():
        assert v.dtype == t[k].dtype and v.shape == t[k].shape
    # the call without gradients gives the same bits
    h2, y2 = flce.block_norm(**t, **options(case))
    assert torch.equal(h, h2) and torch.equal(y, y2)
    # and the same inputs the same gradients
    again = run(case, t, dh, dy)[3]
    assert all(torch.equal(again[k], v) for k, v in grads.items())


def test_batches_of_one_row(gpu_lib):
    """Rows so wide that two do not fit a batch, several for each block."""
    test_against_the_formulas(gpu_lib, (700, 4096, "f32", "f32", "layer", True, -1, "tanh", True))
    test_against_the_formulas(gpu_lib, (200, 16384, "bf16", "f32", "layer", True, 8, "sigmoid", True))


WIDE = [  # rows enough for blocks of up to 640 threads, forward
    (700, 5120, "bf16", "bf16", "rms", True, 0, "none", False),
    (200, 4104, "f32", "f32", "rms", False, 0, "none", False),
    (400, 4608, "f16", "f32", "layer", True, -1, "tanh", True),
    (320, 4616, "bf16", "bf16", "layer", True, 4, "sigmoid", True),
    (301, 2408, "f32", "f32", "layer", False, -1, "sigmoid", False),
    (1300, 1520, "bf16", "f32", "layer", True, 13, "tanh", True),
    (3001, 264, "f16", "f16", "layer", True, 0, "none", False),
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_wide_blocks(gpu_lib, case):
    test_against_the_formulas(gpu_lib, case)


@pytest.mark.parametrize("x,res", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_unaligned_widths(gpu_lib, x, res):
    """Rows that start and end anywhere in 16 bytes, within one warp's columns and over several."""
    for D in (2, 3, 5, 9, 12, 15, 17, 31, 33, 63, 249, 255, 257, 260, 263, 511, 513, 770, 2047, 2049):
        test_against_the_formulas(gpu_lib, (5, D, x, res, "layer" if D % 2 else "rms", D % 3 > 0, (0, 1, -1)[D % 3],
                                            "tanh", D % 2 > 0))


@pytest.mark.parametrize("offset", range(1, 8))
def test_unaligned_bases(gpu_lib, offset):
    """Tensors that start anywhere in 16 bytes, with what is around their rows left as it is."""
    N, D = 7, 264
    g = torch.Generator(device=DEV).manual_seed(offset)
    wide = torch.empty(N * (D + 3) + 16, device=DEV).normal_(generator=g).to(torch.bfloat16)
    x = wide[offset:offset + N * (D + 3)].view(N, D + 3)[:, :D]
    w = torch.empty(D, device=DEV).normal_(1.0, 0.2, generator=g)
    h, y = flce.block_norm(x, None, w, post_weight=w)
    h2, y2 = flce.block_norm(x.contiguous(), None, w, post_weight=w)
    # sums are grouped alike; the aligned kernel of RMS norms multiplies in another order
    assert ((h.float() - h2.float()).abs() <= 2.0 ** -8 * h2.float().abs() * 2).all()
    assert ((y.float() - y2.float()).abs() <= 2.0 ** -8 * y2.float().abs() * 3).all()
    buf = torch.full((N * D + 32,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = buf[offset:offset + N * D].view(N, D)
    d = flce.FlceBlockNormDesc(N=N, D=D, x=x.data_ptr(), post_weight=w.data_ptr(), weight=w.data_ptr(), ld_x=D + 3,
                               post_weight_dtype=2, weight_dtype=2, eps=1e-6, scale=1.0)
    flce.flce_block_norm_forward(d, out, y2)
    assert torch.equal(out, h) and torch.equal(y2, y)
    assert bool((buf[:offset] == 3).all()) and bool((buf[offset + N * D:] == 3).all())


def test_without_a_weight(gpu_lib):
    case = (50, 384, "bf16", "f32", "rms", True, 1, "tanh", False)
    t, dh, _ = make(case)
    t["weight"] = None
    h, y, stats, grads = run(case, t, dh, None)
    assert y is None
    check(case, t, h, None, stats, dh, None, grads)


def test_large_common_offset(gpu_lib):
    """A layer norm of values around 200 with a deviation of 1: no cancellation in the statistics."""
    case = (20, 1024, "f32", "f32", "layer", True, 0, "none", True)
    t, dh, dy = make(case, offset=200.0)
    h, y, stats, grads = run(case, t, dh, dy)
    check(case, t, h, y, stats, dh, dy, grads)


@pytest.mark.parametrize("only", ["dh", "dy"])
def test_one_upstream_gradient(gpu_lib, only):
    case = (60, 768, "bf16", "bf16", "layer", True, 4, "sigmoid", True)
    t, dh, dy = make(case)
    l = leaves(t)
    for v in l.values():
        v.requires_grad_()
    h, y = flce.block_norm(**t, **options(case))
    stats = h.grad_fn.saved_tensors[-1]
    a, b = (dh, None) if only == "dh" else (None, dy)
    grads = dict(zip(l, torch.autograd.grad(h if only == "dh" else y, list(l.values()), a if only == "dh" else b)))
    for v in l.values():
        v.requires_grad_(False)
    check(case, t, h.detach(), y.detach(), stats, a, b, grads)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_misaligned_rows(gpu_lib, dtype):
    """Rows inside wider buffers, at odd offsets; upstream gradients that were expanded."""
    case = (37, 512, dtype, dtype, "rms", True, 1, "none", False)
    for left, wide in [(0, 520), (3, 519), (8, 1024)]:
        t, dh, dy = make(case)
        for k in ("x", "residual"):
            room = torch.full((37, wide + 8), float("nan"), dtype=t[k].dtype, device=DEV)
            room[:, left:left + 512] = t[k]
            t[k] = room[:, left:left + 512]
        h, y, stats, grads = run(case, t, dh, dy)
        check(case, t, h, y, stats, dh, dy, grads)
        one = dy[:1].expand_as(dy)
        grads = run(case, t, dh, one)[3]
        check(case, t, h, y, stats, dh, one, grads)


def test_leading_dimensions_and_gate_shapes(gpu_lib):
    B, S, D = 3, 10, 96
    case = (B * S, D, "bf16", "bf16", "rms", True, B, "sigmoid", False)
    t, dh, dy = make(case)
    flat = run(case, t, dh, dy)
    t3 = {k: (v.view(B, S, D) if k in ("x", "residual") else v.view(B, 1, D) if k == "gate" else v) if v is not None else None
          for k, v in t.items()}
    h, y, _, grads = run(case, t3, dh.view(B, S, D), dy.view(B, S, D))
    assert torch.equal(h.view(-1, D), flat[0]) and torch.equal(y.view(-1, D), flat[1])
    assert grads["gate"].shape == (B, 1, D) and torch.equal(grads["gate"].view(B, D), flat[3]["gate"])


def test_no_rows(gpu_lib):
    case = (2, 64, "bf16", "bf16", "rms", True, 1, "none", False)
    t, _, _ = make(case)
    t["x"], t["residual"] = t["x"][:0], t["residual"][:0]
    h, y, _, grads = run(case, t, t["residual"].clone(), t["x"].clone())
    assert h.shape == y.shape == (0, 64) and all(not v.any() for v in grads.values())


def test_h_in_the_residuals_buffer(gpu_lib):
    case = (70, 1024, "bf16", "f32", "rms", False, 0, "none", False)
    t, _, _ = make(case)
    h, y = flce.block_norm(**t, **options(case))
    d = flce.FlceBlockNormDesc(N=70, D=1024, x=t["x"].data_ptr(), residual=t["residual"].data_ptr(), weight=t["weight"].data_ptr(),
                               ld_x=1024, ld_residual=1024, x_dtype=0, residual_dtype=2, weight_dtype=0, eps=1e-5, scale=0.75,
                               weight_offset=0.125)
    y2 = torch.empty_like(t["x"])
    flce.flce_block_norm_forward(d, t["residual"], y2)
    assert torch.equal(t["residual"], h) and torch.equal(y, y2)


def test_a_bad_row_stays_in_its_row(gpu_lib):
    case = (9, 640, "bf16", "f32", "layer", True, 0, "none", True)
    t, _, _ = make(case)
    good_h, good_y = flce.block_norm(**t, **options(case))
    for bad in (math.inf, -math.inf, math.nan):
        x = t["x"].clone()
        x[4, 17] = bad
        h, y = flce.block_norm(**{**t, "x": x}, **options(case))
        rows = torch.arange(9, device=DEV) != 4
        assert torch.equal(h[rows], good_h[rows]) and torch.equal(y[rows], good_y[rows])
        assert y[4].isnan().all()


def test_zero_rows_are_finite(gpu_lib):
    """A row of zeros has a deviation of 0: eps alone keeps it finite, forward and backward."""
    case = (4, 256, "f32", "f32", "layer", True, 0, "none", True)
    t, dh, dy = make(case)
    t["x"][1] = 0
    t["residual"][1] = 0
    t["post_bias"].zero_()
    h, y, stats, grads = run(case, t, dh, dy)
    check(case, t, h, y, stats, dh, dy, grads)
    assert all(torch.isfinite(v).all() for v in (h, y, *grads.values()))


def test_gradient_against_differences(gpu_lib):
    """Directional differences of the kernel's own forward in fp32 (values near 1, a step of
    2^-7): the cut is of order step^2 of a smooth function, the rounding 2^-24 sqrt(N D) / step."""
    case = (6, 48, "f32", "f32", "layer", True, 2, "tanh", True)
    t, dh, dy = make(case)
    _, _, _, grads = run(case, t, dh, dy)
    g = torch.Generator(device=DEV).manual_seed(3)
    for k, v in leaves(t).items():
        way = torch.randn(v.shape, generator=g, device=DEV)
        step = 2.0 ** -7

        def loss(s):
            h, y = flce.block_norm(**{**t, k: v + s * way}, **options(case))
            return (h.double() * dh.double()).sum() + (y.double() * dy.double()).sum()

        # five-point differences: the cut falls to step^4 = 4e-9 of the fifth derivative
        d = (8 * (loss(step) - loss(-step)) - (loss(2 * step) - loss(-2 * step))) / (12 * step)
        want = (grads[k].double() * way.double()).sum()
        assert abs(float(d - want)) <= 2e-3 * (1 + abs(float(want))), k


def test_on_another_stream_and_in_a_graph(gpu_lib):
    case = (130, 1024, "bf16", "bf16", "rms", True, 1, "sigmoid", False)
    t, dh, dy = make(case)
    want = run(case, t, dh, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(case, t, dh, dy)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and all(torch.equal(got[3][k], v) for k, v in want[3].items())
    # captured with the low-level calls; replayed on new contents of the same buffers
    N, D = 130, 1024
    d = flce.FlceBlockNormDesc(N=N, D=D, gate_rows=1, x=t["x"].data_ptr(), residual=t["residual"].data_ptr(),
                               gate=t["gate"].data_ptr(), post_weight=t["post_weight"].data_ptr(), weight=t["weight"].data_ptr(),
                               ld_x=D, ld_residual=D, ld_gate=D, gate_activation=1, eps=1e-5, scale=0.75, weight_offset=0.125)
    h, y, dx, dw = (torch.empty_like(t["x"]) for _ in range(4))
    dw, stats = torch.empty_like(t["weight"]), torch.empty(N, 4, device=DEV)
    ws = torch.empty(flce.flce_block_norm_workspace_size(N, D, 1), dtype=torch.uint8, device=DEV)
    grads = flce.FlceBlockNormGrads(dx=dx.data_ptr(), dweight=dw.data_ptr())

    def step():
        flce.flce_block_norm_forward(d, h, y, stats)
        flce.flce_block_norm_backward(d, h, stats, dh, dy, grads, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    new = make(case, seed=5)[0]
    for k, v in leaves(t).items():
        v.copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    want = run(case, t, dh, dy)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    assert torch.equal(dx, want[3]["x"]) and torch.equal(dw, want[3]["weight"])


def test_residual_freed_before_the_backward(gpu_lib):
    """The backward pass needs no residual: its memory may be back with the driver by then."""
    case = (4096, 1024, "bf16", "f32", "rms", False, 0, "none", False)
    t, dh, dy = make(case)
    want = run(case, t, dh, dy)
    x, w = (t[k].clone().requires_grad_() for k in ("x", "weight"))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    residual = t.pop("residual").clone()  # 16 MB: a segment of its own
    h, y = flce.block_norm(x, residual, w, **options(case))
    del residual
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = torch.autograd.grad([h, y], [x, w], [dh, dy])
    assert torch.equal(got[0], want[3]["x"]) and torch.equal(got[1], want[3]["weight"])


def test_saved_tensors_brought_back_elsewhere(gpu_lib):
    """Saved-tensor hooks that give back contiguous copies of strided inputs."""
    case = (6, 512, "bf16", "f32", "layer", True, 3, "tanh", True)
    t, dh, dy = make(case)
    want = run(case, t, dh, dy)
    wide = {k: torch.zeros(v.shape[0], 2 * v.shape[1], dtype=v.dtype, device=DEV)[:, :v.shape[1]].copy_(v)
            for k, v in t.items() if k in ("x", "gate")}
    t.update(wide)
    l = leaves(t)
    for v in l.values():
        v.requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(lambda s: s.detach().cpu(), lambda s: s.to(DEV).contiguous()):
        h, y = flce.block_norm(**t, **options(case))
    got = torch.autograd.grad([h, y], list(l.values()), [dh, dy])
    for (k, g) in zip(l, got):
        assert torch.equal(g, want[3][k]), k


def test_refuses_host_memory_and_mixed_types(gpu_lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    before = flce.flce_kernel_launches()
    for kw, exc in [(dict(residual=x[:2]), ValueError), (dict(residual=x.half()), TypeError), (dict(weight=w[:8]), ValueError),
                    (dict(weight=w.cpu()), ValueError), (dict(weight=w.double()), TypeError), (dict(bias=w), ValueError),
                    (dict(post_bias=w), ValueError), (dict(gate=w[:8]), ValueError), (dict(gate=w), TypeError),
                    (dict(weight=w, norm="batch"), ValueError), (dict(weight=w, gate_activation="relu"), ValueError),
                    (dict(residual=x.t().contiguous().t()), ValueError), (dict(weight=w.repeat(2)[::2]), ValueError),
                    (dict(weight=w, eps=-1.0), flce.FLCEError)]:
        with pytest.raises(exc):
            flce.block_norm(x, **kw)
    d = flce.FlceBlockNormDesc(N=4, D=64, x=x.cpu().pin_memory().data_ptr(), ld_x=64, eps=1e-6, scale=1.0)
    assert flce.flce_block_norm_forward(d, x, None, raise_on_error=False) == 1
    assert flce.flce_last_error_detail() == "x: is host memory, not device memory"
    assert flce.flce_kernel_launches() == before


def test_module(gpu_lib):
    m = flce.BlockNorm(320, norm="layer", post_norm=True, gate_init=0.3, gate_activation="tanh", bias=True, device=DEV,
                       dtype=torch.float32)
    x, r = torch.randn(2, 5, 320, device=DEV), torch.randn(2, 5, 320, device=DEV)
    h, y = m(x, r)
    (h.sum() + y.square().sum()).backward()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in m.parameters())
    out, _ = ref.forward(x.view(-1, 320), r.view(-1, 320), m.gate.detach().view(1, -1), m.post_weight.detach(),
                         m.post_bias.detach(), m.weight.detach(), m.bias.detach(), "layer", m.eps, 1.0, "tanh", 0.0)
    ref.close(y.detach().view(-1, 320), *out["y"], "y")

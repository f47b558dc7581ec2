"""The global gradient norm and clipping on the GPU against 64 bits.

The norm: a thread adds at most 32 squares to each of two 32-bit sums (33 roundings of positive
terms), the rest is in 64 bits, the square root halves the relative error, the result is rounded
once: 20 * 2^-24 covers it. An output has the norm's error, the rounding of the factor and of the
product, and half a step of its type."""
import math

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def norm64(grads, p, scale=1.0):
    if p == 2.0:
        return abs(scale) * math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    return abs(scale) * max([float(g.double().abs().max()) for g in grads if g.numel()], default=0.0)


def check(grads, max_norm, p=2.0, eps=1e-6, scale=1.0, out=None):
    before = [g.clone() for g in grads]
    want = norm64(grads, p, scale)
    total = flce.clip_grad_norm(grads, max_norm, norm_type=p, eps=eps, grad_scale=scale, out=out)
    assert total.shape == () and total.dtype == torch.float32
    assert abs(total.item() - want) <= 20 * U * want
    f = scale * min(1.0, max_norm / (want + eps))
    for b, o in zip(before, out if out is not None else grads):
        ref = b.double() * f
        info = torch.finfo(o.dtype)
        allowed = 24 * U * ref.abs() + ref.abs() * (info.eps / 2) + info.tiny * info.eps
        assert bool(((o.double() - ref).abs() <= allowed).all())
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(before, grads))
    return total


def make(sizes, dtype, seed=0, std=0.1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.empty(n, dtype=dtype, device=DEV).normal_(0, std, generator=g) for n in sizes]


@pytest.mark.parametrize("dtype", list(T))
@pytest.mark.parametrize("p", [2.0, math.inf])
@pytest.mark.parametrize("sizes", [[1], [7, 1, 8], [2047, 2048, 2049], [16384 * 3 + 5, 0, 100000, 9], [5000001, 3]],
                         ids=str)
def test_sizes_and_types(gpu_lib, sizes, dtype, p):
    for max_norm in (1e-3, 1e4):
        check(make(sizes, T[dtype]), max_norm, p)
    for o in T.values():
        check(make(sizes, T[dtype]), 0.5, p, out=[torch.empty(n, dtype=o, device=DEV) for n in sizes])


def test_mixed_types_and_many_tensors(gpu_lib):
    """More tensors than one launch takes, of three types, at every alignment of their elements."""
    room = {t: torch.empty(300000, dtype=t, device=DEV).normal_(0, 0.1) for t in T.values()}
    grads, at = [], 0
    for i in range(2300):
        n = 1 + (i * 37) % 101
        t = list(T.values())[i % 3]
        grads.append(room[t][at:at + n])
        at += n + i % 2
    assert at < 300000
    check(grads, 0.25)
    check(grads, 0.25, math.inf)
    check(grads, math.inf, scale=-0.5)


@pytest.mark.parametrize("off,out_off", [(1, 1), (3, 0), (5, 5), (0, 7)])
@pytest.mark.parametrize("dtype", list(T))
def test_misaligned(gpu_lib, dtype, off, out_off):
    n = 70001
    g = torch.empty(n + 8, dtype=T[dtype], device=DEV).normal_(0, 1)
    o = torch.full((n + 8,), 77.0, device=DEV)
    check([g[off:off + n]], 1.0, out=[o[out_off:out_off + n]])
    assert bool((o[:out_off] == 77).all()) and bool((o[out_off + n:] == 77).all())  # nothing beside it is written
    edge = torch.cat([g[:off], g[off + n:]]).clone()
    check([g[off:off + n]], 1.0)
    assert torch.equal(edge, torch.cat([g[:off], g[off + n:]]))


def test_dense_strides(gpu_lib):
    a = torch.randn(30, 40, device=DEV).t()
    b = torch.randn(6, 5, 4, device=DEV).permute(1, 2, 0)
    check([a, b], 0.1)
    out = [torch.empty_strided(t.shape, t.stride(), device=DEV, dtype=torch.bfloat16) for t in (a, b)]
    check([a, b], 0.01, out=out)
    for bad in ([a[:, ::2]], [a[:1].expand(3, -1)]):
        with pytest.raises(ValueError):
            flce.clip_grad_norm(bad, 1.0)
    with pytest.raises(ValueError):
        flce.clip_grad_norm([a], 1.0, out=[a.contiguous()])


@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e22, 1e30])
def test_range_of_the_squares(gpu_lib, std):
    """Squares beyond fp32 on either side: the norm is still right."""
    check(make([5000, 123], torch.float32, std=std), std)
    check(make([5000, 123], torch.bfloat16, std=std), std, eps=0.0)
    grads = make([5000], torch.float32, std=std) + make([4000], torch.float32, std=1.0)
    check(grads, 1.0)


def test_zeros(gpu_lib):
    for max_norm in (0.0, 1.0):
        g = [torch.zeros(5000, device=DEV), torch.zeros(0, device=DEV)]
        assert flce.clip_grad_norm(g, max_norm, eps=0.0).item() == 0.0 and not g[0].any()
    g = [torch.zeros(0, device=DEV)]
    assert flce.clip_grad_norm(g, 1.0).item() == 0.0
    check(make([100], torch.float32), 0.0)


@pytest.mark.parametrize("p", [2.0, math.inf])
def test_not_finite(gpu_lib, p):
    """As torch.nn.utils.clip_grad_norm_ has it: a NaN reaches everything, an infinite norm makes
    finite gradients 0 and infinite ones NaN."""
    g = make([40000, 50], torch.float32)
    g[0][777] = math.nan
    assert math.isnan(flce.clip_grad_norm(g, 1.0, norm_type=p).item())
    assert all(bool(t.isnan().all()) for t in g)
    g = make([40000, 50], torch.bfloat16)
    g[0][777] = -math.inf
    assert flce.clip_grad_norm(g, 1.0, norm_type=p).item() == math.inf
    assert bool(g[0][777].isnan()) and int(g[0].count_nonzero()) == 1 and not g[1].any()


def test_norm_alone_and_parameters(gpu_lib):
    g = make([3000, 17], torch.float16)
    keep = [t.clone() for t in g]
    for p in (2.0, math.inf):
        want = norm64(g, p, 3.0)
        assert abs(flce.grad_norm(g, p, grad_scale=3.0).item() - want) <= 20 * U * want
    assert all(torch.equal(a, b) for a, b in zip(g, keep))
    ps = [torch.nn.Parameter(torch.zeros_like(t)) for t in g] + [torch.nn.Parameter(torch.zeros(2, device=DEV))]
    for q, t in zip(ps, g):
        q.grad = t
    total = flce.clip_grad_norm_(ps, 0.5)
    want = norm64(keep, 2.0)
    assert abs(total.item() - want) <= 20 * U * want and norm64([ps[0].grad, ps[1].grad], 2.0) <= 0.5 * (1 + 2 ** -10)
    assert flce.clip_grad_norm_(ps[0], 0.5).shape == ()


def test_same_bits_and_launches(gpu_lib):
    sizes = [123456, 77, 9000]
    runs = []
    for _ in range(3):
        g = make(sizes, torch.bfloat16)
        before = flce.flce_kernel_launches()
        total = flce.clip_grad_norm(g, 0.1)
        assert flce.flce_kernel_launches() - before == 2
        runs.append((total, *g))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_graph_and_stream(gpu_lib):
    g = make([50000, 33], torch.float32)
    out = [torch.empty_like(t) for t in g]
    check(g, 0.3, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        total = flce.clip_grad_norm(g, 0.3, out=out)
    for t, new in zip(g, make([50000, 33], torch.float32, seed=9)):
        t.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    want = norm64(g, 2.0)
    assert abs(total.item() - want) <= 20 * U * want
    got = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        flce.clip_grad_norm(g, 0.3, out=out)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out))


def test_refuses(gpu_lib):
    g = torch.ones(10, device=DEV)
    before = flce.flce_kernel_launches()
    for grads, kw, exc in [([g.double()], {}, TypeError), ([g, g.cpu()], {}, ValueError), ([g], dict(max_norm=-1.0), flce.FLCEError),
                           ([g], dict(norm_type=1.0), flce.FLCEError), ([g], dict(out=[g[:5]]), ValueError),
                           ([g], dict(out=[g.int()]), TypeError)]:
        with pytest.raises(exc):
            flce.clip_grad_norm(grads, **{"max_norm": 1.0, **kw})
    host = g.cpu().pin_memory()
    ws = torch.empty(flce.flce_clip_grad_norm_workspace_size(1), dtype=torch.uint8, device=DEV)
    assert flce.flce_clip_grad_norm([(host.data_ptr(), 0, 10, 2, 2)], torch.empty((), device=DEV), ws, 1.0, raise_on_error=False) == 1
    assert flce.flce_last_error_detail() == "gradient: is host memory, not device memory"
    assert flce.flce_kernel_launches() == before


def test_large(gpu_lib):
    """More than 2^31 elements in one tensor: offsets pass 32 bits."""
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    g[-1] = 3.0
    total = flce.clip_grad_norm([g], 1e4)
    want = math.sqrt((n - 1) * 0.25 + 9.0)
    assert abs(total.item() - want) <= 20 * U * want
    f = 1e4 / (want + 1e-6)
    assert abs(g[0].item() - 0.5 * f) <= 0.5 * f * 2.0 ** -7 and abs(g[-1].item() - 3.0 * f) <= 3.0 * f * 2.0 ** -7
    assert bool((g[:-1] == g[0]).all())

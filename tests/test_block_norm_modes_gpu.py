"""The block norm under autograd's other modes: what has no derivative here is refused, saved tensors may
come back with other strides, a training step is captured into a graph."""
import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def make(N, D, x=torch.bfloat16, r=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda s, t, m=0.0: torch.empty(s, device=DEV, dtype=t).normal_(m, 0.7, generator=g)  # noqa: E731
    return {"x": n((N, D), x), "residual": n((N, D), r), "weight": n((D,), r, 1.0), "post_weight": n((D,), r, 1.0),
            "gate": n((2, D), r, 0.3)}


def call(t, **kw):
    return flce.block_norm(t["x"], t["residual"], t["weight"], post_weight=t["post_weight"], gate=t["gate"],
                           gate_activation="sigmoid", norm="layer", **kw)


@pytest.mark.parametrize("name", ["x", "residual", "weight", "post_weight", "gate"])
def test_forward_mode_is_refused(gpu_lib, name):
    """A derivative that is not there is an error, not a zero."""
    t = make(6, 64)
    with torch.autograd.forward_ad.dual_level():
        d = torch.autograd.forward_ad.make_dual(t[name], torch.ones_like(t[name]))
        with pytest.raises((RuntimeError, NotImplementedError)):
            call({**t, name: d})
        call(t)  # other calls at this level are not refused
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.func.jvp(lambda v: call({**t, name: v}), (t[name],), (torch.ones_like(t[name]),))


def test_vmap_is_refused(gpu_lib):
    t = make(6, 64)
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.vmap(lambda x: flce.block_norm(x, None, t["weight"]))(t["x"].unsqueeze(0))


def test_tracing_is_refused(gpu_lib):
    """A trace would keep empty outputs that nothing fills."""
    t = make(6, 64)
    z, s = torch.randn(1, 2, 50, device=DEV), torch.zeros(1, 2, device=DEV)
    parents = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    for f, args in [(lambda x: flce.block_norm(x, None, t["weight"])[1], (t["x"],)), (lambda v: flce.beam_select(v, s)[0], (z,)),
                    (lambda v: flce.beam_reorder([v], parents)[0], (torch.zeros(2, 3, device=DEV),)),
                    (lambda v: flce.clip_grad_norm([v], 1.0), (torch.ones(3, device=DEV),))]:
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(f, args, check_trace=False)


@pytest.mark.parametrize("r", [torch.bfloat16, torch.float32])
def test_saved_tensors_with_other_strides(gpu_lib, r):
    """Saved-tensor hooks that give back the same values in wider rows, parameters among them."""
    t = make(6, 512, r=r)
    g = torch.Generator(device=DEV).manual_seed(5)
    up = [torch.empty(6, 512, device=DEV, dtype=d).normal_(generator=g) for d in (r, torch.bfloat16)]
    leaves = [v.requires_grad_() for v in t.values()]
    want = torch.autograd.grad(call(t), leaves, up)

    def wide(s):
        room = torch.full((*s.shape, 2) if s.dim() == 1 else (s.shape[0], 2 * s.shape[1]), 7.0, dtype=s.dtype, device=DEV)
        view = room[:, 0] if s.dim() == 1 else room[:, :s.shape[1]]
        return view.copy_(s.detach())

    with torch.autograd.graph.saved_tensors_hooks(lambda s: s, wide):
        out = call(t)
    got = torch.autograd.grad(out, leaves, up)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_training_step_in_a_graph(gpu_lib):
    """The public call and its backward pass, captured and replayed on new contents."""
    t = make(64, 768, r=torch.float32)
    leaves = [v.requires_grad_() for v in t.values()]
    up = [torch.ones(64, 768, device=DEV), torch.ones(64, 768, device=DEV, dtype=torch.bfloat16)]

    def step():
        out = call(t)
        return [v.detach() for v in out] + list(torch.autograd.grad(out, leaves, up))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    new = make(64, 768, r=torch.float32, seed=3)
    with torch.no_grad():
        for k, v in t.items():
            v.copy_(new[k])
    graph.replay()
    got = [v.clone() for v in out]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("r", [None, torch.bfloat16, torch.float32])
def test_module_with_parameters_of_another_type(gpu_lib, r):
    """Parameters in fp32, as the module makes them unless told, with 16-bit activations."""
    m = flce.BlockNorm(320, post_norm=True, gate_init=0.3, gate_activation="tanh", device=DEV)
    x = torch.randn(40, 320, device=DEV).bfloat16()
    res = None if r is None else torch.randn(40, 320, device=DEV).to(r)
    h, y = m(x, res)
    (h.float().sum() + y.float().square().sum()).backward()
    assert all(p.dtype == p.grad.dtype == torch.float32 and bool(p.grad.isfinite().all()) for p in m.parameters())
    assert bool(m.gate.grad.any())
    gate = m.gate.detach()
    want = flce.block_norm(x, res, m.weight.detach(), post_weight=m.post_weight.detach(), gate_activation="tanh",
                           gate=gate if r == torch.float32 else gate.bfloat16())
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])


def test_rows_of_more_than_one_stride(gpu_lib):
    """All positions but the first of [B, T, D], for the rows and for gates of their shape."""
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda: torch.empty(3, 7, 264, device=DEV, dtype=torch.bfloat16).normal_(generator=g)[:, 1:]  # noqa: E731
    x, res, gate, w = n(), n(), n(), torch.ones(264, device=DEV)
    up = n()
    outs = []
    for f in (lambda t: t, lambda t: t.contiguous()):
        leaves = [f(t).detach().requires_grad_() for t in (x, res, gate)]
        h, y = flce.block_norm(leaves[0], leaves[1], w, gate=leaves[2], gate_activation="sigmoid")
        assert h.shape == y.shape == (3, 6, 264)
        outs.append([h.detach(), y.detach(), *torch.autograd.grad([h, y], leaves, [up, up])])
    assert all(a.shape == b.shape and torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(flce.block_norm(x, res, w, gate=gate, gate_activation="sigmoid")[1], outs[0][1])
    with pytest.raises(ValueError):  # another stride along D stays refused
        flce.block_norm(x.transpose(1, 2), None, torch.ones(6, device=DEV))

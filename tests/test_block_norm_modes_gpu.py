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

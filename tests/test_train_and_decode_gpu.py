"""The example that runs the operators around the head together: it learns, its gradients are
clipped, and its beams are what an exhaustive evaluation of the same model gives."""
import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu


def test_train_and_decode(gpu_lib):
    from examples import train_and_decode as ex
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    model = ex.Model("cuda")
    losses, norms = ex.train(model, 150, g)
    assert torch.isfinite(losses).all() and torch.isfinite(norms).all()
    assert losses[-10:].mean() < 0.5 * losses[:10].mean()
    total = flce.grad_norm([p.grad for p in model.parameters()])  # of the last step, clipped
    assert total <= min(1.0, norms[-1].item()) * (1 + 2 ** -7)

    B, K, steps = 5, 4, 6
    tokens = ex.sequences(B, g, "cuda")
    found, scores = ex.decode(model, tokens[:, :2].int(), K, steps)
    # a sequence's score is the sum of its tokens' log-probabilities under the model. The logits
    # are rounded to bf16 (2^-8 of up to 32, say) in both, from batches of different sizes:
    # 2^-4 a token covers an input of the softmax that is off by a step.
    with torch.no_grad():
        t = found.long()
        total = torch.zeros(B, K, device="cuda", dtype=torch.float64)
        for i in range(steps):
            y = model.hidden(t[:, :, 1 + i].reshape(-1), model.before[t[:, :, i].reshape(-1)])
            logp = torch.log_softmax((y @ model.head.t()).double(), -1)
            total += logp.gather(1, t[:, :, 2 + i].reshape(-1, 1)).view(B, K)
    assert bool(((total - scores).abs() <= steps * 2.0 ** -4).all())
    assert bool((scores[:, :-1] >= scores[:, 1:]).all())
    assert torch.equal(found[:, :, :2].long(), tokens[:, None, :2].expand(-1, K, -1))
    for b in range(B):
        assert len({tuple(r) for r in found[b].tolist()}) == K  # beams differ

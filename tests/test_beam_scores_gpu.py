"""Scores and order of a beam step where 64-bit sums of logit, score and logsumexp would not do: rows
masked with a lowest value, and beams that are alike."""
import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", list(T))
@pytest.mark.parametrize("V", [5000, 50257])
def test_rows_masked_with_a_lowest_value(gpu_lib, dtype, V):
    """A row of one value, however low, is a uniform distribution: score - log V, below the beam's own."""
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.empty(3, 4, V, device=DEV).normal_(0, 2.5, generator=g).to(T[dtype])
    s = torch.empty(3, 4, device=DEV).normal_(-5, 1.0, generator=g)
    lows = (torch.finfo(T[dtype]).min, -65504.0 if dtype == "f16" else -1e30)
    z[0, 0], z[1, 3] = lows[0], lows[1]
    z[2] = lows[0]  # a request whose beams are all at their end
    for M in (4, 64):
        scores, parents, tokens = flce.beam_select(z, s, M)
        c = torch.log_softmax(z.double(), -1) + s.double()[..., None]
        best, at = torch.sort(c.view(3, -1), dim=1, descending=True, stable=True)
        # half a step of fp32, and eight times what the 32-bit sum of exponentials leaves (2^-23)
        assert bool(((scores.double() - best[:, :M]).abs() <= 2.0 ** -20 + best[:, :M].abs() * 2.0 ** -24).all())
        # no continuation is more probable than what it goes on from
        assert bool((scores <= s.gather(1, parents.long()) + 2.0 ** -20).all())
        mine = c.view(3, -1).gather(1, parents.long() * V + tokens.long())
        assert bool(((mine - best[:, :M]).abs() <= 2.0 ** -20).all())
    # by index within such a row, by score between its equals
    assert tokens[2].tolist() == list(range(64)) and bool((parents[2] == s[2].argmax()).all())


@pytest.mark.parametrize("dtype", list(T))
def test_rows_with_few_tokens_left(gpu_lib, dtype):
    """Few, one and no tokens left in rows masked with -inf and with the type's lowest value."""
    g = torch.Generator(device=DEV).manual_seed(0)
    V, low = 5000, torch.finfo(T[dtype]).min
    z = torch.empty(3, 4, V, device=DEV).normal_(0, 2.5, generator=g).to(T[dtype])
    s = torch.empty(3, 4, device=DEV).normal_(-5, 1.0, generator=g)
    z[0, 0, 3:] = z[0, 1] = z[0, 2, 1:] = z[2] = -torch.inf
    z[0, 3, :4000] = -torch.inf
    z[1, 0], z[1, 1, 5:], z[1, 2, 17:], z[1, 3, 1:] = low, low, low, low
    z[2, 3, 4999] = 1.0
    c = torch.log_softmax(z.double(), -1).nan_to_num(nan=-torch.inf, neginf=-torch.inf) + s.double()[..., None]
    best, at = torch.sort(c.view(3, -1), dim=1, descending=True, stable=True)
    for M in (4, 64):
        scores, parents, tokens = flce.beam_select(z, s, M)
        fine = torch.isfinite(best[:, :M])
        assert torch.equal(fine, torch.isfinite(scores))
        assert bool(((scores.double() - best[:, :M]).abs()[fine] <= 2.0 ** -20 + best[:, :M].abs()[fine] * 2.0 ** -24).all())
        index = parents.long() * V + tokens.long()
        assert bool(((c.view(3, -1).gather(1, index) - best[:, :M]).abs()[fine] <= 2.0 ** -20).all())
        assert torch.equal(index[~fine], at[:, :M][~fine])  # what is no candidate, lowest index first


@pytest.mark.parametrize("dtype", list(T))
@pytest.mark.parametrize("V", [7, 1003, 4099, 50257, 128256 + 5])
def test_beams_that_are_alike_come_in_order(gpu_lib, dtype, V):
    """Equal rows at equal scores are exact ties, wherever their rows start in memory: the lower
    beam first."""
    g = torch.Generator(device=DEV).manual_seed(V)
    for trial in range(4):
        B, K, M = 2, 5, 9
        row = torch.empty(B, 1, V, device=DEV).normal_(0, 2.5, generator=g).to(T[dtype])
        z, s = row.expand(B, K, V).contiguous(), torch.full((B, K), -3.25, device=DEV)
        want = torch.sort(z.double().view(B, -1), dim=1, descending=True, stable=True)[1][:, :M]
        for left in (0, 1, 6):
            room = torch.zeros(B, K, V + 11, dtype=T[dtype], device=DEV)
            room[..., left:left + V] = z
            scores, parents, tokens = flce.beam_select(room[..., left:left + V], s, M)
            assert torch.equal(parents.long(), want // V) and torch.equal(tokens.long(), want % V)
            # and the scores do not depend on the layout either
            assert torch.equal(scores, flce.beam_select(z, s, M)[0])

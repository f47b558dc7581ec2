"""The beam-search step on the GPU against 64 bits: selection with its ties, masks and dead beams,
and the reordering of states of every layout."""
import math

import pytest
import torch

import linear_cross_entropy_tcgen05_gb300 as flce

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def reference(logits, scores, M, finished=None, pad=0):
    """All candidates in 64 bits, sorted stably."""
    B, K, V = logits.shape
    z, s = logits.double().cpu(), scores.double().cpu()
    lse = torch.logsumexp(z, -1)
    c = s[..., None] + z - lse[..., None]
    c[~(torch.isfinite(lse) & torch.isfinite(s))] = -math.inf
    if finished is not None:
        f = finished.cpu().bool()
        c[f] = -math.inf
        c[..., pad] = torch.where(f & torch.isfinite(s), s, c[..., pad])
    best, at = torch.sort(c.view(B, -1), dim=1, descending=True, stable=True)
    return best[:, :M], at[:, :M] // V, at[:, :M] % V, c


def check(logits, scores, M=None, finished=None, pad=0):
    got = flce.beam_select(logits, scores, M, finished=finished, pad_token=pad)
    M = logits.shape[1] if M is None else M
    best, parents, tokens, c = reference(logits, scores, M, finished, pad)
    s, p, t = (v.cpu() for v in got)
    assert s.shape == p.shape == t.shape == (logits.shape[0], M) and s.dtype == torch.float32
    # a score: half a step of fp32, and the 32-bit sum of exponentials (2^-20 is over eight times what
    # its 2^-22 exponentials and at most 40 roundings leave of a relative error, which is absolute in the lse)
    fine = torch.isfinite(best)
    assert torch.equal(fine, torch.isfinite(s)) and bool((s[~fine] == best[~fine].float()).all())
    assert bool(((s.double() - best).abs()[fine] <= 2.0 ** -20 + best.abs()[fine] * 2.0 ** -24).all())
    # the choice is the reference's, but for candidates of different beams that are nearer than 2^-20
    wrong = (p.long() != parents) | (t.long() != tokens)
    if wrong.any():
        at = p.long() * logits.shape[2] + t.long()
        mine = c.view(c.shape[0], -1).gather(1, at)
        assert bool(((mine - best).abs()[wrong] <= 2.0 ** -20).all()), (wrong.nonzero()[:4], mine[wrong][:4], best[wrong][:4])
        assert bool((p.long() != parents)[wrong].all()) and all(len(set(r.tolist())) == M for r in at)
    return got


def make(B, K, V, dtype, seed=0, std=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.empty(B, K, V, device=DEV).normal_(0, std, generator=g).to(T[dtype])
    return z, torch.empty(B, K, device=DEV).normal_(-5, 1.0, generator=g)


@pytest.mark.parametrize("dtype", list(T))
@pytest.mark.parametrize("B,K,V,M", [(1, 1, 1, 1), (2, 1, 7, 3), (3, 2, 8, 16), (1, 4, 1000, 4), (2, 3, 2049, 6), (5, 5, 4099, 10),
                                     (1, 4, 128256, 8), (2, 32, 3001, 64), (1, 32, 50257, 32), (40, 8, 32000, 8),
                                     (300, 2, 511, 4)])
def test_select(gpu_lib, B, K, V, M, dtype):
    check(*make(B, K, V, dtype), M)


def test_first_step_and_dead_beams(gpu_lib):
    z, s = make(4, 4, 3000, "bf16")
    s[:, 1:] = -math.inf  # the first step: one beam is alive
    got = check(z, s, 8)
    assert not got[1].any()
    s[0] = -math.inf      # a request without a beam
    s[1, 0] = math.nan
    s[2, 0] = math.inf
    got = check(z, s, 8)
    for b in range(3):
        assert bool((got[0][b] == -math.inf).all()) and got[2][b].tolist() == list(range(8)) and not got[1][b].any()


@pytest.mark.parametrize("B,K,V,M", [(2, 4, 128256, 8), (3, 16, 50257, 32), (1, 8, 5000, 64)])
def test_first_step_of_long_rows(gpu_lib, B, K, V, M):
    z, s = make(B, K, V, "bf16", seed=3)
    s[:, 1:] = -math.inf
    check(z, s, M)
    s[:, 0], s[:, K - 1] = -math.inf, -3.0
    check(z, s, M)


def test_few_tokens_left_in_long_rows(gpu_lib):
    """Constrained decoding: a few tokens, or one run of them, and many rows of equal values."""
    z, s = make(2, 4, 60000, "bf16")
    keep = z.clone()
    z.fill_(-math.inf)
    for v in (5, 777, 30001, 59999):
        z[:, :, v] = keep[:, :, v]
    check(z, s, 8)
    check(z, s, 40)
    z[:, :, 1000:6000] = keep[:, :, 1000:6000]
    check(z, s, 16)
    z[:, :, 1000:6000] = 2.5
    check(z, s, 16)
    z.fill_(torch.finfo(z.dtype).min)  # masked with the lowest value: thousands of equal scores far below
    for v in (5, 59999):
        z[:, :, v] = keep[:, :, v]
    check(z, s, 8)
    check(z, s, 24)


@pytest.mark.parametrize("dtype", list(T))
def test_masked_tokens(gpu_lib, dtype):
    """Rows with few, one and no tokens left, with -inf and with the type's lowest value."""
    z, s = make(3, 4, 5000, dtype)
    low = torch.finfo(T[dtype]).min
    z[0, 0, 3:] = -math.inf
    z[0, 1] = -math.inf
    z[0, 2, 1:] = -math.inf
    z[0, 3, :4000] = -math.inf
    z[1, 0] = low
    z[1, 1, 5:] = low
    z[1, 2, 17:] = low
    z[1, 3, 1:] = low
    z[2] = -math.inf
    z[2, 3, 4999] = 1.0
    check(z, s, 4)
    check(z, s, 64)


@pytest.mark.parametrize("B,K,V,M", [(16, 8, 128256, 8), (2, 16, 4000, 32), (3, 5, 8000, 64), (1, 32, 70001, 64)])
def test_one_beam_far_ahead(gpu_lib, B, K, V, M):
    """All candidates are one beam's, whichever it is."""
    for ahead in (0, K // 2, K - 1):
        z, s = make(B, K, V, "bf16", seed=ahead, std=1.0)
        s[:, ahead] += 12.0
        got = check(z, s, M)
        assert bool((got[1] == ahead).all())


def test_scores_below_the_range_still_fill(gpu_lib):
    """Masks of the lowest value on tokens and on a beam: sums that fp32 does not have come last."""
    low = torch.finfo(torch.float32).min
    z = torch.full((1, 2, 3), low, device=DEV)
    z[..., 0] = 0.0
    s = torch.tensor([[0.0, low]], device=DEV)
    scores, parents, tokens = (v[0].tolist() for v in flce.beam_select(z, s, 6))
    # beam 0: 0 and twice low; beam 1: low, equal to those and after them, and twice 2 low
    assert list(zip(parents, tokens)) == [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (1, 2)]
    assert scores == [0.0, low, low, low, -math.inf, -math.inf]


def test_bad_logits(gpu_lib):
    """A NaN or an infinity in a row takes the row out, wherever it stands."""
    for bad in (math.nan, math.inf):
        for at in (0, 7, 2048, 4998):
            z, s = make(1, 3, 4999, "f32")
            z[0, 1, at] = bad
            got = check(z, s, 6)
            assert not (got[1] == 1).any()
    z, s = make(1, 2, 900, "f32")
    z[0, 0] = math.nan
    z[0, 1] = -math.inf
    z[0, 1, 3] = math.nan
    got = check(z, s, 5)
    assert bool((got[0] == -math.inf).all()) and got[2][0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("K,V,M", [(1, 9000, 64), (4, 9000, 8), (32, 5000, 64), (3, 40, 64)])
def test_ties(gpu_lib, K, V, M):
    """All equal, equal in halves, few distinct values, sorted either way: the lowest index first."""
    s = torch.zeros(2, K, device=DEV)
    z = torch.zeros(2, K, V, device=DEV)
    for w in (z, (torch.arange(V, device=DEV) % 2).float().expand(2, K, V).contiguous(),
              torch.randint(3, (2, 1, V), device=DEV).float().expand(2, K, V).contiguous(),
              (torch.arange(V, device=DEV).float() * 2 ** -6).expand(2, K, V).contiguous(),
              (torch.arange(V, 0, -1, device=DEV).float() * 2 ** -6).expand(2, K, V).contiguous(), -z):
        check(w, s, M)
    # beams that are alike bit for bit: exact ties between beams, the lower beam first
    got = flce.beam_select(z, s, min(M, K * V))
    at = torch.arange(min(M, K * V), device=DEV, dtype=torch.int32).expand(2, -1)
    assert torch.equal(got[1], at // V) and torch.equal(got[2], at % V)


def test_negative_zero_is_zero(gpu_lib):
    z = torch.zeros(1, 1, 100, device=DEV)
    z[0, 0, ::2] = -0.0
    assert flce.beam_select(z, torch.zeros(1, 1, device=DEV), 6)[2][0].tolist() == [0, 1, 2, 3, 4, 5]


def test_finished_beams(gpu_lib):
    z, s = make(6, 5, 2000, "bf16")
    f = torch.zeros(6, 5, dtype=torch.bool, device=DEV)
    f[0, 2] = f[1, :] = f[2, 0] = f[2, 4] = True
    f[3, 1] = True
    s[3, 1] = -math.inf
    z[0, 2] = math.nan  # the logits of a finished beam are not looked at
    for pad in (0, 3, 1999):
        for M in (5, 12):
            check(z, s, M, f, pad)
    got = flce.beam_select(z, s, 5, finished=f, pad_token=7)
    assert bool((got[2][1] == 7).all()) and sorted(got[1][1].tolist()) == [0, 1, 2, 3, 4]
    assert torch.equal(got[0][1], s[1].sort(descending=True).values)


def test_strided_and_misaligned_logits(gpu_lib):
    for dtype in T:
        z, s = make(3, 4, 1003, dtype)
        room = torch.full((4, 3, 1100), math.nan, dtype=T[dtype], device=DEV)
        for left in (0, 1, 5, 8):
            room[..., left:left + 1003] = z.transpose(0, 1)
            view = room[..., left:left + 1003].transpose(0, 1)
            got = check(view, s, 7)
            # the choice does not depend on the layout (a score's last bits may: the sum of
            # exponentials is grouped by the alignment of the row)
            assert all(torch.equal(a, b) for a, b in zip(got[1:], flce.beam_select(z, s, 7)[1:]))


def test_select_offsets_past_32_bits(gpu_lib):
    B, K, V = 40, 8, 1 << 23
    z = torch.zeros(B, K, V, dtype=torch.bfloat16, device=DEV)
    s = torch.zeros(B, K, device=DEV)
    at = torch.randint(V, (B, K), device=DEV)
    z.scatter_(2, at[..., None], 20.0)
    s += torch.arange(K, device=DEV) * -0.5
    got = flce.beam_select(z, s, 8)
    assert torch.equal(got[1], torch.arange(K, device=DEV, dtype=torch.int32).expand(B, K)) and torch.equal(got[2].long(), at)


def gather(state, parents, dim):
    B, K = parents.shape
    rows = (torch.arange(B, device=DEV)[:, None] * K + parents.long()).flatten()
    return state.index_select(dim, rows)


STATES = [((8,), 0, torch.bool), ((8, 7), 0, torch.int64), ((3, 8, 5), 1, torch.float32), ((2, 8, 3, 17, 24), 1, torch.bfloat16),
          ((8, 1), 0, torch.int32), ((5, 8), 1, torch.uint8), ((2, 2, 8, 9), 2, torch.float16), ((8, 4096), 0, torch.float32)]


@pytest.mark.parametrize("B,K", [(1, 8), (2, 4), (8, 1), (4, 2)])
def test_reorder(gpu_lib, B, K):
    g = torch.Generator(device=DEV).manual_seed(B)
    for trial in range(3):
        parents = torch.randint(K, (B, K), generator=g, device=DEV, dtype=torch.int32)
        if trial == 2:
            parents = torch.arange(K, device=DEV, dtype=torch.int32).flip(0).repeat(B, 1)
        states = [torch.randint(0, 2 if t == torch.bool else 100, s, generator=g, device=DEV).to(t) for s, _, t in STATES]
        dims = [d for _, d, _ in STATES]
        want = [gather(s, parents, d) for s, d in zip(states, dims)]
        before = flce.flce_kernel_launches()
        out = flce.beam_reorder(states, parents, dims, out=[torch.empty_like(s) for s in states])
        assert flce.flce_kernel_launches() - before == 1
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        got = flce.beam_reorder(states, parents, dims)
        assert all(a is b for a, b in zip(got, states)) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("K", [3, 9, 17, 32])
def test_reorder_many_beams(gpu_lib, K):
    parents = torch.randint(K, (3, 2 * K), device=DEV, dtype=torch.int32)[:, :K]  # a strided view, as of 2K candidates
    s = torch.randn(2, 3 * K, 100, 3, device=DEV)
    want = gather(s, parents, 1)
    assert torch.equal(flce.beam_reorder([s], parents, 1)[0], want)


def test_reorder_views(gpu_lib):
    """The first positions of a long cache alone, other layouts for the output, odd bytes."""
    parents = torch.tensor([[2, 0, 2], [1, 1, 0]], dtype=torch.int32, device=DEV)
    cache = torch.randn(2, 6, 4, 50, 16, device=DEV).bfloat16()
    keep = cache.clone()
    view = cache[:, :, :, :13]
    want = gather(view, parents, 1)
    flce.beam_reorder([view], parents, 1)
    assert torch.equal(view, want) and torch.equal(cache[:, :, :, 13:], keep[:, :, :, 13:])
    out = torch.zeros(2, 6, 13, 4, 16, device=DEV, dtype=torch.bfloat16).transpose(2, 3)
    flce.beam_reorder([keep[:, :, :, :13]], parents, 1, out=[out])
    assert torch.equal(out, want)
    odd = torch.randint(100, (6, 33), device=DEV, dtype=torch.uint8)[:, 1:30]
    w = gather(odd, parents, 0)
    flce.beam_reorder([odd], parents)
    assert torch.equal(odd, w)
    dims = torch.randn(3, 5, 6, 7, 9, 11, device=DEV)[:, :4, :, :6, :8, :10]
    w = gather(dims, parents, 2)
    assert torch.equal(flce.beam_reorder([dims], parents, 2)[0], w)
    assert flce.beam_reorder([torch.zeros(6, 0, device=DEV)], parents)[0].shape == (6, 0)


def test_reorder_bad_parents_keep_the_beam(gpu_lib):
    parents = torch.tensor([[5, -1, 0]], dtype=torch.int32, device=DEV)
    s = torch.arange(3, device=DEV, dtype=torch.float32)[:, None].repeat(1, 20)
    out = flce.beam_reorder([s], parents, out=[torch.empty_like(s)])[0]
    assert out[:, 0].tolist() == [0.0, 1.0, 0.0]


def test_reorder_many_states(gpu_lib):
    parents = torch.tensor([[1, 0], [0, 0], [1, 1]], dtype=torch.int32, device=DEV)
    states = [torch.randn(6, 1 + i % 5, device=DEV) for i in range(150)]
    want = [gather(s, parents, 0) for s in states]
    assert all(torch.equal(a, b) for a, b in zip(flce.beam_reorder(states, parents), want))


def test_reorder_offsets_past_32_bits(gpu_lib):
    parents = torch.tensor([[1, 0], [0, 0]], dtype=torch.int32, device=DEV)
    s = torch.zeros(4, 3 << 30, dtype=torch.uint8, device=DEV)
    for k in range(4):
        s[k, -5:] = k + 1
        s[k, :3] = 10 + k
    flce.beam_reorder([s], parents)
    assert s[:, -1].tolist() == [2, 1, 3, 3] and s[:, 0].tolist() == [11, 10, 12, 12]


def test_refuses(gpu_lib):
    z, s = make(2, 3, 50, "f32")
    p = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    before = flce.flce_kernel_launches()
    for args, kw, exc in [((z, s, 0), {}, ValueError), ((z, s, 151), {}, ValueError), ((z, s, 65), {}, flce.FLCEError),
                          ((z, s.cpu()), {}, ValueError), ((z.transpose(1, 2), s), {}, ValueError),
                          ((z, s), dict(finished=s), TypeError), ((z, s), dict(finished=s[:1].bool()), ValueError),
                          ((z, s), dict(finished=s.bool(), pad_token=50), flce.FLCEError)]:
        with pytest.raises(exc):
            flce.beam_select(*args, **kw)
    st = torch.zeros(4, 6, 5, device=DEV)
    for states, kw, exc in [([st], {}, ValueError), ([st], dict(dims=2), ValueError), ([st], dict(dims=5), ValueError),
                            ([st], dict(dims=1, out=[]), ValueError), ([st], dict(dims=1, out=[st.half()]), ValueError),
                            ([st], dict(dims=[1, 1]), ValueError), ([st.cpu()], dict(dims=1), ValueError),
                            ([st[:1].expand(4, 6, 5)], dict(dims=1), ValueError)]:
        with pytest.raises(exc):
            flce.beam_reorder(states, p, **kw)
    assert flce.flce_kernel_launches() == before


def test_graph_and_stream(gpu_lib):
    z, s = make(4, 4, 5000, "bf16")
    cache = torch.randn(2, 16, 300, device=DEV)
    nxt = torch.empty_like(cache)

    def step():
        out = flce.beam_select(z, s)
        flce.beam_reorder([cache], out[1], 1, out=[nxt])
        return out

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    z2, s2 = make(4, 4, 5000, "bf16", seed=4)
    z.copy_(z2)
    s.copy_(s2)
    graph.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in out]
    assert torch.equal(nxt, gather(cache, got[1], 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    check(z, s)


def test_empty_batch(gpu_lib):
    out = flce.beam_select(torch.zeros(0, 3, 10, device=DEV), torch.zeros(0, 3, device=DEV))
    assert [v.shape for v in out] == [(0, 3)] * 3

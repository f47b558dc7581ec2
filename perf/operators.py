"""Cases that measure the operators around the language-model head: the block norm (norms after and
before a block with its gate and residual scale, forward and backward), the global gradient norm with
clipping, and a beam-search step (selection over beams and vocabulary, reordering of the states).

``own`` False computes the plain form (elementary torch operations in 32 bits, or in 64 where an order
is decided); True makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    norm = {"op": "norm", "res": "same", "post": True, "gate": "none", "act": "none", "norm": "rms", "bias": False,
            "train": False}
    return [
        # one token of one sequence between two blocks: launch latency is all there is
        dict(norm, name="norm 1 token", N=1, D=4096, dtype="bf16"),
        # a decode batch of 48 sequences with a learned gate for each channel, layer norms
        dict(norm, name="norm decode batch", N=48, D=5120, dtype="f16", norm="layer", bias=True, gate="channel"),
        # a prompt of 8192 tokens at the head's width, residual stream kept in 32 bits
        dict(norm, name="norm prompt", N=8192, D=4096, dtype="bf16", res="f32"),
        # the training step in front of the loss at the headline workload's rows and width
        dict(norm, name="norm train headline", N=65536, D=4096, dtype="bf16", train=True),
        # training with a tanh gate for each of 16 sequences, layer norms, 32-bit residual stream and parameters
        dict(norm, name="norm train gated", N=16384, D=2304, dtype="bf16", res="f32", norm="layer", bias=True,
             gate="group", groups=16, act="tanh", train=True),
        # odd width and rows, a sigmoid gate for each token, everything in 32 bits, no norm after the block
        dict(norm, name="norm train odd", N=1777, D=1001, dtype="f32", norm="layer", bias=True, gate="full",
             act="sigmoid", post=False, train=True),
        # a small model's gradients, clipped in place
        {"op": "clip", "name": "clip small", "tensors": 12, "total": 50000, "dtype": "f32", "out": "same", "p": 2.0},
        # bf16 gradients of a few blocks, into the 32-bit gradients that an optimizer reads
        {"op": "clip", "name": "clip blocks", "tensors": 44, "total": 218000000, "dtype": "bf16", "out": "f32", "p": 2.0},
        # the head's 32-bit dW at the headline workload beside small tensors, in place
        {"op": "clip", "name": "clip head", "tensors": 9, "total": 525340672, "dtype": "f32", "out": "same", "p": 2.0},
        # one request with four beams; the cache of a shallow model
        {"op": "beam", "name": "beam 1 x 4", "B": 1, "K": 4, "V": 128256, "M": 4, "dtype": "bf16", "finished": False,
         "layers": 2, "row": 4096, "T": 37, "inplace": False},
        # a batch of requests, some of their beams finished, 32-bit logits of the 32000 vocabulary
        {"op": "beam", "name": "beam 48 x 6", "B": 48, "K": 6, "V": 32000, "M": 6, "dtype": "f32", "finished": True,
         "layers": 4, "row": 1024, "T": 211, "inplace": True},
        # the widest vocabulary, twice as many candidates as beams, a long cache
        {"op": "beam", "name": "beam 16 x 16", "B": 16, "K": 16, "V": 256000, "M": 32, "dtype": "bf16", "finished": False,
         "layers": 4, "row": 1024, "T": 900, "inplace": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "beam"])
    if op == "norm":
        D = _log(rng, 64, 8192)
        D = D if rng.random() < 0.3 else max(64, D // 64 * 64)
        N = _log(rng, 1, min(65536, 65536 * 4096 // D))
        gate = rng.choice(["none", "channel", "group", "full"])
        dtype = rng.choice(["bf16", "f16", "f32"])
        c = {"op": "norm", "N": N, "D": D, "dtype": dtype, "res": rng.choice(["same", "f32"]),
             "post": rng.random() < 0.6, "gate": gate, "act": rng.choice(["none", "sigmoid", "tanh"]) if gate != "none" else "none",
             "norm": rng.choice(["rms", "layer"]), "bias": rng.random() < 0.5, "train": rng.random() < 0.6}
        if dtype == "f32" or gate == "full":  # no dearer than the largest listed case
            c["N"] = max(1, N // 2)
        if gate == "group":
            c["groups"] = rng.randint(2, 32)
            c["N"] = c["groups"] * max(1, c["N"] // c["groups"])
        return c
    if op == "clip":
        tensors = _log(rng, 1, 56)
        dtype = rng.choice(["bf16", "f16", "f32"])
        return {"op": "clip", "tensors": tensors, "total": max(8 * tensors, _log(rng, 1000, 300000000)), "dtype": dtype,
                "out": rng.choice(["same", "f32"]), "p": rng.choice([2.0, 2.0, math.inf])}
    K = rng.randint(1, 16)
    V = _log(rng, 1000, 256000)
    B = _log(rng, 1, min(64, max(1, 16 * 16 * 256000 // (K * V))))
    row = 64 * _log(rng, 1, 32)
    layers = rng.randint(1, 4)
    T = _log(rng, 1, max(1, min(2000, 900 * 16 * 16 * 4096 // (B * K * row * layers))))
    return {"op": "beam", "B": B, "K": K, "V": V, "M": rng.choice([K, 2 * K]), "dtype": rng.choice(["bf16", "f16", "f32"]),
            "finished": rng.random() < 0.5, "layers": layers, "row": row, "T": T, "inplace": rng.random() < 0.4}


def _tensor_sizes(case):
    """Ragged sizes that add up to the case's total: a few large ones, many of medium and odd size."""
    n, total = case["tensors"], case["total"]
    share = [1.0 / (1 + i % 7 * 3 + (i % 3)) ** 2 for i in range(n)]
    sizes = [max(1, int(total * s / sum(share)) - (i % 5)) for i, s in enumerate(share)]
    sizes[0] += max(0, total - sum(sizes))
    return sizes


def _normal(g, shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        N, D, t = case["N"], case["D"], DTYPES[case["dtype"]]
        tr = t if case["res"] == "same" else torch.float32  # the parameters have the residual stream's type
        rows = {"none": 0, "channel": 1, "group": case.get("groups", 1), "full": N}[case["gate"]]
        s["x"] = _normal(g, (N, D), t, 1.5, 0.2)
        s["residual"] = _normal(g, (N, D), tr, 2.0, -0.1)
        s["gate"] = _normal(g, (rows, D), tr, 0.7, 0.3) if rows else None
        s["weight"] = _normal(g, (D,), tr, 0.2, 1.0)
        s["post_weight"] = _normal(g, (D,), tr, 0.2, 1.0) if case["post"] else None
        s["bias"] = _normal(g, (D,), tr, 0.2) if case["bias"] else None
        s["post_bias"] = _normal(g, (D,), tr, 0.2) if case["bias"] and case["post"] else None
        if case["train"]:
            s["dh"] = _normal(g, (N, D), tr, 0.05)
            s["dy"] = _normal(g, (N, D), t, 0.05)
            s["leaves"] = [s[k].requires_grad_() for k in NAMES if s[k] is not None]
    elif case["op"] == "clip":
        t = DTYPES[case["dtype"]]
        sizes = _tensor_sizes(case)
        s["grads"] = [_normal(g, (n,), t, 0.02 / (1 + i % 4)) for i, n in enumerate(sizes)]
        s["out"] = [torch.empty(n, dtype=torch.float32, device="cuda") for n in sizes] if case["out"] == "f32" else None
        s["max_norm"] = 0.01 if case["p"] == math.inf else 1e-3 * math.sqrt(case["total"])
    else:
        B, K, V, t = case["B"], case["K"], case["V"], DTYPES[case["dtype"]]
        # a few tokens stand out of the noise of the vocabulary, as in a trained model's answers
        z = _normal(g, (B, K, V), torch.float32, 1.7)
        top = torch.randint(V, (B, K, min(V, 40)), generator=g, device="cuda")
        s["logits"] = z.scatter_add_(2, top, _normal(g, top.shape, torch.float32, 2.0, 7.0)).to(t)
        del z
        s["scores"] = _normal(g, (B, K), torch.float32, 1.0, -9.0)
        s["finished"] = torch.rand(B, K, generator=g, device="cuda") < 0.25 if case["finished"] else None
        s["cache"] = _normal(g, (case["layers"], B * K, case["T"], case["row"]), torch.bfloat16)
        s["history"] = torch.randint(V, (B * K, case["T"]), generator=g, device="cuda", dtype=torch.int32)
        # parents of the K beams that go on: the next step's states have the same number of beams
        s["next"] = None if case["inplace"] else [torch.empty_like(s["cache"]), torch.empty_like(s["history"])]
    return s


NAMES = ("x", "residual", "gate", "weight", "post_weight", "bias", "post_bias")


def _plain_norm(v, weight, bias, kind, eps=1e-6):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * weight
    return v + bias if bias is not None else v


def _plain_block(s, case):
    f = {k: s[k].float() if s[k] is not None else None for k in NAMES}
    u = _plain_norm(f["x"], f["post_weight"], f["post_bias"], case["norm"]) if case["post"] else f["x"]
    if f["gate"] is not None:
        a = {"none": lambda v: v, "sigmoid": lambda v: 1 / (1 + torch.exp(-v)), "tanh": torch.tanh}[case["act"]](f["gate"])
        u = (u.unflatten(0, (a.shape[0], -1)) * a.unsqueeze(1)).flatten(0, 1)
    h = f["residual"] + SCALE * u
    y = _plain_norm(h, f["weight"], f["bias"], case["norm"])
    return h.to(s["residual"].dtype), y.to(s["x"].dtype)


SCALE = 0.7


def _run_norm(s, case):
    if own:
        import linear_cross_entropy_tcgen05_gb300 as flce
        h, y = flce.block_norm(s["x"], s["residual"], s["weight"], bias=s["bias"], post_weight=s["post_weight"],
                               post_bias=s["post_bias"], gate=s["gate"], gate_activation=case["act"], scale=SCALE,
                               norm=case["norm"], eps=1e-6)
    else:
        h, y = _plain_block(s, case)
    if not case["train"]:
        return h, y
    return (h.detach(), y.detach(), *torch.autograd.grad((h, y), s["leaves"], (s["dh"], s["dy"])))


def _run_clip(s, case):
    if own:
        import linear_cross_entropy_tcgen05_gb300 as flce
        total = flce.clip_grad_norm(s["grads"], s["max_norm"], norm_type=case["p"], out=s["out"])
    else:
        if case["p"] == 2.0:
            total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
        else:
            total = torch.stack([g.abs().amax().double() for g in s["grads"]]).amax()
        c = (s["max_norm"] / (total + 1e-6)).clamp(max=1.0).float()
        total = total.float()
        [o.copy_(g.float() * c) for o, g in zip(s["out"] or s["grads"], s["grads"])]
    return [total, *(s["out"] or s["grads"])]


def _plain_select(s, case):
    B, K, V = s["logits"].shape
    z = s["logits"].double()
    m = z.amax(-1, keepdim=True)
    lse = m + (z - m).exp().sum(-1, keepdim=True).log()
    z = z.sub_(lse).add_(s["scores"].double().unsqueeze(-1))
    if s["finished"] is not None:  # a finished beam goes on with its score and the padding token alone
        only = torch.full((V,), -math.inf, dtype=torch.float64, device=z.device)
        only[PAD] = 0
        z = torch.where(s["finished"].unsqueeze(-1), s["scores"].double().unsqueeze(-1) + only, z)
    z = z.view(B, K * V)
    least = z.topk(case["M"], dim=1).values[:, -1:]
    more = (z > least).sum(1, keepdim=True)
    tie = z == least
    keep = (z > least) | (tie & (tie.cumsum(1) <= case["M"] - more))
    at = K * V - (keep * torch.arange(K * V, 0, -1, device=z.device)).topk(case["M"], dim=1).values
    best, order = torch.sort(z.gather(1, at), dim=1, descending=True, stable=True)
    at = at.gather(1, order)
    return best.float(), (at // V).int(), (at % V).int()


PAD = 2


def _run_beam(s, case):
    if own:
        import linear_cross_entropy_tcgen05_gb300 as flce
        scores, parents, tokens = flce.beam_select(s["logits"], s["scores"], case["M"], finished=s["finished"], pad_token=PAD)
        cache, history = flce.beam_reorder([s["cache"], s["history"]], parents[:, : case["K"]], dims=[1, 0], out=s["next"])
    else:
        scores, parents, tokens = _plain_select(s, case)
        first = torch.arange(0, case["B"] * case["K"], case["K"], device=parents.device).unsqueeze(1)
        rows = (first + parents[:, : case["K"]]).flatten()
        cache, history = s["next"] or (s["cache"], s["history"])
        cache.copy_(s["cache"][:, rows])
        history.copy_(s["history"][rows])
    return scores, parents, tokens, cache, history


def run(state):
    case = state["case"]
    return {"norm": _run_norm, "clip": _run_clip, "beam": _run_beam}[case["op"]](state, case)


def work(case):
    if case["op"] == "norm":
        n, e, r = case["N"] * case["D"], SIZES[case["dtype"]], 4 if case["res"] == "f32" else SIZES[case["dtype"]]
        rows = {"none": 0, "channel": 1, "group": case.get("groups", 1), "full": case["N"]}[case["gate"]]
        params = (rows + 1 + case["post"] + case["bias"] * (1 + case["post"])) * case["D"] * r
        forward, backward = n * 2 * (e + r) + params, n * (2 * e + 2 * r) + params
        # a training step reads x, the residual, dh and dy, and writes h, y, dx and the residual's gradient
        return {"bytes": forward + (backward if case["train"] else 0), "flops": n * (14 + 30 * case["train"])}
    if case["op"] == "clip":
        e = SIZES[case["dtype"]]
        return {"bytes": case["total"] * (e + (4 if case["out"] == "f32" else e)), "flops": 3 * case["total"]}
    logits = case["B"] * case["K"] * case["V"]
    state = case["B"] * case["K"] * case["T"] * (case["layers"] * case["row"] * 2 + 4)
    return {"bytes": logits * SIZES[case["dtype"]] + 2 * state + case["B"] * (5 * case["K"] + 12 * case["M"]), "flops": 5 * logits}


def _exact_norm(case, s):
    """Forward and gradients from the formulas, in 64 bits."""
    v = {k: s[k].detach().double() if s.get(k) is not None else None for k in NAMES + ("dh", "dy")}
    D, layer = case["D"], case["norm"] == "layer"

    def normed(t):
        mean = t.sum(1, keepdim=True) / D if layer else 0.0
        r = 1.0 / torch.sqrt(((t - mean) ** 2).sum(1, keepdim=True) / D + 1e-6)
        return (t - mean) * r, r

    def back(g, n, r):
        g = g - n * ((g * n).sum(1, keepdim=True) / D) - (g.sum(1, keepdim=True) / D if layer else 0.0)
        return g * r

    n1 = r1 = None
    u = v["x"]
    if case["post"]:
        n1, r1 = normed(u)
        u = n1 * v["post_weight"]
        if v["post_bias"] is not None:
            u = u + v["post_bias"]
    a = da = None
    if v["gate"] is not None:
        each = case["N"] // v["gate"].shape[0]
        t = v["gate"].repeat_interleave(each, 0)
        if case["act"] == "sigmoid":
            a = torch.sigmoid(t)
            da = a * (1 - a)
        elif case["act"] == "tanh":
            a = torch.tanh(t)
            da = 1 - a * a
        else:
            a, da = t, None
        del t
    h = v["residual"] + SCALE * (u * a if a is not None else u)
    n2, r2 = normed(h)
    y = n2 * v["weight"]
    if v["bias"] is not None:
        y = y + v["bias"]
    if not case["train"]:
        return h, y
    d = {"weight": (v["dy"] * n2).sum(0), "bias": v["dy"].sum(0)}
    dh = v["dh"] + back(v["dy"] * v["weight"], n2, r2)
    del n2, r2
    d["residual"] = dh
    du = SCALE * dh
    if a is not None:
        dg = du * u if da is None else du * u * da
        d["gate"] = dg.view(v["gate"].shape[0], -1, D).sum(1)
        du = du * a
        del dg, a, da
    d["x"] = du
    if case["post"]:
        d["post_weight"] = (du * n1).sum(0)
        d["post_bias"] = du.sum(0)
        d["x"] = back(du * v["post_weight"], n1, r1)
    return (h, y, *[d[k] for k in NAMES if s[k] is not None])


def _exact_clip(case, s):
    if case["p"] == 2.0:
        total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
    else:
        total = max(float(g.double().abs().max()) for g in s["grads"])
    c = min(1.0, s["max_norm"] / (total + 1e-6))
    return [torch.tensor(total, dtype=torch.float64), *[g.double() * c for g in s["grads"]]]


def _exact_beam(case, s):
    B, K, V, M = case["B"], case["K"], case["V"], case["M"]
    c = torch.log_softmax(s["logits"].double(), -1) + s["scores"].double()[..., None]
    if s["finished"] is not None:
        c[s["finished"]] = -math.inf
        c[..., PAD][s["finished"]] = s["scores"].double()[s["finished"]]
    best, at = zip(*[[t[:M] for t in torch.sort(row.flatten(), descending=True, stable=True)] for row in c])
    best, at = torch.stack(best), torch.stack(at)
    parents = (at // V).int()
    rows = (parents[:, :K] + torch.arange(B, device=parents.device, dtype=torch.int32)[:, None] * K).flatten()
    return best, parents, (at % V).int(), s["cache"].index_select(1, rows), s["history"].index_select(0, rows)


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "clip": _exact_clip, "beam": _exact_beam}[case["op"]](case, s)

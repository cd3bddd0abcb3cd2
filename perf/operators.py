"""Scoring of given tokens: the cases that are measured, their inputs and their plain forms.

Three operators over a language model's output distribution:

  score  log probabilities of given tokens, with entropy, rank and the n most likely
         alternatives, from logits [B, V] under per-row temperatures and legal-token masks;
  grad   the gradient of those log probabilities and entropies with respect to the logits;
  head   log probabilities and entropy straight from hidden states [N, D] and the output
         head's weights [V, D], without the [N, V] logits.

The plain forms use elementary torch operations in float32; ``exact`` has the definitions in
float64.  With ``own`` set, ``run`` calls the library's operators instead.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}
OK, EMPTY = 0, 1
LIMIT = 4096 * 128256         # logits of the largest score / grad case
HEAD_LIMIT = 4096 * 128256 * 4096  # products of the largest head case


def listed():
    return [
        # one decode step of one sequence that reports the 20 best alternatives: latency
        dict(name="score_1x128256_bf16_top20", op="score", B=1, V=128256, pad=0, dtype="bf16", n=20, masked=False),
        # a small batch's decode step, float32 logits, a few alternatives
        dict(name="score_64x32000_f32_top5", op="score", B=64, V=32000, pad=0, dtype="f32", n=5, masked=False),
        # grammar-constrained decode: packed legal-token masks, one row that allows nothing
        dict(name="score_512x151936_bf16_mask_top8", op="score", B=512, V=151936, pad=0, dtype="bf16", n=8,
             masked=True),
        # a large decode batch with the most alternatives that a call gives
        dict(name="score_1024x256000_f16_top32", op="score", B=1024, V=256000, pad=0, dtype="f16", n=32,
             masked=False),
        # log probabilities of a prompt's tokens, an odd number of them, no alternatives
        dict(name="score_4093x128256_bf16", op="score", B=4093, V=128256, pad=0, dtype="bf16", n=0, masked=False),
        # fine-tuning of a small vocabulary of odd size: rows that start at any alignment
        dict(name="grad_37x50001_f32", op="grad", B=37, V=50001, pad=0, dtype="f32", entropy=False, masked=False),
        # policy gradient with an entropy bonus over masked rows, padded row stride
        dict(name="grad_256x151936_f16_mask_entropy", op="grad", B=256, V=151936, pad=64, dtype="f16",
             entropy=True, masked=True),
        # a training step's cross entropy: the largest logits
        dict(name="grad_4096x128256_bf16", op="grad", B=4096, V=128256, pad=0, dtype="bf16", entropy=False,
             masked=False),
        # one token's score without its logits: the head's weights are read once
        dict(name="head_1x128256x4096_bf16", op="head", N=1, V=128256, D=4096, dtype="bf16"),
        # a short ragged prompt on a small head, sizes that fill no tile
        dict(name="head_203x32001x1000_f16", op="head", N=203, V=32001, D=1000, dtype="f16"),
        # a long prompt on a large head: bound by the matrix product
        dict(name="head_4096x128256x4096_bf16", op="head", N=4096, V=128256, D=4096, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "score", "grad", "grad", "head"])
    if op == "head":
        V, D = _log_int(rng, 200, 128256), 8 * (2 * _log_int(rng, 4, 320) + rng.choice([-1, 1]))
        N = _log_int(rng, 1, max(1, min(4096, HEAD_LIMIT // (V * D))))
        return dict(op=op, N=N, V=V, D=D, dtype=rng.choice(["bf16", "f16"]))
    V = _log_int(rng, 100, 262143)
    case = dict(op=op, B=_log_int(rng, 1, max(1, min(4096, LIMIT // (2 * V)))), V=V, pad=rng.choice([0, 1, -V % 8, -V % 8]),
                dtype=rng.choice(["f32", "bf16", "f16"]), masked=rng.random() < 0.3)
    if op == "score":
        case["n"] = rng.choice([0, rng.randint(1, 32)])
    else:
        case["entropy"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _logits(case, g):
    """Gaussian background and a head of up to 300 tokens shifted by U(3, 12), as a model's
    logits have it; what is past V in a row is not part of it."""
    B, V = case["B"], case["V"]
    x = torch.randn(B, V + case["pad"], generator=g, device="cuda") * 2.0
    k = min(300, V // 4)
    first = torch.randint(0, V, (B, 1), generator=g, device="cuda")
    ids = (first + 7919 * torch.arange(k, device="cuda")) % V  # distinct: 7919 is prime
    x.scatter_(1, ids, x.gather(1, ids) + 3.0 + 9.0 * _uniform(g, B, k))
    return x.to(DTYPES[case["dtype"]])


def _bitmask(case, g):
    """Grammar masks: most rows allow everything, 30 % allow one token in twenty, 5 % allow a
    handful, and one row (of 16 or more) allows nothing."""
    B, V = case["B"], case["V"]
    W = (V + 31) // 32
    share = torch.ones(B, 1, device="cuda")
    kind = _uniform(g, B, 1)
    share[kind < 0.30] = 0.05
    share[kind > 0.95] = 4.0 / V
    if B >= 16:
        share[B // 2] = 0.0
    bits = torch.zeros(B, W * 32, dtype=torch.bool, device="cuda")
    bits[:, :V] = _uniform(g, B, V) < share
    shifts = torch.arange(32, device="cuda", dtype=torch.int32)
    return (bits.view(B, W, 32).to(torch.int32) << shifts).sum(2, dtype=torch.int32)


def _targets(x, case, g):
    """Mostly tokens drawn from the row's distribution, one in ten any token at all, one in
    thirty none (-1: a padded position)."""
    B, V = case["B"], case["V"]
    noise = -torch.log(-torch.log(_uniform(g, B, V).clamp_(1e-7, 1 - 1e-6)))
    t = (x[:, :V].float() + noise).argmax(1)
    kind = _uniform(g, B)
    t = torch.where(kind < 0.10, torch.randint(0, V, (B,), generator=g, device="cuda"), t)
    return torch.where(kind > 0.967, -torch.ones_like(t), t).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "head":
        N, V, D, dt = case["N"], case["V"], case["D"], DTYPES[case["dtype"]]
        return dict(case=case, hidden=torch.randn(N, D, generator=g, device="cuda").to(dt),
                    weight=(torch.randn(V, D, generator=g, device="cuda") * (2.0 / math.sqrt(D))).to(dt),
                    targets=torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32),
                    temperature=0.7 + 0.6 * _uniform(g, N))
    x = _logits(case, g)
    B, V = case["B"], case["V"]
    s = dict(case=case, logits=x, bitmask=_bitmask(case, g) if case["masked"] else None,
             targets=_targets(x, case, g), temperature=0.7 + 0.6 * _uniform(g, B))
    if case["op"] == "grad":
        # what the forward pass left: (largest legal logit, log of the mass relative to it), entropy
        f = _plain_forward(s)
        s.update(stats=f["stats"], entropy=f["entropy"],
                 grad_logprobs=-(0.5 + _uniform(g, B)) / B,
                 grad_entropy=-0.01 * (0.5 + _uniform(g, B)) / B if case["entropy"] else None)
    return s


# --------------------------------------------------------------------------
# The plain forms: float32, rounded once at the end
# --------------------------------------------------------------------------
def _legal(s, x):
    legal = x > -math.inf
    if s["bitmask"] is not None:
        bit = (s["bitmask"].unsqueeze(2) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        legal &= bit.flatten(1)[:, :x.shape[1]].bool()
    return legal


def _plain_forward(s):
    V = s["case"]["V"]
    x = s["logits"][:, :V].float()
    x = x.masked_fill(~_legal(s, x), -math.inf)
    m = x.amax(1)
    empty = m == -math.inf
    z = (x - m.masked_fill(empty, 0.0).unsqueeze(1)) / s["temperature"].unsqueeze(1)
    e = z.exp()
    S = e.sum(1)
    L = S.log()
    H = L - (e * z.masked_fill(z == -math.inf, 0.0)).sum(1) / S
    nan = torch.full_like(m, math.nan)
    return dict(x=x, z=z, empty=empty, L=L, entropy=torch.where(empty, nan, H),
                stats=torch.stack([torch.where(empty, nan, m), torch.where(empty, nan, L)], 1))


def _plain_score(s):
    f = _plain_forward(s)
    x, z, empty, L = f["x"], f["z"], f["empty"], f["L"]
    B, V = x.shape
    ids = torch.arange(V, device="cuda")
    t = s["targets"].long()
    none = t < 0
    at = t.clamp(min=0).unsqueeze(1)
    xt = x.gather(1, at)
    lp = (z.gather(1, at)[:, 0] - L).masked_fill(none, 0.0).masked_fill(empty, math.nan)
    ahead = (x > xt) | ((x == xt) & (ids < at) & (x > -math.inf))
    rank = ahead.sum(1, dtype=torch.int32).masked_fill(none | empty, -1)
    out = dict(logprobs=lp, entropy=f["entropy"], rank=rank, stats=f["stats"],
               status=torch.where(empty, EMPTY, OK).to(torch.int32))
    n = s["case"]["n"]
    if n:
        b = (x + 0.0).view(torch.int32).long()
        key = torch.where(b < 0, -(b & 0x7FFFFFFF), b) * (1 << 32) + (0xFFFFFFFF - ids)
        best = key.topk(min(n, V), dim=1).values
        top = 0xFFFFFFFF - (best & 0xFFFFFFFF)
        lps = z.gather(1, top) - L.unsqueeze(1)
        out["top_ids"] = top.masked_fill((lps == -math.inf) | empty.unsqueeze(1), -1).to(torch.int32)
        out["top_logprobs"] = lps.masked_fill(empty.unsqueeze(1), math.nan)
    return out


def _plain_grad(s):
    V = s["case"]["V"]
    x = s["logits"][:, :V].float()
    legal = _legal(s, x)
    dead = s["stats"][:, 0].isnan()
    m, L = s["stats"].masked_fill(dead.unsqueeze(1), 0.0).unbind(1)
    T = s["temperature"].unsqueeze(1)
    logp = (x - m.unsqueeze(1)) / T - L.unsqueeze(1)
    p = logp.exp().masked_fill(~legal | dead.unsqueeze(1), 0.0)
    t = s["targets"].long()
    g = s["grad_logprobs"].masked_fill((t < 0) | dead, 0.0).unsqueeze(1)
    at = t.clamp(min=0).unsqueeze(1)
    g = g * legal.gather(1, at)
    d = -g * p
    d.scatter_add_(1, at, g)
    if s["grad_entropy"] is not None:
        H = s["entropy"].masked_fill(dead, 0.0).unsqueeze(1)
        d -= s["grad_entropy"].unsqueeze(1) * p * (logp + H).masked_fill(~legal, 0.0)
    return dict(grad=(d / T).to(s["logits"].dtype))


def _plain_head(s):
    x = s["hidden"].float() @ s["weight"].float().t()
    m = x.amax(1, keepdim=True)
    z = (x - m) / s["temperature"].unsqueeze(1)
    e = z.exp()
    S = e.sum(1)
    L = S.log()
    lp = z.gather(1, s["targets"].long().unsqueeze(1))[:, 0] - L
    return dict(logprobs=lp, entropy=L - (e * z).sum(1) / S, stats=torch.stack([m[:, 0], L], 1),
                status=torch.zeros(x.shape[0], dtype=torch.int32, device="cuda"))


def run(state):
    case = state["case"]
    if not own:
        return {"score": _plain_score, "grad": _plain_grad, "head": _plain_head}[case["op"]](state)
    import top_selection_stats_gb300 as lib
    s = state
    if case["op"] == "score":
        s["out"] = lib.token_logprobs(s["logits"], s["targets"], temperature=s["temperature"], bitmask=s["bitmask"],
                                      n_top=case["n"], V=case["V"], out=s.get("out"))
        return s["out"]
    if case["op"] == "grad":
        s["out"] = lib.token_logprobs_grad(s["logits"], s["targets"], s["stats"], s["grad_logprobs"],
                                           entropy=s["entropy"], grad_entropy=s["grad_entropy"],
                                           temperature=s["temperature"], bitmask=s["bitmask"], V=case["V"],
                                           out=s.get("out"))
        return dict(grad=s["out"][:, :case["V"]])
    s["out"] = lib.head_logprobs(s["hidden"], s["weight"], s["targets"], temperature=s["temperature"],
                                 out=s.get("out"))
    return s["out"]


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "head":
        N, V, D = case["N"], case["V"], case["D"]
        return dict(bytes=2 * D * (N + V) + 28 * N, flops=2 * N * V * D)
    B, V, es = case["B"], case["V"], ESIZE[case["dtype"]]
    row = V * es + (4 * ((V + 31) // 32) if case["masked"] else 0)
    if case["op"] == "score":
        return dict(bytes=B * (row + 8 + 24 + 8 * case["n"]), flops=6 * B * V)
    return dict(bytes=B * (row + V * es + (28 if case["entropy"] else 20)), flops=6 * B * V)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def _row_blocks(s, rows=128):
    """(slice, float64 logits with -inf where illegal, legal) for blocks of rows."""
    B, V = s["case"]["B"], s["case"]["V"]
    for a in range(0, B, rows):
        r = slice(a, min(B, a + rows))
        x = s["logits"][r, :V].double()
        if s["bitmask"] is not None:
            words = s["bitmask"][r].long()[:, torch.arange(V, device="cuda") // 32]
            ok = (words >> (torch.arange(V, device="cuda") % 32)) % 2 == 1
            x = torch.where(ok, x, torch.full_like(x, -math.inf))
        yield r, x, x != -math.inf


def _exact_score(s):
    n, V = s["case"]["n"], s["case"]["V"]
    got = []
    for r, x, legal in _row_blocks(s):
        T, t = s["temperature"][r].double()[:, None], s["targets"][r].long()
        m = x.max(1).values
        logp = torch.log_softmax(x / T, 1)
        p = logp.exp()
        out = dict(entropy=-torch.where(legal, p * logp, 0.0).sum(1))
        out["entropy"][m == -math.inf] = math.nan
        bad = ~legal.any(1)
        lp = logp[torch.arange(len(t), device="cuda"), t.clamp(min=0)]
        out["logprobs"] = torch.where(bad, math.nan, torch.where(t < 0, 0.0, lp))
        stats = torch.stack([m, torch.logsumexp(x / T, 1) - m / T[:, 0]], 1)
        out["stats"] = torch.where(bad[:, None], math.nan, stats)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        place = torch.empty_like(order).scatter_(1, order, torch.arange(V, device="cuda").expand_as(order))
        rank = place.gather(1, t.clamp(min=0)[:, None])[:, 0]
        rank = torch.minimum(rank, legal.sum(1))  # an illegal token comes after every legal one
        out["rank"] = torch.where(bad | (t < 0), -1, rank).to(torch.int32)
        out["status"] = torch.where(bad, EMPTY, OK).to(torch.int32)
        if n:
            top = order[:, :n]
            lps = logp.gather(1, top)
            out["top_ids"] = torch.where(legal.gather(1, top), top, -1).to(torch.int32)
            out["top_logprobs"] = torch.where(bad[:, None], math.nan, lps)
        got.append(out)
    return {k: torch.cat([o[k] for o in got]) for k in got[0]}


def _exact_grad(s):
    got = []
    for r, x, legal in _row_blocks(s):
        T, t = s["temperature"][r].double()[:, None], s["targets"][r].long()
        live = legal.any(1, keepdim=True)
        logp = torch.where(legal, torch.log_softmax(x / T, 1), 0.0)
        p = torch.where(legal, logp.exp(), 0.0)
        hit = (torch.arange(x.shape[1], device="cuda") == t[:, None]) & legal
        glp = s["grad_logprobs"][r].double()[:, None] * hit.any(1, keepdim=True)
        d = glp * (hit.double() - p)
        if s["grad_entropy"] is not None:
            H = -(p * logp).sum(1, keepdim=True)
            d = d - s["grad_entropy"][r].double()[:, None] * p * (logp + H)
        got.append(torch.where(live, d / T, 0.0))
    return dict(grad=torch.cat(got))


def _exact_head(s):
    h, T = s["hidden"].double(), s["temperature"].double()[:, None]
    x = torch.cat([h @ w.double().t() for w in s["weight"].split(8192)], 1)
    logp = [torch.log_softmax(a / b, 1) for a, b in zip(x.split(256), T.split(256))]
    H = torch.cat([-(a.exp() * a).sum(1) for a in logp])
    lp = torch.cat(logp).gather(1, s["targets"].long()[:, None])[:, 0]
    m = x.max(1).values
    L = torch.cat([torch.logsumexp((a - a.max(1, keepdim=True).values) / b, 1)
                   for a, b in zip(x.split(256), T.split(256))])
    return dict(logprobs=lp, entropy=H, stats=torch.stack([m, L], 1),
                status=torch.zeros(len(m), dtype=torch.int32, device="cuda"))


def exact(case, seed):
    return {"score": _exact_score, "grad": _exact_grad, "head": _exact_head}[case["op"]](prepare(case, seed))

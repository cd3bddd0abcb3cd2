"""Processing of logits and distillation: the cases that are measured, their inputs and their
plain forms.

Three operators around a language model's output distribution:

  process  penalties for repeated tokens, biases and grammar masks on logits [B, V] before they
           are sampled from;
  distill  a student's divergence from a teacher's top tokens: forward or reverse divergence
           with one class for all other tokens, or the truncated teacher's cross entropy form;
           optionally with the log probabilities of given tokens;
  distgrad the gradient of that divergence, and of those log probabilities, with respect to
           the student's logits.

The plain forms use elementary torch operations in float32 (the teacher's rest, one minus a
sum near one, in float64); ``exact`` has the definitions in float64.  With ``own`` set, ``run``
calls the library's operators instead.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}
OK, EMPTY = 0, 1
LIMIT = 4096 * 128256  # logits of the largest distill / distgrad case
LEAST = 2.0 ** -24     # the teacher's rest counts as this at least


def listed():
    return [
        # one decode step of one conversation with all penalties and a few biases: latency
        dict(name="process_1x128256_bf16_h1000", op="process", B=1, V=128256, pad=0, dtype="bf16", out="bf16",
             H=1000, NB=20, penalties=True, masked=False, in_place=False),
        # a small batch, float32 logits, ragged histories, the most biases a request carries
        dict(name="process_64x32000_f32_h4096_bias300", op="process", B=64, V=32000, pad=0, dtype="f32", out="f32",
             H=4096, NB=300, penalties=True, masked=False, in_place=False),
        # long contexts: histories longer than the vocabulary, rows that start at any alignment
        dict(name="process_16x50001_bf16_h65536", op="process", B=16, V=50001, pad=0, dtype="bf16", out="bf16",
             H=65536, NB=0, penalties=True, masked=False, in_place=False),
        # grammar-constrained decode in place: masks and a few banned tokens, nothing else
        dict(name="process_512x151936_bf16_mask_inplace", op="process", B=512, V=151936, pad=0, dtype="bf16",
             out="bf16", H=0, NB=16, penalties=False, masked=True, in_place=True),
        # a large decode batch that keeps its raw logits and samples in float32
        dict(name="process_1024x256000_f16_to_f32", op="process", B=1024, V=256000, pad=0, dtype="f16", out="f32",
             H=512, NB=8, penalties=True, masked=False, in_place=False),
        # a small vocabulary of odd size, a teacher that reports 20 logits
        dict(name="distill_37x50001_f32_top20_truncated", op="distill", B=37, V=50001, pad=0, dtype="f32", K=20,
             kind="truncated", targets=False, masked=False),
        # on-policy distillation under grammar masks, one row that allows nothing, with labels
        dict(name="distill_512x151936_bf16_top32_mask_reverse", op="distill", B=512, V=151936, pad=0, dtype="bf16",
             K=32, kind="reverse", targets=True, masked=True),
        # a wide teacher, the largest vocabulary
        dict(name="distill_1024x256000_f16_top128", op="distill", B=1024, V=256000, pad=0, dtype="f16", K=128,
             kind="forward", targets=False, masked=False),
        # a training step's tokens, soft and hard labels together
        dict(name="distill_4096x128256_bf16_top32_targets", op="distill", B=4096, V=128256, pad=0, dtype="bf16",
             K=32, kind="forward", targets=True, masked=False),
        # the small case's gradient: rows that start at any alignment
        dict(name="distgrad_37x50001_f32_top20", op="distgrad", B=37, V=50001, pad=0, dtype="f32", K=20,
             kind="truncated", targets=False, masked=False),
        # masked rows, padded row stride, soft and hard labels
        dict(name="distgrad_256x151936_f16_top32_mask_targets", op="distgrad", B=256, V=151936, pad=64, dtype="f16",
             K=32, kind="reverse", targets=True, masked=True),
        # a training step's gradient, the largest logits
        dict(name="distgrad_4096x128256_bf16_top64", op="distgrad", B=4096, V=128256, pad=0, dtype="bf16", K=64,
             kind="forward", targets=False, masked=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["process", "distill", "distgrad"])
    V = _log_int(rng, 100, 262143)
    B = _log_int(rng, 1, max(1, min(4096, LIMIT // (2 * V))))
    dtype = rng.choice(["f32", "bf16", "f16"])
    case = dict(op=op, B=B, V=V, pad=rng.choice([0, 1, -V % 8, -V % 8]), dtype=dtype, masked=rng.random() < 0.3)
    if op == "process":
        # in place: masks and bans, which a second pass leaves as they are
        in_place = rng.random() < 0.3
        case.update(in_place=in_place, penalties=not in_place, out=dtype if in_place else rng.choice([dtype, "f32"]),
                    H=0 if in_place else _log_int(rng, 1, max(1, min(65536, (1 << 22) // B))),
                    NB=_log_int(rng, 1, 512) if in_place or rng.random() < 0.5 else 0)
    else:
        case.update(K=min(V, _log_int(rng, 1, 256)), kind=rng.choice(["forward", "reverse", "truncated"]),
                    targets=rng.random() < 0.5)
    return case


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _logits(case, g):
    """Gaussian background and a head of up to 300 tokens shifted by U(3, 12), as a model's
    logits have it; what is past V in a row is not part of it.  float32."""
    B, V = case["B"], case["V"]
    x = torch.randn(B, V + case["pad"], generator=g, device="cuda") * 2.0
    k = min(300, V // 4)
    first = torch.randint(0, V, (B, 1), generator=g, device="cuda")
    ids = (first + 7919 * torch.arange(k, device="cuda")) % V  # distinct: 7919 is prime
    x.scatter_(1, ids, x.gather(1, ids) + 3.0 + 9.0 * _uniform(g, B, k))
    return x


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


def _unpack(bitmask, V):
    shifts = torch.arange(32, device="cuda", dtype=torch.int32)
    return ((bitmask.unsqueeze(2) >> shifts) & 1).flatten(1)[:, :V].bool()


def _prepare_process(case, g):
    """Histories as text has them: few tokens often, many once; ragged, with -1 behind each
    row's end.  One request in four has no penalties of its own (1, 0, 0)."""
    B, V, H, NB = case["B"], case["V"], case["H"], case["NB"]
    s = dict(case=case, logits=_logits(case, g).to(DTYPES[case["dtype"]]),
             bitmask=_bitmask(case, g) if case["masked"] else None)
    if H:
        length = (H * (0.25 + 0.75 * _uniform(g, B))).ceil().int().clamp(1, H)
        if B >= 8:
            length[3] = 0
        prompt = (length * _uniform(g, B)).int()
        ids = (V * _uniform(g, B, H) ** 4).long().clamp(max=V - 1) * 7919 % V
        past = torch.arange(H, device="cuda") >= length.unsqueeze(1)
        s.update(history=ids.masked_fill(past, -1).int(), lengths=length, prompt_lengths=prompt)
    if case["penalties"]:
        off = _uniform(g, B) < 0.25
        s.update(repetition=(1.0 + 0.3 * _uniform(g, B)).masked_fill(off, 1.0),
                 presence=_uniform(g, B).masked_fill(off, 0.0),
                 frequency=(0.5 * _uniform(g, B) - 0.1).masked_fill(off, 0.0))
    if NB:
        ids = torch.randint(0, V, (B, NB), generator=g, device="cuda")
        ids[:, NB // 2:] = ids[:, NB // 2:].masked_fill(_uniform(g, B, NB - NB // 2) < 0.2, -1)  # unused slots
        bias = 4.0 * _uniform(g, B, NB) - 2.0
        ban = _uniform(g, B, NB) < (1.1 if case["in_place"] else 0.2)
        s.update(bias_ids=ids.int(), bias=bias.masked_fill(ban, -math.inf))
    return s


def _prepare_distill(case, g):
    """A teacher that saw the same context: the student's logits with noise, its K best legal
    tokens in descending order (unused slots: -1, -inf), as log probabilities, or as logits for
    the truncated kind.  Labels: mostly one of the teacher's, one in ten any token, one in
    thirty none (-1)."""
    B, V, K = case["B"], case["V"], case["K"]
    x = _logits(case, g)
    s = dict(case=case, bitmask=_bitmask(case, g) if case["masked"] else None,
             temperature=0.7 + 0.6 * _uniform(g, B))
    y = x[:, :V] + 0.7 * torch.randn(B, V, generator=g, device="cuda")
    if case["masked"]:
        y.masked_fill_(~_unpack(s["bitmask"], V), -math.inf)
    top, ids = y.topk(K, dim=1)
    if case["kind"] != "truncated":
        y /= s["temperature"].unsqueeze(1)
        top = top / s["temperature"].unsqueeze(1) - torch.logsumexp(y, 1, keepdim=True)
        top = top.nan_to_num(nan=-math.inf)
    none = top == -math.inf
    s.update(logits=x.to(DTYPES[case["dtype"]]), teacher_ids=ids.masked_fill(none, -1).int(), teacher=top.contiguous())
    if case["targets"]:
        kind = _uniform(g, B)
        t = ids.gather(1, torch.randint(0, K, (B, 1), generator=g, device="cuda"))[:, 0]
        t = torch.where(kind < 0.10, torch.randint(0, V, (B,), generator=g, device="cuda"), t)
        s["targets"] = torch.where(kind > 0.967, -torch.ones_like(t), t).int()
    if case["op"] == "distgrad":
        # what the forward pass left, and the loss's own gradient
        f = _plain_distill(s)
        s.update({k: f[k] for k in ("slot_logprobs", "slot_grads", "stats")},
                 grad_loss=(0.5 + _uniform(g, B)) / B)
        if case["targets"]:
            s.update(logprobs=f["logprobs"], grad_logprobs=-0.3 * (0.5 + _uniform(g, B)) / B)
    return s


def prepare(case, seed):
    return (_prepare_process if case["op"] == "process" else _prepare_distill)(case, _generator(seed))


# --------------------------------------------------------------------------
# The plain forms: float32, rounded once at the end
# --------------------------------------------------------------------------
def _plain_process(s):
    case, V = s["case"], s["case"]["V"]
    x = s["logits"][:, :V].float()
    B = x.shape[0]
    v = x
    if case["H"]:
        place = torch.arange(case["H"], device="cuda")
        ids = s["history"].long()
        ids = ids.masked_fill((ids < 0) | (place >= s["lengths"].unsqueeze(1)), V)  # column V: none
        seen = torch.zeros(B, V + 1, dtype=torch.bool, device="cuda").scatter_(1, ids, True)[:, :V]
        made = ids.masked_fill(place < s["prompt_lengths"].unsqueeze(1), V)
        n = torch.zeros(B, V + 1, device="cuda").scatter_add_(1, made, torch.ones_like(made, dtype=torch.float32))[:, :V]
        theta = s["repetition"].unsqueeze(1)
        v = torch.where(seen, torch.where(x > 0, x / theta, x * theta), x)
        v = v - (s["frequency"].unsqueeze(1) * n + s["presence"].unsqueeze(1) * (n > 0))
    if case["NB"]:
        ids = s["bias_ids"].long()
        ids = ids.masked_fill(ids < 0, V)
        v = v + torch.zeros(B, V + 1, device="cuda").scatter_add_(1, ids, s["bias"])[:, :V]
    if case["masked"]:
        v = v.masked_fill(~_unpack(s["bitmask"], V), -math.inf)
    if case["in_place"]:
        s["logits"][:, :V] = v
        v = s["logits"][:, :V]
    return dict(logits=v.to(DTYPES[case["out"]]), status=torch.zeros(B, dtype=torch.int32, device="cuda"))


def _legal_logits(s):
    x = s["logits"][:, :s["case"]["V"]].float()
    return x.masked_fill(~_unpack(s["bitmask"], s["case"]["V"]), -math.inf) if s["case"]["masked"] else x


def _members(s):
    """(ids with V for unused slots, used, [B, V]: whether a token has a slot)."""
    V = s["case"]["V"]
    used = s["teacher_ids"] >= 0
    ids = s["teacher_ids"].long().masked_fill(~used, V)
    has = torch.zeros(ids.shape[0], V + 1, dtype=torch.bool, device="cuda").scatter_(1, ids, True)
    return ids, used, has[:, :V]


def _plain_distill(s):
    kind = s["case"]["kind"]
    x = _legal_logits(s)
    T = s["temperature"]
    ids, used, has = _members(s)
    xk = x.gather(1, ids.clamp(max=x.shape[1] - 1)).masked_fill(~used, -math.inf)
    xr = x.masked_fill(has, -math.inf)
    mr = xr.amax(1)
    m = torch.maximum(mr, xk.amax(1))
    empty, bare = m == -math.inf, mr == -math.inf  # no legal token; none outside the slots
    m0, mr0 = m.masked_fill(empty, 0.0), mr.masked_fill(bare, 0.0)
    Lr = ((xr - mr0.unsqueeze(1)) / T.unsqueeze(1)).exp().sum(1).log()
    zk = (xk - m0.unsqueeze(1)) / T.unsqueeze(1)
    L = (zk.exp().sum(1) + (Lr + (mr0 - m0) / T).exp()).log()
    a = zk - L.unsqueeze(1)  # log probabilities of the slots
    p = a.exp()
    log_s = (mr0 - m0) / T + Lr - L
    sm = log_s.exp()
    v = s["teacher"].masked_fill(~used, -math.inf)
    if kind == "truncated":
        v = v / T.unsqueeze(1)
        mv = v.amax(1, keepdim=True).nan_to_num(neginf=0.0)
        e = (v - mv).exp()
        lq = v - mv - e.sum(1, keepdim=True).log()
        q = lq.exp().masked_fill(v == -math.inf, 0.0)
        r = torch.zeros_like(T)
    else:
        lq, q = v, v.exp()
        r = (1.0 - v.double().exp().sum(1)).clamp(min=LEAST).float().masked_fill(bare, 0.0)
    Q = q.sum(1)
    live = ~bare & (r > 0)
    if kind == "reverse":
        u = (a - lq).masked_fill(p == 0.0, 0.0)
        ur = (log_s - r.log()).masked_fill(~live, 0.0)
        loss = (p * u).sum(1) + sm * ur
        A = sm * (ur - loss)
        G = p * (u - loss.unsqueeze(1))
    else:
        loss = (q * (lq - a)).masked_fill(q == 0.0, 0.0).sum(1)
        loss = loss + (r * (r.log() - log_s)).masked_fill(~live, 0.0)
        A = sm * (Q + r) - r
        G = p * (Q + r).unsqueeze(1) - q
    nan = torch.full_like(T, math.nan)
    dead = empty.unsqueeze(1)
    out = dict(loss=torch.where(empty, nan, loss), slot_logprobs=a.masked_fill(dead, math.nan),
               slot_grads=G.masked_fill(~used, 0.0).masked_fill(dead, math.nan),
               stats=torch.stack([mr, Lr, A, sm], 1).masked_fill(dead, math.nan),
               status=torch.where(empty, EMPTY, OK).to(torch.int32))
    if s["case"]["targets"]:
        t = s["targets"].long()
        xt = x.gather(1, t.clamp(min=0).unsqueeze(1))[:, 0]
        out["logprobs"] = ((xt - m0) / T - L).masked_fill(t < 0, 0.0).masked_fill(empty, math.nan)
    return out


def _plain_distgrad(s):
    x = _legal_logits(s)
    T = s["temperature"].unsqueeze(1)
    ids, used, has = _members(s)
    dead = s["stats"][:, 2].isnan().unsqueeze(1)
    mr, Lr, A, sm = s["stats"].split(1, 1)
    g = s["grad_loss"].unsqueeze(1)
    gl = torch.zeros_like(g)
    if s["case"]["targets"]:
        t = s["targets"].long()
        gl = s["grad_logprobs"].masked_fill((t < 0) | ~(s["logprobs"] > -math.inf), 0.0).unsqueeze(1)
    rho = ((x - mr) / T - Lr).exp().masked_fill(has | (x == -math.inf), 0.0)
    d = rho * ((g * A - gl * sm) / T)
    dk = (g * s["slot_grads"] - gl * s["slot_logprobs"].exp()) / T
    d = torch.cat([d, torch.zeros_like(g)], 1).scatter_(1, ids, dk)[:, :x.shape[1]]
    if s["case"]["targets"]:
        d.scatter_add_(1, t.clamp(min=0).unsqueeze(1), gl / T)
    return dict(grad=d.masked_fill(dead, 0.0).to(s["logits"].dtype))


def run(state):
    case, s = state["case"], state
    if not own:
        return {"process": _plain_process, "distill": _plain_distill, "distgrad": _plain_distgrad}[case["op"]](s)
    import top_selection_stats_gb300 as lib
    if case["op"] == "process":
        s["out"] = lib.process_logits(s["logits"], history=s.get("history"), lengths=s.get("lengths"),
                                      prompt_lengths=s.get("prompt_lengths"), repetition=s.get("repetition"),
                                      presence=s.get("presence"), frequency=s.get("frequency"),
                                      bias_ids=s.get("bias_ids"), bias=s.get("bias"), bitmask=s["bitmask"],
                                      V=case["V"], dtype=DTYPES[case["out"]], in_place=case["in_place"],
                                      out=s.get("out"))
        return dict(logits=s["out"]["logits"][:, :case["V"]], status=s["out"]["status"])
    if case["op"] == "distill":
        s["out"] = lib.distill_loss(s["logits"], s["teacher_ids"], s["teacher"], kind=case["kind"],
                                    targets=s.get("targets"), temperature=s["temperature"], bitmask=s["bitmask"],
                                    V=case["V"], out=s.get("out"))
        return s["out"]
    s["out"] = lib.distill_loss_grad(s["logits"], s["teacher_ids"], s["slot_logprobs"], s["slot_grads"], s["stats"],
                                     grad_loss=s["grad_loss"], targets=s.get("targets"), logprobs=s.get("logprobs"),
                                     grad_logprobs=s.get("grad_logprobs"), temperature=s["temperature"],
                                     bitmask=s["bitmask"], V=case["V"], out=s.get("out"))
    return dict(grad=s["out"][:, :case["V"]])


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    B, V, es = case["B"], case["V"], ESIZE[case["dtype"]]
    mask = 4 * ((V + 31) // 32) if case["masked"] else 0
    if case["op"] == "process":
        side = 4 * case["H"] + 8 * case["NB"] + (8 if case["H"] else 0) + (12 if case["penalties"] else 0) + 4 + mask
        if case["in_place"]:  # what is touched: a third of the rows lose nearly all their tokens
            return dict(bytes=int(B * (side + (0.335 * V if case["masked"] else 0) * es + 2 * es * case["NB"])),
                        flops=B * case["NB"])
        return dict(bytes=B * (side + V * (es + ESIZE[case["out"]])), flops=B * (4 * case["H"] + case["NB"]))
    side = B * (8 * case["K"] + 4 + mask + (8 if case["targets"] else 0))
    if case["op"] == "distill":
        return dict(bytes=side + B * (V * es + 8 * case["K"] + 24), flops=4 * B * V)
    return dict(bytes=side + B * (2 * V * es + 4 * case["K"] + 24), flops=5 * B * V)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_process(s):
    case, V = s["case"], s["case"]["V"]
    v = s["logits"][:, :V].double()
    if case["H"]:
        lengths, prompts = s["lengths"].tolist(), s["prompt_lengths"].tolist()
        for r in range(case["B"]):
            seen, n = s["history"][r, :lengths[r]].long(), s["history"][r, prompts[r]:lengths[r]].long()
            theta, x = s["repetition"][r].double(), v[r]
            which = torch.bincount(seen, minlength=V) > 0
            n = torch.bincount(n, minlength=V).double()
            y = torch.where(which & (x > 0), x / theta, torch.where(which, x * theta, x))
            v[r] = y - s["frequency"][r].double() * n - torch.where(n > 0, s["presence"][r].double(), 0.0)
    if case["NB"]:
        row = torch.arange(case["B"], device="cuda").unsqueeze(1).expand_as(s["bias_ids"])
        used = s["bias_ids"] >= 0
        v.index_put_((row[used], s["bias_ids"][used].long()), s["bias"][used].double(), accumulate=True)
    if case["masked"]:
        j = torch.arange(V, device="cuda")
        v[(s["bitmask"].long()[:, j // 32] >> (j % 32)) % 2 == 0] = -math.inf
    return dict(logits=v, status=torch.zeros(case["B"], dtype=torch.int32, device="cuda"))


def _exact_rows(s, r):
    """The definitions for a block of rows, the divergence as a function of the logits."""
    case = s["case"]
    V, kind = case["V"], case["kind"]
    x = s["logits"][r, :V].double()
    if case["masked"]:
        j = torch.arange(V, device="cuda")
        x[(s["bitmask"][r].long()[:, j // 32] >> (j % 32)) % 2 == 0] = -math.inf
    legal = x > -math.inf
    ok = legal.any(1)
    T = s["temperature"][r].double().unsqueeze(1)
    x = torch.where(ok.unsqueeze(1), x, 0.0).requires_grad_()
    ids = s["teacher_ids"][r].long()
    used = ids >= 0
    logp = torch.log_softmax(x / T, 1)
    a = torch.where(used, logp.gather(1, ids.clamp(min=0)), -math.inf)
    outside = torch.ones_like(legal).index_put_((used.nonzero()[:, 0], ids[used]), torch.tensor(False, device="cuda"))
    outside &= legal | ~ok.unsqueeze(1)
    sm = torch.where(outside, logp, -math.inf).exp().sum(1)
    log_s = torch.where(sm > 0, sm, 1.0).log()
    v = torch.where(used, s["teacher"][r].double(), -math.inf)
    if kind == "truncated":
        lq = torch.where(used.any(1, keepdim=True), torch.log_softmax(v / T, 1), -math.inf)
        rest = torch.zeros_like(sm)
    else:
        lq = v
        rest = torch.where(outside.any(1), (1.0 - v.exp().sum(1)).clamp(min=LEAST), 0.0)
    q = lq.exp()
    log_r = torch.where(rest > 0, rest, 1.0).log()
    fin = (q > 0) & (a > -math.inf)
    af, lf = torch.where(fin, a, 0.0), torch.where(fin, lq, 0.0)
    if kind == "reverse":
        ur = torch.where(rest > 0, log_s - log_r, 0.0)
        loss = (torch.where(fin, a, -math.inf).exp() * (af - lf)).sum(1) + sm * ur
        A = sm * (ur - loss)
    else:
        loss = (q * (lf - af)).sum(1) + rest * (log_r - log_s)
        A = sm * (q.sum(1) + rest) - rest
    return x, ok, T, a, used, outside, sm, loss, A, logp, q, lq, rest


def _exact_distill(s, rows=128):
    got = []
    for b in range(0, s["case"]["B"], rows):
        r = slice(b, min(s["case"]["B"], b + rows))
        x, ok, T, a, used, outside, sm, loss, A, logp, q, lq, rest = _exact_rows(s, r)
        with torch.no_grad():
            # the divergence's derivative by a slot's scaled logit
            p = a.exp()
            if s["case"]["kind"] == "reverse":
                G = torch.where(p > 0, p * (a - lq - loss.unsqueeze(1)), 0.0)
            else:
                G = p * (q.sum(1) + rest).unsqueeze(1) - q
            xr = torch.where(outside, x, -math.inf)
            mr = xr.max(1).values
            Lr = torch.logsumexp((xr - torch.where(mr == -math.inf, 0.0, mr).unsqueeze(1)) / T, 1)
            dead = ~ok
            out = dict(loss=torch.where(dead, math.nan, loss), slot_logprobs=torch.where(dead[:, None], math.nan, a),
                       slot_grads=torch.where(dead[:, None], math.nan, torch.where(used, G, 0.0)),
                       stats=torch.where(dead[:, None], math.nan, torch.stack([mr, Lr, A, sm], 1)),
                       status=torch.where(dead, EMPTY, OK).to(torch.int32))
            if s["case"]["targets"]:
                t = s["targets"][r].long()
                lp = logp.gather(1, t.clamp(min=0)[:, None])[:, 0]
                out["logprobs"] = torch.where(dead, math.nan, torch.where(t < 0, 0.0, lp))
            got.append({k: w.detach() for k, w in out.items()})
    return {k: torch.cat([o[k] for o in got]) for k in got[0]}


def _exact_distgrad(s, rows=128):
    got = []
    for b in range(0, s["case"]["B"], rows):
        r = slice(b, min(s["case"]["B"], b + rows))
        x, ok, T, a, used, outside, sm, loss, A, logp, q, lq, rest = _exact_rows(s, r)
        total = (loss * s["grad_loss"][r].double())[ok].sum()
        if s["case"]["targets"]:
            t = s["targets"][r].long()
            lp = logp.gather(1, t.clamp(min=0)[:, None])[:, 0]
            total = total + (lp * s["grad_logprobs"][r].double())[ok & (t >= 0) & (lp > -math.inf)].sum()
        d, = torch.autograd.grad(total, x)
        got.append(torch.where(ok.unsqueeze(1), d, 0.0))
    return dict(grad=torch.cat(got))


def exact(case, seed):
    s = prepare(case, seed)
    return {"process": _exact_process, "distill": _exact_distill, "distgrad": _exact_distgrad}[case["op"]](s)

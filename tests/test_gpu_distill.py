"""Distillation from a teacher's top tokens on the GPU (smp_distill_loss,
smp_distill_loss_grad) against the float64 oracle.

Tolerances.  u = 2^-24.  As for the scoring calls, the logarithm of a mass of V weights is off
by at most u (4 zbar + 4 L + V / 256 + 80), zbar the mean of |z| under it: eL for all legal
tokens, eR for those outside the slots.  Then
  log p_k, log s     (x - m) / T twice rounded, two masses:   e_k = eL + eR + 4u |z| + 8u
  q_k                an exponential of at most 2 units, in the truncated kind of a difference
                     with a logarithm of K weights:           e_q = 8u + 8u max|log q| (relative)
  sums over slots    8 per lane and 5 additions of lanes:     16u relative to their terms
  r                  from a binary64 sum, rounded once:       2u r
The loss is a sum of weight times difference, its error the weights' times the differences
plus the differences' own; slot gradients and A are differences of two such products.  All
factors below are at least those counts, doubled."""
import numpy as np
import pytest
import torch

import top_selection_stats_gb300 as lib
from oracle import distill as D
from oracle import scoring as S
from top_selection_stats_gb300 import workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = workloads.TORCH_DTYPE
OUT_EPS = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # relative, one rounding
OUT_TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}
KINDS = ["forward", "reverse", "truncated"]


def make(B, V, K, dtype, seed, kind="forward", pad=0, shift=0, masked=False, temps=None, neg_inf=0.0, unused=0.1,
         near=0.7):
    """Logits whose first value lies ``shift`` elements past an aligned address; a teacher with the
    logits plus noise, its K best legal tokens in random order, some slots unused."""
    case = workloads.random_case(seed, B, V, dtype=dtype, mask_frac=0.6 if masked else 0.0, neg_inf_frac=neg_inf)
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    ld = V + pad
    buf = torch.full((shift + B * ld,), float("nan"), dtype=DT[dtype], device="cuda")
    x = buf[shift:].view(B, ld)
    x[:, :V] = case["logits"].cuda()
    T = (rng.uniform(0.5, 1.5, B) if temps is None else np.resize(temps, B)).astype(np.float32)
    y = case["logits"].double().numpy() + near * rng.standard_normal((B, V))
    bm = None if case["bitmask"] is None else case["bitmask"].numpy().view(np.uint32)
    if bm is not None:
        y[~S.unpack(bm, V)] = -np.inf
    ids, q = np.full((B, K), -1), np.full((B, K), -np.inf)
    Tq = np.where(np.isfinite(T) & (T > 0), T, 1.0)
    for r in range(B):
        k = min(K, V)
        top = rng.permutation(np.argsort(-y[r], kind="stable")[:k])
        top = top[y[r, top] > -np.inf]
        with np.errstate(over="ignore", invalid="ignore"):
            lq = y[r] if kind == "truncated" else y[r] / Tq[r] - np.logaddexp.reduce(y[r] / Tq[r])
        keep = rng.random(len(top)) >= unused
        ids[r, :len(top)] = np.where(keep, top, -1)
        q[r, :len(top)] = lq[top]
    t = rng.integers(0, V, B).astype(np.int32)
    t[::2] = np.where(ids[::2, 0] >= 0, ids[::2, 0], t[::2])
    t[5::7] = -1
    q = np.maximum(q, np.where(q > -np.inf, -3e38, q))  # finite stays finite in float32
    return dict(x=x, V=V, K=K, kind=kind, targets=torch.from_numpy(t).cuda(), temperature=torch.from_numpy(T).cuda(),
                bitmask=None if bm is None else case["bitmask"].cuda(),
                ids=torch.from_numpy(ids.astype(np.int32)).cuda(),
                teacher=torch.from_numpy(q.astype(np.float32)).cuda())


def run(c, **more):
    out = lib.distill_loss(c["x"], c["ids"], c["teacher"], kind=c["kind"], targets=c["targets"],
                           temperature=c["temperature"], bitmask=c["bitmask"], V=c["V"], **more)
    torch.cuda.synchronize()
    return out


def host(c):
    B, V = c["x"].shape[0], c["V"]
    x = c["x"][:, :V].double().cpu().numpy()
    legal = np.ones((B, V), bool) if c["bitmask"] is None else S.unpack(c["bitmask"].cpu().numpy().view(np.uint32), V)
    t = np.full(B, -1) if c["targets"] is None else c["targets"].cpu().numpy()
    T = np.ones(B) if c["temperature"] is None else c["temperature"].double().cpu().numpy()
    return x, legal, c["ids"].cpu().numpy(), c["teacher"].double().cpu().numpy(), t, T


def reference(c):
    x, legal, ids, q, t, T = host(c)
    return [D.distill_row(x[r], ids[r], q[r], c["kind"], int(t[r]), float(T[r]), legal[r]) for r in range(len(x))]


def errors(o, V, T, kind):
    """Bounds for a row's results, from the module's docstring."""
    with np.errstate(invalid="ignore", over="ignore"):
        eL = U * (4 * o["zbar"] + 4 * o["L"] + V / 256 + 80)
        # the bound holds for any mass outside the slots, one that binary64 shows as s = 0 among
        # them (its logarithm is relative to its own largest value); there is none in a bare row
        eR = 0.0 if not o["outside"].any() else U * (4 * o["zbar_r"] + 4 * abs(o["stats"][1]) + V / 256 + 80)
        live = o["slot_logprobs"] > -np.inf
        ek = np.where(live, eL + eR + 8 * U + 4 * U * np.where(live, np.abs(o["slot_logprobs"]) + o["L"], 0.0), 0.0)
        es = eL + eR + 8 * U + (4 * U * (abs(o["log_s"]) + o["L"] + abs(o["stats"][1])) if o["stats"][3] > 0 else 0.0)
        lq = np.where(o["q"] > 0, np.abs(np.where(o["q"] > 0, o["lq"], 0.0)), 0.0)
        eq = 8 * U + 8 * U * lq.max(initial=0.0)
        p, q, s, r = o["p"], o["q"], o["stats"][3], o["r"]
        du = np.where((p > 0) & (q > 0), np.abs(np.where((p > 0) & (q > 0), o["u"], 0.0)), 0.0)
        dr = abs(o["ur"]) if s > 0 and r > 0 else 0.0
        er = es + (8 * U * (1 + abs(o["log_r"]) + abs(o["log_s"])) if s > 0 and r > 0 else 0.0)
        Q = q.sum()
        if kind == "reverse":
            loss = (p * (du * (ek + 40 * U) + ek + eq)).sum() + s * (dr * (es + 40 * U) + er)
            G = p * ((ek + 8 * U) * (du + abs(o["loss"])) + ek + eq + loss)
            A = s * ((es + 8 * U) * (dr + abs(o["loss"])) + er + loss)
        else:
            loss = (q * (du * (eq + 40 * U) + ek + eq)).sum() + r * (dr * 40 * U + er)
            G = p * (Q + r) * (ek + 8 * U) + q * (eq + 8 * U)
            A = s * (Q + r) * (es + 8 * U) + 4 * U * r
    if not np.isfinite(o["loss"]):  # no gradient: G and A are 0, with nothing computed
        G, A = 0 * p, 0.0
    return dict(loss=loss, slot_logprobs=ek, slot_grads=G, A=A, s=s * (es + 8 * U), Lr=eR, logprob=eL + eR + 8 * U)


def close(got, want, tol, what):
    """Within tol; what is past float32 is an infinity."""
    got, want = np.atleast_1d(got).astype(np.float64), np.atleast_1d(want)
    tol = np.broadcast_to(tol, want.shape)
    with np.errstate(over="ignore"):
        past = ~np.isfinite(want.astype(np.float32))
    assert np.array_equal(got[past], want.astype(np.float32)[past].astype(np.float64)), (what, got[past], want[past])
    err = np.abs(got[~past] - want[~past])
    assert np.all(err <= tol[~past]), (what, err.max(), tol[~past][err.argmax()], want[~past][err.argmax()])


def check_forward(c):
    got = {k: v.cpu().numpy() for k, v in run(c).items()}
    ref = reference(c)
    x, _, ids, _, t, T = host(c)
    for r, o in enumerate(ref):
        assert got["status"][r] == o["status"], (r, got["status"][r], o["status"])
        if o["status"] != D.OK:
            for k in ("loss", "slot_logprobs", "slot_grads", "stats") + (("logprobs",) if c["targets"] is not None else ()):
                assert np.all(np.isnan(got[k][r])), (r, k)
            continue
        e = errors(o, c["V"], T[r], c["kind"])
        close(got["slot_logprobs"][r], o["slot_logprobs"], e["slot_logprobs"], (r, "slot_logprobs"))
        close(got["loss"][r], o["loss"], e["loss"], (r, "loss"))
        close(got["slot_grads"][r], o["slot_grads"], e["slot_grads"] + 2.0 ** -126, (r, "slot_grads"))
        m, Lr, A, s = got["stats"][r]
        assert m == o["stats"][0], r
        if m > -np.inf:
            close(Lr, o["stats"][1], e["Lr"], (r, "Lr"))
            close(A, o["stats"][2], e["A"] + 2.0 ** -126, (r, "A"))
        close(s, o["stats"][3], e["s"] + 2.0 ** -126, (r, "s"))
        if c["targets"] is not None:
            close(got["logprobs"][r], o["logprob"], e["logprob"] + 4 * U * (abs(o["logprob"]) + o["L"])
                  if o["logprob"] > -np.inf else 0.0, (r, "logprob"))
    return got, ref


def check_grad(c, dtype, in_place=False, hard=True):
    """The gradient from the forward call's own outputs: their errors, those of rho (a weight of
    the mass outside) and of a handful of products, and the rounding to dtype."""
    B, V = c["x"].shape[0], c["V"]
    f = run(c)
    ref = reference(c)
    x, legal, ids, _, t, T = host(c)
    rng = np.random.Generator(np.random.PCG64(B * 31 + V))
    g = torch.from_numpy(rng.standard_normal(B).astype(np.float32)).cuda()
    gl = torch.from_numpy(rng.standard_normal(B).astype(np.float32)).cuda() if hard else None
    after = c["x"][:, V:].clone()
    d = lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], grad_loss=g,
                              targets=c["targets"] if hard else None, logprobs=f["logprobs"] if hard else None,
                              grad_logprobs=gl, temperature=c["temperature"], bitmask=c["bitmask"], V=V,
                              out=c["x"] if in_place else None)
    torch.cuda.synchronize()
    if in_place:
        assert torch.equal(d[:, V:].contiguous().view(torch.uint8), after.contiguous().view(torch.uint8))
    else:
        assert not d[:, V:].any()
    d = d[:, :V].double().cpu().numpy()
    g = g.double().cpu().numpy()
    gl = np.zeros(B) if gl is None else gl.double().cpu().numpy()
    for r, o in enumerate(ref):
        want = D.grad_row(o, ids[r], int(t[r]), T[r], g[r], gl[r])
        if want is None:
            assert not d[r].any(), r
            continue
        ok = o["log_p"] > -np.inf
        assert not d[r][~ok].any(), r
        e = errors(o, V, T[r], c["kind"])
        err = np.zeros(V)
        out = o["outside"]
        if out.any():
            mr, Lr, A, s = o["stats"]
            zr = np.where(out, (mr - np.where(out, x[r], mr)) / T[r], 0.0)
            rho = np.where(out, np.exp(-zr - Lr), 0.0)
            rel = e["Lr"] + U * (8 * zr + 4 * Lr + 120)  # the exponent: 24 more than log2
            err += rho * (abs(g[r]) * (e["A"] + rel * abs(A)) + abs(gl[r]) * (e["s"] + rel * s))
        used = ids[r] >= 0
        np.add.at(err, ids[r][used], (abs(g[r]) * (e["slot_grads"] + 8 * U * np.abs(o["slot_grads"]))
                                      + abs(gl[r]) * o["p"] * (e["slot_logprobs"] + 8 * U))[used])
        if t[r] >= 0:
            err[t[r]] += 8 * U * abs(gl[r])
        w, er = want[ok], 2 * err[ok] / T[r]
        tol = er + (np.abs(w) + er) * (OUT_EPS[dtype] + 8 * U) + 2 * OUT_TINY[dtype]
        close(d[r][ok], w, tol, r)


SIZES = [1, 2, 7, 8, 31, 33, 255, 1000, 4097, 32000, 70001, 128256]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_forward(kind, V, dtype):
    for K, pad, shift, masked in ((1, 0, 0, False), (20, 3, 1, True), (33, -V % 8, 0, True), (256, 1, 3, False)):
        check_forward(make(7, V, K, dtype, V + K, kind, pad=pad, shift=shift, masked=masked,
                           neg_inf=0.05 if masked else 0.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_gradient(kind, V, dtype):
    for K, pad, shift, masked, hard in ((1, 0, 0, False, True), (20, 3, 1, True, True), (64, -V % 8, 0, True, False),
                                        (256, 1, 3, False, True)):
        c = make(5, V, K, dtype, V + K, kind, pad=pad, shift=shift, masked=masked, neg_inf=0.05 if masked else 0.0)
        check_grad(c, dtype, hard=hard)
        check_grad(c, dtype, in_place=True, hard=hard)


@pytest.mark.parametrize("B", [1, 2, 150, 700])
def test_batches(B):
    c = make(B, 5003, 20, "bf16", B)
    check_forward(c)
    check_grad(c, "bf16")


@pytest.mark.parametrize("kind", KINDS)
def test_every_token_has_a_slot(kind):
    """No term outside, in whole rows and under masks that leave less than K tokens."""
    for V, K, masked in ((5, 5, False), (9, 20, False), (200, 200, False), (300, 256, True)):
        c = make(9, V, K, "f32", V, kind, masked=masked, unused=0.0)
        got, ref = check_forward(c)
        if not masked:
            assert np.all(got["stats"][:, 0] == -np.inf)
        check_grad(c, "f32")


@pytest.mark.parametrize("kind", KINDS)
def test_slots_at_the_ends(kind):
    """Members in the first and last values of rows at every alignment, in every CTA's part."""
    for dtype, V in (("bf16", 40003), ("f32", 20001), ("bf16", 61), ("f16", 16)):
        for shift in range(8):
            c = make(3, V, 16, dtype, shift, kind, shift=shift, pad=1)
            ends = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, V - 8, V - 7, V - 6, V - 5, V - 4, V - 3, V - 2, V - 1])
            c["ids"][:] = ends.int()
            c["teacher"][:] = torch.linspace(-4, -2.9, 16)
            c["targets"] = torch.tensor([0, V - 1, V // 2], dtype=torch.int32, device="cuda")
            check_forward(c)
            check_grad(c, dtype)


def test_rest_next_to_one_and_to_nothing():
    """A student with all but 1e-5 to 1e-30 of its mass on the slots, and one with that little
    there: the mass outside keeps its bits, and gradients stay bounded."""
    for kind in KINDS:
        c = make(8, 4001, 10, "f32", 5, kind, temps=[1.0], unused=0.0)
        for r, up in enumerate((0.0, 10.0, 20.0, 40.0, 60.0, 80.0, -20.0, -60.0)):
            c["x"][r, c["ids"][r].long()] += up
        got, ref = check_forward(c)
        assert got["stats"][5, 3] < 1e-25 and got["stats"][5, 3] > 0
        check_grad(c, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [77, 20008])
@pytest.mark.parametrize("kind", KINDS)
def test_extreme_values(kind, V, dtype):
    """Rows at the type's lowest value, beside -inf; far from zero; a huge range; NaN and
    infinities in legal slots, in masked ones, and in the teacher's."""
    low = torch.finfo(DT[dtype]).min
    inf, nan = float("inf"), float("nan")
    c = make(20, V, 6, dtype, V, kind, temps=[1.0], unused=0.0)
    x, ids = c["x"], c["ids"].long()
    x[0] = low
    x[1] = low
    x[1, ::2] = -inf
    x[2] = -inf
    x[2, V // 3] = low
    x[3] = -inf
    x[4] += 900.0
    x[5, 1] = low
    x[6, V - 1] = nan
    x[7, 0] = inf
    x[8, ids[8, 2]] = nan
    x[9, 3] = nan
    x[10, V - 2] = inf
    x[11] = low
    x[11, V // 2] = 0.0
    x[12, ids[12, 0]] = -inf
    x[13, ids[13]] = -inf
    c["teacher"][14, 1] = nan
    c["teacher"][15, 2] = inf
    c["teacher"][16, 0] = -inf
    c["teacher"][17] = -inf
    allowed = np.ones((20, V), bool)
    allowed[9, 3] = allowed[10, V - 2] = False
    allowed[18] = False
    allowed[19] = False
    allowed[19, c["ids"][19, 0].item()] = True
    c["bitmask"] = torch.from_numpy(workloads.mask_from_allowed(allowed).view(np.int32)).cuda()
    got, _ = check_forward(c)
    st = list(got["status"])
    assert st[3] == st[18] == 1 and st[6:9] == [2, 2, 2] and st[14:16] == [2, 2]
    assert [st[r] for r in (0, 1, 2, 4, 5, 9, 10, 11, 12, 13, 16, 17, 19)] == [0] * 13
    assert got["loss"][12] == np.inf or kind == "reverse"
    check_grad(c, dtype)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_slots(kind):
    """Ids out of range and repeated, far ones among them, and probabilities above one."""
    c = make(12, 600, 40, "bf16", 4, kind, unused=0.3)
    ids = c["ids"]
    ids[0, 0] = 600
    ids[1, 39] = -2
    ids[2, 7] = 1 << 30
    ids[3, 8] = -(1 << 31)
    ids[4, 0] = ids[4, 39] = 17
    ids[5, 38] = ids[5, 39] = 599
    ids[6, :] = -1
    ids[7, 0], ids[7, 32] = 3, 3
    c["teacher"][8] = -3.0
    ids[8] = torch.arange(40)
    got, _ = check_forward(c)
    st = list(got["status"])
    assert st[:6] == [3] * 6 and st[6] == 0 and st[7] == 3 and st[8] == (0 if kind == "truncated" else 3)
    assert abs(got["loss"][6]) < 1e-6 and not got["slot_grads"][6].any()
    check_grad(c, "bf16")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_temperatures(kind, dtype):
    c = make(11, 3001, 12, dtype, 3, kind, temps=[1e-3, 0.05, 1.0, 20.0, 1e4, 1e30, 0.0, -1.0, float("nan"), float("inf"), 1.0])
    got, _ = check_forward(c)
    assert list(got["status"]) == [0] * 6 + [3] * 4 + [0]
    check_grad(c, dtype)
    c["temperature"] = None
    check_forward(c)
    check_grad(c, dtype)


def test_targets_outside_and_illegal():
    c = make(8, 500, 5, "bf16", 4, masked=True)
    c["targets"] = torch.tensor([500, -2, 1 << 30, -(1 << 31), -1, 0, 1, 499], dtype=torch.int32, device="cuda")
    got, _ = check_forward(c)
    assert list(got["status"][:4]) == [3] * 4
    check_grad(c, "bf16")


def test_tiny_and_huge_gradients():
    """Incoming gradients from 1e-42 to 1e37 and temperatures down to 1e-42: results are the
    formula's, infinite only where it is past the type."""
    temps = [1.0, 1.0, 1e-3, 1e-20, 1e-42, 1e3, 1e38, 1.0]
    gs = np.array([1e-42, 1e37, 1e37, 1e-30, 1e-38, 1e-36, 1e37, 0.0], np.float32)
    c = make(8, 900, 6, "f32", 9, temps=temps)
    c["x"][:, :900] = torch.randint(0, 2, (8, 900), device="cuda").float()  # differences survive small T as 0 or -inf
    c["teacher"][:] = -2.5
    f = run(c)
    d = lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"],
                              grad_loss=torch.from_numpy(gs).cuda(), temperature=c["temperature"], V=900)
    torch.cuda.synchronize()
    d = d.double().cpu().numpy()
    ids = c["ids"].cpu().numpy()
    stats, G = f["stats"].double().cpu().numpy(), f["slot_grads"].double().cpu().numpy()
    x, _, _, _, _, T = host(c)
    assert not np.isnan(d).any() and not d[7].any()
    for r in range(7):
        if f["status"][r] != 0 or not np.isfinite(float(f["loss"][r])):
            assert not d[r].any()
            continue
        m, Lr, A, s = stats[r]
        with np.errstate(over="ignore", under="ignore"):
            want = np.exp((x[r] - m) / T[r] - Lr) * A * gs[r].astype(np.float64) / T[r]
            used = ids[r] >= 0
            want[ids[r][used]] = G[r][used] * gs[r].astype(np.float64) / T[r]
            w32 = want.astype(np.float32).astype(np.float64)
        inf = np.isinf(w32)
        assert np.array_equal(d[r][inf], w32[inf]), r
        assert np.all(np.abs(d[r][~inf] - want[~inf]) <= 200 * U * np.abs(want[~inf]) + 2.0 ** -126), r


def test_grad_parts_may_be_missing():
    c = make(6, 700, 9, "f32", 8)
    f = run(c)
    a = (c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"])
    more = dict(temperature=c["temperature"], V=700)
    assert not lib.distill_loss_grad(*a, **more).any()
    g = torch.ones(6, device="cuda")
    soft = lib.distill_loss_grad(*a, grad_loss=g, **more)
    both = lib.distill_loss_grad(*a, grad_loss=g, targets=c["targets"], logprobs=f["logprobs"], grad_logprobs=0 * g, **more)
    assert torch.equal(soft, both) and soft.any()
    # the hard part alone is token_logprobs_grad's
    hard = lib.distill_loss_grad(*a, targets=c["targets"], logprobs=f["logprobs"], grad_logprobs=g, **more)
    t = lib.token_logprobs(c["x"], c["targets"], temperature=c["temperature"], V=700)
    want = lib.token_logprobs_grad(c["x"], c["targets"], t["stats"], g, **more)
    assert torch.allclose(hard, want, rtol=1e-5, atol=1e-7)
    # without targets the forward call has no log probabilities
    assert "logprobs" not in lib.distill_loss(c["x"], c["ids"], c["teacher"], V=700)


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_against_differences(kind):
    """float32 gradient against central differences of the float64 forward pass."""
    V, K, h = 50, 6, 1e-5
    c = make(3, V, K, "f32", 21, kind, temps=[0.8])
    f = run(c)
    g, gl = torch.full((3,), -0.6, device="cuda"), torch.full((3,), 0.25, device="cuda")
    d = lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], grad_loss=g,
                              targets=c["targets"], logprobs=f["logprobs"], grad_logprobs=gl,
                              temperature=c["temperature"], V=V).double().cpu().numpy()
    x, legal, ids, q, t, T = host(c)
    for r in range(3):
        for j in range(V):
            y = []
            for e in (h, -h):
                z = x[r].copy()
                z[j] += e
                o = D.distill_row(z, ids[r], q[r], kind, int(t[r]), T[r], legal[r])
                y.append(float(g[r]) * o["loss"] + float(gl[r]) * o["logprob"])
            # differences: 1e-9; the float32 gradient: its terms, at most 4 in size, to 100u
            assert abs((y[0] - y[1]) / (2 * h) - d[r, j]) <= 1e-9 + 400 * U


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_bit_for_bit(dtype):
    c = make(40, 60001, 100, dtype, 2, masked=True, pad=7)
    a, b = run(c), run(c)
    for k in a:
        assert torch.equal(a[k].view(torch.int32), b[k].view(torch.int32)), k


def test_offsets_past_32_bits():
    B, V, ld = 4, 1000, (1 << 30) + 8
    small = make(B, V, 20, "bf16", 6)
    big = torch.empty((B, ld), dtype=torch.bfloat16, device="cuda")
    big[:, :V] = small["x"][:, :V]
    c = dict(small, x=big)
    a, b = run(c), run(small)
    for k in a:
        assert torch.equal(a[k].view(torch.int32), b[k].view(torch.int32)), k
    g = torch.ones(B, device="cuda")
    more = (c["ids"], a["slot_logprobs"], a["slot_grads"], a["stats"], g)
    ds = lib.distill_loss_grad(small["x"], *more, temperature=c["temperature"], V=V)
    db = lib.distill_loss_grad(big, *more, temperature=c["temperature"], V=V, out=big)
    torch.cuda.synchronize()
    assert torch.equal(ds, db[:, :V])


def test_streams_and_graphs():
    c = make(17, 20000, 20, "bf16", 12, masked=True)
    want = {k: v.clone() for k, v in run(c).items()}
    g = torch.randn(17, device="cuda")

    def grad(f, out=None):
        return lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], g,
                                     temperature=c["temperature"], bitmask=c["bitmask"], out=out)

    want_d = grad(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(c)
        got_d = grad(got)
    side.synchronize()
    for k in want:
        assert torch.equal(want[k].view(torch.int32), got[k].view(torch.int32)), k
    assert torch.equal(want_d, got_d)
    out, d = {k: torch.zeros_like(v) for k, v in want.items()}, torch.zeros_like(want_d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.distill_loss(c["x"], c["ids"], c["teacher"], targets=c["targets"], temperature=c["temperature"],
                         bitmask=c["bitmask"], out=out)
        grad(out, d)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(want[k].view(torch.int32), out[k].view(torch.int32)), k
        assert torch.equal(want_d, d)


def test_empty_batch_and_refusals():
    c = make(4, 300, 8, "bf16", 1)
    x, ids, q = c["x"], c["ids"], c["teacher"]
    z = lib.distill_loss(x[:0], ids[:0], q[:0])
    assert z["loss"].shape == (0,) and z["slot_grads"].shape == (0, 8)
    f = run(c)
    assert lib.distill_loss_grad(x[:0], ids[:0], f["slot_logprobs"][:0], f["slot_grads"][:0], f["stats"][:0]).shape == (0, 300)
    bad = [dict(kind="backward"), dict(teacher=q[:, :7]), dict(teacher=q.double()), dict(ids=ids.long()), dict(ids=ids[0]),
           dict(ids=ids[:, :0], teacher=q[:, :0]), dict(ids=ids.cpu()), dict(x=x.t()), dict(x=x.double()), dict(V=301),
           dict(V=0), dict(targets=c["targets"][:3]), dict(temperature=c["temperature"].double()),
           dict(bitmask=torch.zeros(4, 9, dtype=torch.int32, device="cuda")), dict(ids=ids.t().contiguous().t())]
    for b in bad:
        a = dict(x=x, ids=ids, teacher=q) | b
        with pytest.raises(ValueError):
            lib.distill_loss(a.pop("x"), a.pop("ids"), a.pop("teacher"), **a)
    with pytest.raises(lib.SmpError):  # more slots than a call takes
        lib.distill_loss(x, torch.full((4, 257), -1, dtype=torch.int32, device="cuda"), torch.zeros(4, 257, device="cuda"))
    g = torch.ones(4, device="cuda")
    a = (x, ids, f["slot_logprobs"], f["slot_grads"], f["stats"], g)
    for b in (dict(grad_logprobs=g), dict(grad_logprobs=g, targets=c["targets"]), dict(out=torch.empty_like(x)[:, :299]),
              dict(out=torch.empty(4, 300, device="cuda")), dict(temperature=g[:2])):
        with pytest.raises(ValueError):
            lib.distill_loss_grad(*a, **b)
    for i, t in ((2, f["slot_logprobs"][:, :7].contiguous()), (3, f["slot_grads"].double()), (4, f["stats"][:3])):
        with pytest.raises(ValueError):
            lib.distill_loss_grad(*a[:i], t, *a[i + 1:])

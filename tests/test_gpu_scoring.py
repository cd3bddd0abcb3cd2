"""Scoring of given tokens on the GPU (smp_token_logprobs,
smp_token_logprobs_grad, smp_head_logprobs) against the float64 oracle.

Tolerances.  u = 2^-24.  A scaled difference d = (x - m) s carries at most three
roundings, 2^d two units in the last place, and a sum of V weights at most V / 256 +
64 additions in a chain (a row is split over 256 threads or more, then joined):
a weight's relative error is 3u |z| + 4u, the mass's the weights' mean plus (V /
256 + 64) u.  A logarithm and a product round L and log p once more each.  So
    |log p - exact| <= u (4 |z_t| + 4 zbar + 4 L + V / 256 + 80),
zbar the mean of |z| under p, which L and the entropy bound: zbar = H - L.
The entropy adds zbar times the same relative error.  Ids, ranks and statuses
are exact: they come from comparisons of the stored logits."""
import numpy as np
import pytest
import torch

import top_selection_stats_gb300 as lib
from oracle import scoring as S
from top_selection_stats_gb300 import binding, workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = workloads.TORCH_DTYPE
OUT_EPS = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # relative, one rounding
OUT_TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}


def forward_tolerance(o, V, z):
    L, H = o["stats"][1], o["entropy"]
    return U * (4 * abs(z) + 4 * max(H - L, 0.0) + 4 * L + V / 256 + 80)


def make(B, V, dtype, seed, pad=0, shift=0, masked=False, temps=None, grid=None, neg_inf=0.0):
    """Logits [B, V + pad] whose first value lies ``shift`` elements past an aligned address."""
    case = workloads.random_case(seed, B, V, dtype=dtype, mask_frac=0.6 if masked else 0.0,
                                 grid=grid, neg_inf_frac=neg_inf)
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    ld = V + pad
    buf = torch.full((shift + B * ld,), float("nan"), dtype=DT[dtype], device="cuda")
    x = buf[shift:].view(B, ld)
    x[:, :V] = case["logits"].cuda()
    t = rng.integers(0, V, B).astype(np.int32)
    best = case["logits"].float().numpy().argmax(1)
    t[::3] = best[::3]
    t[5::7] = -1
    T = (rng.uniform(0.5, 1.5, B) if temps is None else np.resize(temps, B)).astype(np.float32)
    return dict(x=x, V=V, targets=torch.from_numpy(t).cuda(), temperature=torch.from_numpy(T).cuda(),
                bitmask=None if case["bitmask"] is None else case["bitmask"].cuda())


def reference(c, n=0):
    x = c["x"][:, :c["V"]].double().cpu().numpy()
    bm = None if c["bitmask"] is None else c["bitmask"].cpu().numpy().view(np.uint32)
    T = None if c["temperature"] is None else c["temperature"].cpu().numpy()
    return S.score(x, c["targets"].cpu().numpy(), T, bm, n)


def run(c, n=0):
    out = lib.token_logprobs(c["x"], c["targets"], temperature=c["temperature"],
                             bitmask=c["bitmask"], n_top=n, V=c["V"])
    torch.cuda.synchronize()
    return out


def check_forward(c, n):
    got = {k: v.cpu().numpy() for k, v in run(c, n).items()}
    ref = reference(c, n)
    x = c["x"][:, :c["V"]].double().cpu().numpy()
    T = np.ones(len(ref)) if c["temperature"] is None else c["temperature"].double().cpu().numpy()
    t = c["targets"].cpu().numpy()
    for r, o in enumerate(ref):
        assert got["status"][r] == o["status"], (r, got["status"][r], o["status"])
        assert got["rank"][r] == o["rank"], (r, got["rank"][r], o["rank"])
        if n:
            assert np.array_equal(got["top_ids"][r], o["top_ids"]), (r, got["top_ids"][r], o["top_ids"])
        if o["status"] != S.OK:
            for k in ("logprobs", "entropy", "stats"):
                assert np.all(np.isnan(got[k][r])), (r, k)
            if n:
                assert np.all(np.isnan(got["top_logprobs"][r])), r
            continue
        m, L = o["stats"]
        base = forward_tolerance(o, c["V"], 0.0)
        assert got["stats"][r, 0] == m, r
        assert abs(got["stats"][r, 1] - L) <= base, (r, got["stats"][r, 1], L, base)
        zbar = max(o["entropy"] - L, 0.0)
        assert abs(got["entropy"][r] - o["entropy"]) <= base * (1 + zbar) + 8 * U * zbar, (
            r, got["entropy"][r], o["entropy"])
        if o["logprob"] < -np.finfo(np.float32).max:  # -inf, or past float32
            assert got["logprobs"][r] == -np.inf, r
        else:
            z = 0.0 if t[r] < 0 else (x[r, t[r]] - m) / T[r]
            assert abs(got["logprobs"][r] - o["logprob"]) <= base + 4 * U * abs(z), (
                r, got["logprobs"][r], o["logprob"])
        if n:
            k = int((o["top_ids"] >= 0).sum())
            assert np.all(got["top_logprobs"][r, k:] == -np.inf), r
            z = (x[r, o["top_ids"][:k]] - m) / T[r]
            with np.errstate(over="ignore"):  # past float32: -inf
                want = o["top_logprobs"][:k].astype(np.float32).astype(np.float64)
            past = want == -np.inf
            assert np.all(got["top_logprobs"][r, :k][past] == -np.inf), r
            with np.errstate(invalid="ignore"):
                err = np.abs(np.where(past, 0.0, got["top_logprobs"][r, :k].astype(np.float64) - want))
            assert np.all(err <= base + 6 * U * np.abs(z)), (r, err.max())
    return got, ref


def check_grad(c, entropy, dtype, in_place=False):
    """The gradient from the forward call's own outputs.  p's relative error is the
    weight's (8u |log p| + 8u) plus L's absolute one, which base bounds; the rounding
    to dtype comes on top."""
    B, V = c["x"].shape[0], c["V"]
    f = run(c)
    rng = np.random.Generator(np.random.PCG64(B * 31 + V))
    g = torch.from_numpy(rng.standard_normal(B).astype(np.float32)).cuda()
    gh = torch.from_numpy(rng.standard_normal(B).astype(np.float32)).cuda() if entropy else None
    ref = reference(c)
    pad_before = c["x"][:, V:].clone()
    d = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], grad_logprobs=g,
                                entropy=f["entropy"] if entropy else None, grad_entropy=gh,
                                temperature=c["temperature"], bitmask=c["bitmask"], V=V,
                                out=c["x"] if in_place else None)
    torch.cuda.synchronize()
    if in_place:
        assert torch.equal(d[:, V:].view(torch.uint8), pad_before.view(torch.uint8)) if V < d.shape[1] else True
    else:
        assert not d[:, V:].any()
    d = d[:, :V].double().cpu().numpy()
    t = c["targets"].cpu().numpy()
    T = np.ones(B) if c["temperature"] is None else c["temperature"].double().cpu().numpy()
    g = g.double().cpu().numpy()
    gh = np.zeros(B) if gh is None else gh.double().cpu().numpy()
    for r, o in enumerate(ref):
        want = S.grad_row(o, int(t[r]), T[r], g[r], gh[r])
        if want is None:
            assert not d[r].any(), r
            continue
        lp = o["log_p"]
        legal = lp != -np.inf
        assert not d[r][~legal].any(), r
        p, al = np.exp(lp[legal]), np.abs(lp[legal])
        base = forward_tolerance(o, V, 0.0)
        zbar = max(o["entropy"] - o["stats"][1], 0.0)
        part = (abs(g[r]) * p + abs(gh[r]) * p * (al + o["entropy"] + 1)) / T[r]
        err = part * (base * (2 + zbar) + 8 * U * (1 + al + zbar))
        w = want[legal]
        tol = err + (np.abs(w) + err) * (OUT_EPS[dtype] + 4 * U) + OUT_TINY[dtype]
        if t[r] >= 0 and legal[t[r]]:
            tol[np.nonzero(legal)[0] == t[r]] += 4 * U * abs(g[r]) / T[r]
        off = np.abs(d[r][legal] - w)
        assert np.all(off <= tol), (r, off.max(), tol[off.argmax()], w[off.argmax()])


SIZES = [1, 2, 7, 8, 31, 33, 255, 1000, 4097, 32000, 70001, 128256]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", SIZES)
def test_forward(V, dtype):
    for n, pad, shift, masked in ((0, 0, 0, False), (5, 3, 1, True), (32, -V % 8, 0, True)):
        check_forward(make(13, V, dtype, V + n, pad=pad, shift=shift, masked=masked,
                           neg_inf=0.05 if masked else 0.0), n)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", SIZES)
def test_gradient(V, dtype):
    for entropy, pad, shift, masked in ((False, 0, 0, False), (True, 3, 1, True),
                                        (True, -V % 8, 0, True)):
        c = make(9, V, dtype, V + 5, pad=pad, shift=shift, masked=masked,
                 neg_inf=0.05 if masked else 0.0)
        check_grad(c, entropy, dtype)
        check_grad(c, entropy, dtype, in_place=True)


@pytest.mark.parametrize("B", [1, 2, 150, 700])
def test_batches(B):
    check_forward(make(B, 5003, "bf16", B), 4)
    check_grad(make(B, 5003, "bf16", B), True, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [40, 9000, 40000])
def test_ties(V, dtype):
    """Few distinct values: the alternatives' ids and the ranks are decided by id."""
    check_forward(make(12, V, dtype, V, grid=3, masked=True), 32)
    c = make(6, V, dtype, V, grid=1)  # all logits equal
    c["targets"] = torch.tensor([0, 1, V // 2, V - 1, -1, 7], dtype=torch.int32, device="cuda")
    check_forward(c, 32)
    check_grad(c, True, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [77, 20008])
def test_extreme_values(V, dtype):
    """Rows at the type's lowest value, beside -inf; one finite token; far from zero; a
    huge range; NaN and infinities in legal and in masked slots."""
    low = torch.finfo(DT[dtype]).min
    inf, nan = float("inf"), float("nan")
    c = make(16, V, dtype, V, temps=[1.0])
    x = c["x"]
    x[0] = low
    x[1] = low
    x[1, ::2] = -inf
    x[2] = -inf
    x[2, V // 3] = low
    x[3] = -inf
    x[4] += 900.0
    x[5, 1] = low
    x[5, 2] = -low
    x[6, V - 1] = nan
    x[7, 0] = inf
    x[8, :] = -inf
    x[8, 9] = inf
    x[9, 3] = nan
    x[10, V - 2] = inf
    x[11] = low
    x[11, V // 2] = 0.0
    x[12] = -low
    x[13] = 0.0
    x[13, ::3] = -0.0
    allowed = np.ones((16, V), bool)
    allowed[9, 3] = False
    allowed[10, V - 2] = False
    allowed[14] = False
    allowed[15] = False
    allowed[15, V - 1] = True
    c["bitmask"] = torch.from_numpy(workloads.mask_from_allowed(allowed).view(np.int32)).cuda()
    c["targets"] = torch.arange(16, dtype=torch.int32, device="cuda") % V
    c["targets"][2] = V // 3
    got, _ = check_forward(c, 6)
    st = list(got["status"])
    assert st[:4] == [0, 0, 0, 1] and st[6:9] == [2, 2, 2] and st[9:12] == [0, 0, 0] and st[14] == 1
    check_grad(c, True, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_temperatures(dtype):
    temps = [1e-30, 1e-3, 0.05, 1.0, 20.0, 1e4, 1e30, 0.0, -1.0, float("nan"), float("inf"), 1e-42]
    c = make(12, 3001, dtype, 3, temps=temps)
    got, _ = check_forward(c, 3)
    assert list(got["status"]) == [0] * 7 + [3] * 4 + [0]
    c = make(12, 3001, dtype, 3, temps=[1e-3, 0.05, 20.0, 1e4, 0.0, float("nan")])
    check_grad(c, True, dtype)
    c["temperature"] = None
    check_forward(c, 3)
    check_grad(c, False, dtype)


def test_targets_outside_and_illegal():
    c = make(8, 500, "bf16", 4, masked=True)
    c["targets"] = torch.tensor([500, -2, 1 << 30, -(1 << 31), -1, 0, 1, 499], dtype=torch.int32, device="cuda")
    got, _ = check_forward(c, 2)
    assert list(got["status"][:4]) == [3] * 4
    check_grad(c, True, "bf16")


def test_grad_parts_may_be_missing():
    c = make(6, 700, "f32", 8)
    f = run(c)
    z = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], temperature=c["temperature"], V=700)
    assert not z.any()
    gh = torch.ones(6, device="cuda")
    a = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], entropy=f["entropy"], grad_entropy=gh,
                                temperature=c["temperature"], V=700)
    b = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], grad_logprobs=0 * gh, entropy=f["entropy"],
                                grad_entropy=gh, temperature=c["temperature"], V=700)
    assert torch.equal(a, b) and a.any()


def test_gradient_against_differences():
    """float32 gradient against central differences of the float64 forward pass."""
    V, T, h = 50, 0.8, 1e-5
    c = make(3, V, "f32", 21, temps=[T])
    c["targets"] = torch.tensor([0, 49, 7], dtype=torch.int32, device="cuda")
    f = run(c)
    g, gh = torch.full((3,), -0.6, device="cuda"), torch.full((3,), 0.25, device="cuda")
    d = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], grad_logprobs=g, entropy=f["entropy"],
                                grad_entropy=gh, temperature=c["temperature"], V=V).double().cpu().numpy()
    x = c["x"][:, :V].double().cpu().numpy()
    T = float(c["temperature"][0])
    for r, t in enumerate([0, 49, 7]):
        for j in range(V):
            y = []
            for e in (h, -h):
                z = x[r].copy()
                z[j] += e
                o = S.score_row(z, t, T, np.ones(V, bool), 0)
                y.append(float(g[r]) * o["logprob"] + float(gh[r]) * o["entropy"])
            # differences: 1e-9; the float32 gradient: its terms, at most 3 in size, to 100u
            assert abs((y[0] - y[1]) / (2 * h) - d[r, j]) <= 1e-9 + 300 * U


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_bit_for_bit(dtype):
    c = make(40, 60001, dtype, 2, masked=True, pad=7)
    a, b = run(c, 32), run(c, 32)
    for k in a:
        assert torch.equal(a[k].view(torch.int32), b[k].view(torch.int32)), k


def test_offsets_past_32_bits():
    B, V, ld = 4, 1000, (1 << 30) + 8
    small = make(B, V, "bf16", 6)
    big = torch.empty((B, ld), dtype=torch.bfloat16, device="cuda")
    big[:, :V] = small["x"][:, :V]
    c = dict(small, x=big)
    a, b = run(c, 4), run(small, 4)
    for k in a:
        assert torch.equal(a[k].view(torch.int32), b[k].view(torch.int32)), k
    g = torch.ones(B, device="cuda")
    ds = lib.token_logprobs_grad(small["x"], c["targets"], a["stats"], grad_logprobs=g,
                                 temperature=c["temperature"], V=V)
    db = lib.token_logprobs_grad(big, c["targets"], a["stats"], grad_logprobs=g,
                                 temperature=c["temperature"], V=V, out=big)
    torch.cuda.synchronize()
    assert torch.equal(ds, db[:, :V])


def test_streams_and_graphs():
    c = make(17, 20000, "bf16", 12, masked=True)
    want = {k: v.clone() for k, v in run(c, 8).items()}
    g = torch.randn(17, device="cuda")
    want_d = lib.token_logprobs_grad(c["x"], c["targets"], want["stats"], grad_logprobs=g,
                                     temperature=c["temperature"], bitmask=c["bitmask"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = lib.token_logprobs(c["x"], c["targets"], temperature=c["temperature"], bitmask=c["bitmask"], n_top=8)
    side.synchronize()
    for k in want:
        assert torch.equal(out[k].view(torch.int32), want[k].view(torch.int32)), k
    graph = torch.cuda.CUDAGraph()
    d = torch.empty_like(c["x"])
    for v in out.values():
        v.zero_()
    with torch.cuda.graph(graph):
        lib.token_logprobs(c["x"], c["targets"], temperature=c["temperature"], bitmask=c["bitmask"], n_top=8, out=out)
        lib.token_logprobs_grad(c["x"], c["targets"], out["stats"], grad_logprobs=g, temperature=c["temperature"],
                                bitmask=c["bitmask"], out=d)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(out[k].view(torch.int32), want[k].view(torch.int32)), k
    assert torch.equal(d, want_d)


def test_no_rows():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    out = lib.token_logprobs(e, t, n_top=3)
    assert out["logprobs"].numel() == 0 and out["top_ids"].shape == (0, 3)
    assert lib.token_logprobs_grad(e, t, out["stats"]).shape == (0, 64)
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    assert lib.head_logprobs(e, w, t)["logprobs"].numel() == 0


# -- from hidden states ---------------------------------------------------------
def head_case(N, V, D, dtype, seed, pad=0, temps=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.full((N, D + pad), float("nan"), dtype=DT[dtype], device="cuda")
    w = torch.full((V, D + pad), float("nan"), dtype=DT[dtype], device="cuda")
    h[:, :D] = torch.randn(N, D, generator=g, device="cuda").to(DT[dtype])
    w[:, :D] = (torch.randn(V, D, generator=g, device="cuda") * (3.0 / D ** 0.5)).to(DT[dtype])
    t = torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32)
    t[3::11] = -1
    T = 0.6 + torch.rand(N, generator=g, device="cuda") if temps else None
    return dict(h=h, w=w, targets=t, temperature=T, D=D)


def check_head(c, **kw):
    """The products of 16-bit values are exact in binary32; a sum of D of them is taken as D / 16
    blocks whose roundings, each at most two units in the last place of the terms' size,
    do not conspire: |x - exact| <= 8 sqrt(D / 16 + 1) 2u |h| |w| (Cauchy-Schwarz)."""
    out = lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"], D=c["D"], **kw)
    torch.cuda.synchronize()
    h, w = c["h"][:, :c["D"]].double().cpu(), c["w"][:, :c["D"]].double().cpu()
    x = (h @ w.t()).numpy()
    V = x.shape[1]
    T = None if c["temperature"] is None else c["temperature"].cpu().numpy()
    ref = S.score(x, c["targets"].cpu().numpy(), T)
    size = h.norm(dim=1).numpy() * float(w.norm(dim=1).max())
    dx = 16 * U * (c["D"] / 16 + 1) ** 0.5 * size
    got = {k: v.cpu().numpy() for k, v in out.items()}
    t = c["targets"].cpu().numpy()
    for r, o in enumerate(ref):
        assert got["status"][r] == o["status"] == S.OK, r
        Tr = 1.0 if T is None else float(T[r])
        m, L = o["stats"]
        zbar = max(o["entropy"] - L, 0.0)
        z = 0.0 if t[r] < 0 else (x[r, t[r]] - m) / Tr
        tol = forward_tolerance(o, V, z) + 2 * dx[r] / Tr
        assert abs(got["stats"][r, 0] - m) <= dx[r] + 2 * U * abs(m), r
        assert abs(got["stats"][r, 1] - L) <= tol, r
        assert abs(got["logprobs"][r] - o["logprob"]) <= tol, (r, got["logprobs"][r], o["logprob"], tol)
        assert abs(got["entropy"][r] - o["entropy"]) <= tol * (2 + zbar), (r, got["entropy"][r], o["entropy"])
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,V,D,pad", [
    (1, 1, 8, 0), (1, 300, 64, 0), (2, 257, 136, 0), (5, 1000, 1, 7), (3, 511, 100, 4),
    (127, 1025, 72, 0), (128, 2048, 256, 0), (129, 2049, 264, 8), (300, 700, 1000, 0),
    (17, 33000, 128, 0), (1, 40001, 512, 0), (700, 5000, 192, 0)])
def test_head(N, V, D, pad, dtype):
    check_head(head_case(N, V, D, dtype, N + V, pad=pad))


def test_head_without_temperature_and_with_reused_buffers():
    c = head_case(200, 3001, 96, "bf16", 5, temps=False)
    ws = torch.empty(lib.head_workspace(200, 3001), dtype=torch.uint8, device="cuda")
    out = check_head(c, workspace=ws)
    again = check_head(c, workspace=ws, out=out)
    assert again is out
    a = {k: v.clone() for k, v in out.items()}
    b = check_head(c)
    for k in a:  # no atomics: the same bits each time
        assert torch.equal(a[k].view(torch.int32), b[k].view(torch.int32)), k


def test_head_agrees_with_the_logits_path():
    """The same distribution through float32 logits: the chain a user would write."""
    c = head_case(50, 4000, 320, "bf16", 9)
    out = check_head(c)
    x = (c["h"].double() @ c["w"].double().t()).float()
    o2 = lib.token_logprobs(x, c["targets"], temperature=c["temperature"])
    torch.cuda.synchronize()
    assert (out["logprobs"] - o2["logprobs"]).abs().max() < 1e-3
    assert (out["entropy"] - o2["entropy"]).abs().max() < 1e-3


def test_head_statuses():
    c = head_case(6, 600, 64, "bf16", 3)
    c["h"][1, 5] = float("nan")
    c["h"][2, 5] = float("inf")
    c["targets"] = torch.tensor([600, 0, 1, -1, 3, 4], dtype=torch.int32, device="cuda")
    c["temperature"][4] = 0.0
    out = lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"])
    torch.cuda.synchronize()
    assert out["status"].tolist() == [3, 2, 2, 0, 3, 0]
    lp = out["logprobs"].cpu()
    assert torch.isnan(lp[[0, 1, 2, 4]]).all() and lp[3] == 0 and torch.isfinite(lp[5])
    assert torch.isnan(out["stats"].cpu()[[0, 1, 2, 4]]).all()


def test_head_weight_rows_of_minus_infinity_are_not_legal():
    """A weight row that gives -inf for a state leaves its token out, as -inf logits do."""
    c = head_case(4, 70, 8, "f16", 2, temps=False)
    c["h"][:] = c["h"].abs() + 0.1
    c["w"][10:30, 0] = float("-inf")
    c["targets"] = torch.tensor([0, 10, 69, 29], dtype=torch.int32, device="cuda")
    out = lib.head_logprobs(c["h"], c["w"], c["targets"])
    torch.cuda.synchronize()
    x = c["h"].double().cpu() @ c["w"].double().cpu().t()
    ref = S.score(x.numpy(), c["targets"].cpu().numpy())
    assert out["status"].tolist() == [0] * 4
    for r in range(4):
        if r in (1, 3):
            assert out["logprobs"][r] == -float("inf")
        else:
            assert abs(float(out["logprobs"][r]) - ref[r]["logprob"]) < 1e-4
        assert abs(float(out["entropy"][r]) - ref[r]["entropy"]) < 1e-4


# -- refusals -------------------------------------------------------------------
def test_refusals():
    x = torch.zeros((4, 64), device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = lib.token_logprobs(x, t)
    for bad in (dict(targets=t.long()), dict(targets=t[:3]), dict(temperature=torch.ones(4)),
                dict(temperature=torch.ones(3, device="cuda")), dict(V=65), dict(V=0), dict(n_top=-1),
                dict(bitmask=torch.zeros((4, 3), dtype=torch.int32, device="cuda")),
                dict(logits=x.double()), dict(logits=x.t()), dict(logits=x[0]), dict(logits=x.cpu())):
        with pytest.raises(ValueError):
            lib.token_logprobs(**{**dict(logits=x, targets=t), **bad})
        torch.cuda.synchronize()
    with pytest.raises(lib.SmpError) as e:
        lib.token_logprobs(x, t, n_top=33)
    assert e.value.code == lib.SMP_ERR_CAPACITY
    with pytest.raises(ValueError):
        lib.token_logprobs_grad(x, t, ok["stats"], grad_entropy=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        lib.token_logprobs_grad(x, t, ok["stats"], out=x.half())
    with pytest.raises(ValueError):
        lib.token_logprobs_grad(x, t, ok["stats"].t())
    h = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((100, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(hidden=h.float(), weight=w.float()), dict(weight=w.half()), dict(weight=w[:, :32].contiguous()),
                dict(hidden=h[:, :60].contiguous(), weight=w[:, :60].contiguous()), dict(D=65),
                dict(workspace=torch.empty(3, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            lib.head_logprobs(**{**dict(hidden=h, weight=w, targets=t), **bad})
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.SmpError) as e:  # not 16-byte aligned
        lib.head_logprobs(flat[1:257].view(4, 64), w, t)
    assert e.value.code == lib.SMP_ERR_INVALID_PARAM
    torch.cuda.synchronize()


def test_c_entry_refusals():
    L = lib.load_library()
    p = torch.zeros(1024, device="cuda").data_ptr()
    ok = [p, 0, 4, 64, 64, None, None, p, p, p, p, p, p, 0, None, None, None]
    for i, v in ((0, None), (1, 3), (2, -1), (3, 0), (4, 63), (8, None), (12, None), (13, -1), (13, 2)):
        a = list(ok)
        a[i] = v
        assert L.smp_token_logprobs(*a) == lib.SMP_ERR_INVALID_PARAM, i
    a = list(ok)
    a[3] = a[4] = (1 << 24) + 1
    assert L.smp_token_logprobs(*a) == lib.SMP_ERR_CAPACITY
    ok = [p, 0, 4, 64, 64, None, None, p, p, p, p, None, p, 64, None]
    for i, v in ((0, None), (1, -1), (4, 60), (7, None), (8, None), (12, None), (13, 60), (13, 128)):
        a = list(ok)
        a[i] = v
        assert L.smp_token_logprobs_grad(*a) == lib.SMP_ERR_INVALID_PARAM, i
    need = L.smp_head_workspace(4, 100)
    ok = [p, 64, p, 64, binding.SMP_BF16, 4, 100, 64, None, p, p, p, p, p, p, need, None]
    for i, v in ((0, None), (1, 60), (1, 68), (3, 68), (4, 0), (5, -1), (6, 0), (7, 0), (7, 72), (10, None),
                 (13, None), (14, None), (14, p + 8), (0, p + 2), (15, need - 1)):
        a = list(ok)
        a[i] = v
        assert L.smp_head_logprobs(*a) == lib.SMP_ERR_INVALID_PARAM, (i, v)
    assert L.smp_head_workspace(0, 5) == 0 and L.smp_head_workspace(5, 0) == 0

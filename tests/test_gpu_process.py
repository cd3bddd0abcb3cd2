"""Processing of logits on the GPU (smp_process_logits) against the float64 oracle.

Tolerance: each binary32 operation is correctly rounded (u = 2^-24 relative to its result), so a
result is off by at most u times the sum of the intermediate results' magnitudes, and by one
rounding to the result's type.  Values that no history or bias names are the logits', bit for
bit."""
import numpy as np
import pytest
import torch

import top_selection_stats_gb300 as lib
from oracle import processing as P
from oracle import scoring as S
from top_selection_stats_gb300 import workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = workloads.TORCH_DTYPE
EPS = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # relative, one rounding
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}
NAMES = ("history", "lengths", "prompt_lengths", "repetition", "presence", "frequency", "bias_ids", "bias", "bitmask")


def make(B, V, H, NB, dtype, seed, pad=0, shift=0, masked=False, neg_inf=0.0, spread=None):
    """Logits whose first value lies ``shift`` elements past an aligned address; histories with
    padding inside and behind, tokens that repeat, biases with repeated ids and bans."""
    case = workloads.random_case(seed, B, V, dtype=dtype, mask_frac=0.6 if masked else 0.0, neg_inf_frac=neg_inf)
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    ld = V + pad
    buf = torch.full((shift + B * ld,), 7.0, dtype=DT[dtype], device="cuda")
    x = buf[shift:].view(B, ld)
    x[:, :V] = case["logits"].cuda()
    c = dict(x=x, V=V, bitmask=None if case["bitmask"] is None else case["bitmask"].cuda())

    def dev(a, dt):
        return torch.from_numpy(np.ascontiguousarray(a.astype(dt))).cuda()

    if H:
        h = rng.integers(-1, V + 1, (B, H)) if spread is None else rng.integers(0, spread, (B, H)) * (V // spread)
        length = rng.integers(0, H + 1, B)
        length[0] = H
        c.update(history=dev(h, np.int32), lengths=dev(length, np.int32),
                 prompt_lengths=dev((length * rng.random(B)).astype(int), np.int32),
                 repetition=dev(rng.uniform(0.7, 1.6, B), np.float32), presence=dev(rng.uniform(-1, 1, B), np.float32),
                 frequency=dev(rng.uniform(-0.2, 0.5, B), np.float32))
    if NB:
        ids = rng.integers(-2, V + 2, (B, NB))
        ids[:, NB // 2:] = ids[:, :NB - NB // 2]  # every id twice
        b = rng.uniform(-5, 5, (B, NB))
        b[rng.random((B, NB)) < 0.1] = -np.inf
        c.update(bias_ids=dev(ids, np.int32), bias=dev(b, np.float32))
    return c


def reference(c):
    B, V = c["x"].shape[0], c["V"]
    x = c["x"][:, :V].double().cpu().numpy()
    h = {k: None if c.get(k) is None else c[k].cpu().numpy() for k in NAMES}
    legal = np.ones((B, V), bool) if h["bitmask"] is None else S.unpack(h["bitmask"].view(np.uint32), V)
    rows = []
    for r in range(B):
        at = lambda k, other: other if h[k] is None else h[k][r]  # noqa: E731
        hist = at("history", np.zeros(0, int))
        n, prompt = int(at("lengths", len(hist))), int(at("prompt_lengths", 0))
        if not 0 <= n <= len(hist):
            rows.append((P.INVALID, x[r].copy(), np.zeros(V)))
            continue
        f = lambda k, other: float(np.float64(at(k, other)))  # noqa: E731
        rows.append(P.process_row(x[r], hist[:n], prompt, f("repetition", 1.0), f("presence", 0.0), f("frequency", 0.0),
                                  at("bias_ids", np.zeros(0, int)), at("bias", np.zeros(0)).astype(np.float64), legal[r]))
    return rows


def call(c, **more):
    return lib.process_logits(c["x"], **{k: c.get(k) for k in NAMES}, V=c["V"], **more)


def check(c, dtype, out="same", in_place=False):
    V = c["V"]
    rows = reference(c)
    raw = c["x"].clone()
    odt = dtype if out == "same" else out
    got = call(c, dtype=DT[odt], in_place=in_place)
    torch.cuda.synchronize()
    y = got["logits"]
    assert (y.data_ptr() == c["x"].data_ptr()) == in_place and y.dtype == DT[odt] and y.shape == c["x"].shape
    if in_place:
        assert torch.equal(y[:, V:], raw[:, V:])
    else:
        assert torch.equal(c["x"].view(torch.uint8), raw.view(torch.uint8)) and (y[:, V:] == -float("inf")).all()
    st, y = got["status"].cpu().numpy(), y[:, :V].double().cpu().numpy()
    x = raw[:, :V].double().cpu().numpy()
    most = float(torch.finfo(DT[odt]).max)
    for r, (status, want, size) in enumerate(rows):
        assert st[r] == status, (r, st[r], status)
        same = size == 0
        plain = same & ((want == x[r]) | (np.isnan(want) & np.isnan(x[r])))
        assert np.array_equal(y[r][plain], x[r][plain], equal_nan=True), r
        inf = np.isinf(want) | (np.abs(want) > most * (1 - 1e-3))
        assert np.array_equal(y[r][np.isinf(want)], want[np.isinf(want)]), r
        rest = ~inf & ~np.isnan(want)
        tol = U * size + (np.abs(want) + U * size) * EPS[odt] * (1 + 1e-6) + TINY[odt]
        off = np.abs(y[r] - np.where(rest, want, 0.0))
        bad = rest & (off > tol)
        assert not bad.any(), (r, np.nonzero(bad)[0][:5], y[r][bad][:5], want[bad][:5])
        assert np.array_equal(np.isnan(y[r]), np.isnan(want)), r


SIZES = [1, 2, 7, 8, 31, 33, 255, 1000, 4097, 8192, 8193, 32000, 70001, 128256]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", SIZES)
def test_sizes(V, dtype):
    for H, NB, pad, shift, masked in ((0, 0, 0, 0, False), (1, 1, 3, 1, True), (50, 7, -V % 8, 0, False),
                                      (700, 300, 1, 3, True)):
        for out in ("same", "f32"):
            check(make(5, V, H, NB, dtype, V + H, pad, shift, masked, 0.05 if masked else 0.0), dtype, out)
        check(make(5, V, H, NB, dtype, V + H, pad, shift, masked, 0.05 if masked else 0.0), dtype, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H", [2047, 4096, 20001, 140000])
def test_long_histories(H, in_place):
    check(make(3, 50001, H, 0, "bf16", H, masked=True), "bf16", in_place=in_place)
    # few tokens, each thousands of times: the counts are exact
    check(make(3, 9001, H, 5, "f32", H + 1, spread=9), "f32", in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [1, 2, 150, 700])
def test_batches(B, in_place):
    check(make(B, 5003, 100, 9, "bf16", B, masked=True), "bf16", in_place=in_place)
    check(make(B, 5003, 100, 9, "f16", B, pad=5), "f16", in_place=in_place)


@pytest.mark.parametrize("NB", [1, 33, 1000, 4096])
def test_biases(NB):
    """Many biases, each id twice, on a small vocabulary: sums in slot order."""
    for V in (40, 9000):
        check(make(4, V, 20, NB, "f32", NB), "f32")
        check(make(4, V, 0, NB, "bf16", NB), "bf16", in_place=True)


def test_binary32_steps():
    """Bit for bit the binary32 operations in the order that the header states."""
    c = make(4, 300, 60, 40, "f32", 77)
    got = call(c)["logits"].cpu().numpy()
    x = c["x"].cpu().numpy()
    h = {k: c[k].cpu().numpy() for k in NAMES if c.get(k) is not None}
    f = np.float32
    for r in range(4):
        n, prompt = h["lengths"][r], h["prompt_lengths"][r]
        hist, made = h["history"][r, :n], h["history"][r, prompt:n]
        for j in range(300):
            v = x[r, j]
            if (hist == j).any():
                v = f(v / h["repetition"][r]) if v > 0 else f(v * h["repetition"][r])
                k = int((made == j).sum())
                v = f(v - f(f(h["frequency"][r] * f(k)) + (h["presence"][r] if k else f(0))))
            for i in np.nonzero(h["bias_ids"][r] == j)[0]:
                v = f(-np.inf) if -np.inf in (v, h["bias"][r, i]) else f(v + h["bias"][r, i])
            assert got[r, j] == v, (r, j)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_extreme_values(dtype, in_place):
    """The type's lowest and largest values, -inf, NaN and +inf, touched, masked and neither."""
    V = 5000
    c = make(10, V, 2000, 20, dtype, 3, masked=True)
    low = torch.finfo(DT[dtype]).min
    inf, nan = float("inf"), float("nan")
    x = c["x"]
    x[0] = low
    x[1] = -inf
    x[2, ::2] = nan
    x[3, ::3] = inf
    x[4, ::2] = -inf
    x[5] = 0.0
    x[6, ::2] = -0.0
    x[7] = torch.finfo(DT[dtype]).tiny
    c["repetition"][0] = 1.0
    c["frequency"][3:4] = c["presence"][3:4] = 0.25
    check(c, dtype, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H", [40, 3000])
def test_ids_far_outside(H, in_place):
    """Entries and biases at the ends of int32 are padding."""
    c = make(3, 30001, H, 40, "bf16", 9, shift=3, masked=H == 40)
    far = torch.tensor([-(1 << 31), (1 << 31) - 1, -(1 << 31) + 30000, 1 << 30, 30001, -1], dtype=torch.int32, device="cuda")
    c["history"][:, 3:9] = far
    c["bias_ids"][:, 3:9] = far
    check(c, "bf16", in_place=in_place)
    del c["bitmask"]
    check(c, "bf16", in_place=in_place)


def test_masks_that_leave_nothing():
    c = make(4, 3000, 10, 3, "bf16", 1, masked=True)
    c["bitmask"][1] = 0
    c["bitmask"][2] = -1
    check(c, "bf16")
    y = call(c)["logits"]
    assert (y[1] == -float("inf")).all() and not (y[2] == -float("inf")).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_invalid_rows_go_through(in_place):
    nan, inf = float("nan"), float("inf")
    c = make(16, 9000, 30, 6, "bf16", 8, masked=True)
    for r, (k, v) in enumerate([("repetition", 0.0), ("repetition", -1.0), ("repetition", nan), ("repetition", inf),
                                ("presence", nan), ("presence", -inf), ("frequency", inf), ("frequency", nan),
                                ("lengths", 31), ("lengths", -1), ("prompt_lengths", -1)]):
        c[k][r] = v
    c["lengths"][11], c["prompt_lengths"][11] = 4, 5
    c["bias_ids"][12:15, 2] = torch.tensor([1, 8999, -1], dtype=torch.int32)
    c["bias"][12:15, 2] = torch.tensor([nan, inf, nan])  # the last in an unused slot
    raw = c["x"].clone()
    check(c, "bf16", in_place=in_place)
    if in_place:
        c["x"].copy_(raw)
    st = call(c)["status"].cpu()
    assert list(st[:14]) == [3] * 14 and st[14] == 0 and st[15] == 0


def test_parts_may_be_missing():
    c = make(5, 2000, 40, 6, "f32", 2, masked=True)
    for drop in (("lengths",), ("prompt_lengths",), ("repetition",), ("presence", "frequency"), ("history", "lengths", "prompt_lengths"),
                 ("bias_ids", "bias"), ("bitmask",), NAMES):
        check({k: v for k, v in c.items() if k not in drop}, "f32")
        check({k: v.clone() if torch.is_tensor(v) else v for k, v in c.items() if k not in drop}, "f32", in_place=True)


def test_matches_the_repetition_penalty():
    """Without the other steps in place: what Sampler.repetition_penalty does."""
    s = lib.Sampler(0, max_batch=8, max_vocab=1 << 16)
    for dtype in ("f32", "bf16", "f16"):
        c = make(8, 40000, 500, 0, dtype, 5)
        want = c["x"].clone()
        s.repetition_penalty(want, c["history"], c["repetition"])
        got = lib.process_logits(c["x"], history=c["history"], repetition=c["repetition"], in_place=True)
        assert got["logits"] is c["x"] and torch.equal(got["logits"], want)
    s.close()


def test_repeats_bit_for_bit():
    c = make(40, 60001, 3000, 200, "f32", 2, masked=True, pad=7)
    a, b = call(c), call(c)
    assert torch.equal(a["logits"].view(torch.int32), b["logits"].view(torch.int32))


def test_offsets_past_32_bits():
    B, V, ld = 4, 1000, (1 << 30) + 8
    c = make(B, V, 50, 5, "bf16", 6, masked=True)
    want = call(c)["logits"]
    big = torch.empty((B, ld), dtype=torch.bfloat16, device="cuda")
    big[:, :V] = c["x"]
    got = call(dict(c, x=big), in_place=True)["logits"]
    assert torch.equal(got[:, :V].view(torch.int16), want.view(torch.int16))
    del big, got
    # the longest history that a call takes
    h = torch.full((2, 1 << 24), -1, dtype=torch.int32, device="cuda")
    h[1, -1] = 5
    x = torch.ones(2, 100, device="cuda")
    y = lib.process_logits(x, history=h, presence=torch.ones(2, device="cuda"))["logits"]
    assert y[1, 5] == 0 and y.sum() == 199


def test_streams_graphs_and_reuse():
    c = make(17, 20000, 300, 20, "bf16", 12, masked=True)
    want = call(c)
    wl, ws = want["logits"].clone(), want["status"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(c)
    side.synchronize()
    assert torch.equal(got["logits"], wl) and torch.equal(got["status"], ws)
    want["logits"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert call(c, out=want) is want
    for _ in range(2):
        want["logits"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want["logits"], wl)
    # a result with other rows, aligned unlike the logits
    wide = dict(logits=torch.zeros(17, 20003, dtype=torch.bfloat16, device="cuda"), status=ws)
    call(c, out=wide)
    assert torch.equal(wide["logits"][:, :20000], wl) and not wide["logits"][:, 20000:].any()


def test_empty_batch_and_refusals():
    c = make(4, 300, 8, 4, "bf16", 1)
    x, h, b, ids = c["x"], c["history"], c["bias"], c["bias_ids"]
    z = lib.process_logits(x[:0], history=h[:0])
    assert z["logits"].shape == (0, 300) and z["status"].shape == (0,)
    assert torch.equal(lib.process_logits(x, history=h[:, :0])["logits"], x)
    for bad in (dict(history=h[:3]), dict(history=h.long()), dict(history=h[0]), dict(history=h.cpu()),
                dict(history=h.t().contiguous().t()), dict(lengths=c["lengths"]), dict(prompt_lengths=c["lengths"]),
                dict(history=h, lengths=c["lengths"][:2]), dict(repetition=c["repetition"].double()), dict(bias=b),
                dict(bias_ids=ids), dict(bias=b[:, :2], bias_ids=ids), dict(bias=b.half(), bias_ids=ids), dict(V=301),
                dict(dtype=torch.float16), dict(dtype=torch.float32, in_place=True), dict(dtype=torch.float64),
                dict(bitmask=torch.zeros(4, 9, dtype=torch.int32, device="cuda")),
                dict(out=dict(logits=x[:3], status=c["lengths"])), dict(out=dict(logits=x[:, :299].contiguous(), status=c["lengths"])),
                dict(out=dict(logits=x.float(), status=c["lengths"])), dict(out=dict(logits=x.clone(), status=c["lengths"][:3]))):
        with pytest.raises(ValueError):
            lib.process_logits(x, **bad)
    with pytest.raises(ValueError):
        lib.process_logits(x.t())
    with pytest.raises(ValueError):
        lib.process_logits(x.double())
    with pytest.raises(lib.SmpError):  # more biases than a call takes
        lib.process_logits(x, bias_ids=torch.zeros(4, 4097, dtype=torch.int32, device="cuda"),
                           bias=torch.zeros(4, 4097, device="cuda"))

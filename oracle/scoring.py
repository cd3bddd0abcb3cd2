"""Scoring of given tokens in float64 with numpy, row by row: log probability,
entropy, rank and alternatives of softmax(x / T) over the legal tokens, and the
gradient of the first two.  Test infrastructure only."""
import numpy as np

OK, EMPTY, NONFINITE, INVALID = 0, 1, 2, 3


def unpack(bitmask, V):
    """uint32 [B, W] -> bool [B, V]."""
    bits = (bitmask[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1
    return bits.reshape(bitmask.shape[0], -1)[:, :V].astype(bool)


def score_row(x, t, T, legal, n):
    """x float64 [V]; legal bool [V].  Returns a dict; NaN / -1 on an error row."""
    V = x.size
    bad = dict(logprob=np.nan, entropy=np.nan, rank=-1, stats=(np.nan, np.nan), log_p=None,
               top_ids=np.full(n, -1), top_logprobs=np.full(n, np.nan))
    if not (T > 0 and np.isfinite(T)) or not -1 <= t < V:
        return dict(bad, status=INVALID)
    legal = legal & (x != -np.inf)
    if np.any(~(x[legal] < np.inf)):  # NaN or +inf
        return dict(bad, status=NONFINITE)
    if not legal.any():
        return dict(bad, status=EMPTY)
    ids = np.nonzero(legal)[0]
    m = x[ids].max()
    z = (x[ids] - m) / T
    w = np.exp(z)
    L = np.log(w.sum())
    log_p = np.full(V, -np.inf)
    log_p[ids] = z - L
    order = ids[np.argsort(-x[ids], kind="stable")]
    rank = -1
    if t >= 0:
        rank = int(np.nonzero(order == t)[0][0]) if legal[t] else len(ids)
    top = np.full(n, -1)
    tlp = np.full(n, -np.inf)
    k = min(n, len(order))
    top[:k] = order[:k]
    tlp[:k] = log_p[order[:k]]
    return dict(status=OK, logprob=0.0 if t < 0 else log_p[t], rank=rank, stats=(m, L),
                entropy=L - float((w * z).sum() / w.sum()), log_p=log_p, top_ids=top,
                top_logprobs=tlp)


def score(x, targets, temperature=None, bitmask=None, n=0):
    """x float64 [B, V], targets [B].  A list of score_row's dicts."""
    B, V = x.shape
    T = np.ones(B) if temperature is None else np.asarray(temperature, np.float64)
    legal = np.ones((B, V), bool) if bitmask is None else unpack(bitmask, V)
    return [score_row(x[r], int(targets[r]), T[r], legal[r], n) for r in range(B)]


def grad_row(row, t, T, g, gh):
    """Gradient of g * logprob + gh * entropy for one score_row result, float64
    [V], or None for a row that failed (its gradient is zero)."""
    if row["status"] != OK:
        return None
    log_p = row["log_p"]
    legal = log_p != -np.inf
    p = np.exp(log_p)
    lead = g if t >= 0 and legal[t] else 0.0
    d = -lead * p
    if lead:
        d[t] += lead
    d[legal] -= gh * p[legal] * (log_p[legal] + row["entropy"])
    return d / T

"""Divergence from a teacher's top tokens and its gradient in float64 with numpy, row by
row.  Test infrastructure only."""
import numpy as np

from .scoring import EMPTY, INVALID, NONFINITE, OK

LEAST, MOST = 2.0 ** -24, 1 + 2.0 ** -10


def _xlogy(w, d):
    """w d with 0 where w is 0."""
    return np.where(w > 0, w * np.where(w > 0, d, 0.0), 0.0)


def distill_row(x, ids, teacher, kind, t, T, legal):
    """x float64 [V]; ids int [K] (-1: unused), teacher float64 [K]; t: target or -1; legal bool
    [V].  A dict; status alone on an error row."""
    V = x.size
    used = ids >= 0
    if (not (T > 0 and np.isfinite(T)) or not -1 <= t < V or np.any((ids < -1) | (ids >= V))
            or len(set(ids[used])) != used.sum()):
        return dict(status=INVALID)
    v = np.where(used, teacher, -np.inf)
    legal = legal & (x != -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind != "truncated" and np.exp(v[v < np.inf]).sum() > MOST:
            return dict(status=INVALID)
    if np.any(~(x[legal] < np.inf)) or np.any(~(v < np.inf)):
        return dict(status=NONFINITE)
    if not legal.any():
        return dict(status=EMPTY)
    m = x[legal].max()
    z = np.where(legal, (np.where(legal, x, m) - m) / T, -np.inf)
    w = np.exp(z)
    L = np.log(w.sum())
    log_p = z - L
    outside = legal.copy()
    outside[ids[used]] = False
    bare = not outside.any()
    mr = -np.inf if bare else x[outside].max()
    zr = (x[outside] - mr) / T
    Lr = -np.inf if bare else np.log(np.exp(zr).sum())
    log_s = -np.inf if bare else (mr - m) / T + Lr - L
    s = np.exp(log_s)
    a = np.where(used, log_p[np.where(used, ids, 0)], -np.inf)
    p = np.exp(a)
    if kind == "truncated":
        top = v.max()
        lq = (v - top) / T - np.log(np.exp((v - top) / T).sum()) if top > -np.inf else np.full(v.size, -np.inf)
        q, r = np.exp(lq), 0.0
    else:
        lq, q = v, np.exp(v)
        r = 0.0 if bare else max(1.0 - q.sum(), LEAST)
    Q = q.sum()
    with np.errstate(divide="ignore", invalid="ignore"):
        log_r = np.log(r)
        u, ur = a - lq, log_s - log_r
    if kind == "reverse":
        loss = _xlogy(p, u).sum() + (s * ur if r > 0 and s > 0 else 0.0)
    else:
        loss = _xlogy(q, -u).sum() + (r * -ur if r > 0 else 0.0)
    G, A, d = np.zeros(len(ids)), 0.0, np.zeros(V)  # d: T times the loss's gradient
    if np.isfinite(loss):
        if kind == "reverse":
            G = np.where(used, _xlogy(p, u - loss), 0.0)
            A = s * (ur - loss) if s > 0 else 0.0
        else:
            G = np.where(used, p * (Q + r) - q, 0.0)
            A = s * (Q + r) - r
        if not bare:
            d[outside] = np.exp(zr - Lr) * A
        d[ids[used]] = G[used]
    zbar = float((np.exp(log_p[legal]) * -z[legal]).sum())
    zbar_r = 0.0 if bare else float((np.exp(zr - Lr) * -zr).sum())
    return dict(status=OK, loss=loss, logprob=0.0 if t < 0 else log_p[t], slot_logprobs=a, slot_grads=G,
                stats=np.array([mr, Lr, A, s]), d=d, log_p=log_p, p=p, q=q, lq=lq, r=r, log_r=log_r, log_s=log_s,
                u=u, ur=ur, m=m, L=L, zbar=zbar, zbar_r=zbar_r, outside=outside)


def grad_row(row, ids, t, T, g, gl):
    """Gradient of g * loss + gl * logprob for a distill_row result, float64 [V], or None for a
    row that failed (its gradient is zero)."""
    if row["status"] != OK:
        return None
    d = g * row["d"]
    if t >= 0 and row["log_p"][t] > -np.inf:
        d = d - gl * np.exp(row["log_p"])
        d[t] += gl
    return d / T

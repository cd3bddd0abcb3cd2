"""Processing of logits in float64 with numpy, row by row: penalties for repeated tokens,
biases, masks.  Test infrastructure only."""
import numpy as np

from .scoring import INVALID, OK


def process_row(x, history, prompt, theta, presence, frequency, bias_ids, bias, legal):
    """x float64 [V]; history: the row's entries (ids outside [0, V) are padding), the first
    `prompt` of them its prompt; legal bool [V].  (status, result, size): size bounds the sum of
    the magnitudes of all intermediate results, for the tolerance of a binary32 computation."""
    V = x.size
    used = (bias_ids >= 0) & (bias_ids < V)
    if (not (np.isfinite(theta) and theta > 0 and np.isfinite(presence) and np.isfinite(frequency))
            or not 0 <= prompt <= len(history) or np.any(~(bias[used] < np.inf))):
        return INVALID, x.copy(), np.zeros(V)
    v, size = x.copy(), np.zeros(V)
    for t in np.unique(history[(history >= 0) & (history < V)]):
        n = int((history[prompt:] == t).sum())
        if v[t] == -np.inf:
            continue
        v[t] = v[t] / theta if v[t] > 0 else v[t] * theta
        size[t] += abs(v[t])
        take = frequency * n + (presence if n else 0.0)
        size[t] += abs(frequency * n) + abs(take)
        v[t] -= take
        size[t] += abs(v[t])
    for i in np.nonzero(used)[0]:
        t = bias_ids[i]
        v[t] = -np.inf if -np.inf in (v[t], bias[i]) else v[t] + bias[i]
        size[t] += abs(v[t]) if np.isfinite(v[t]) else 0.0
    v[~legal] = -np.inf
    return OK, v, size

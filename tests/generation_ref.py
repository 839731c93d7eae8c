"""Plain 64-bit references of the generation operators (no tests here)."""
import math

import numpy as np


def sample_reference(z, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """The definition of include/rlhead.h (rl_sample), row by row.  Returns tokens, logq, the
    support rows (lists of ids and log q) and the replayed flags, and for each draw how far its
    random number is from a border of the cumulative weights, relative to the total (a draw
    nearer than the sums' accuracy may take the neighbour), and the same for the set's border."""
    z = np.asarray(z, np.float64).copy()
    z[np.isnan(z) | (z == np.inf)] = -np.inf
    N, V = z.shape
    u = np.asarray(u, np.float64)
    K = u.shape[1]
    at = lambda a, r, d: d if a is None else float(a[r])  # noqa: E731
    tok, lq = np.full((N, K), -1), np.full((N, K), -np.inf)
    ids, slq, rep, margin = [], [], np.zeros(N, int), np.full(N, np.inf)
    for r in range(N):
        T, k, p, mp = at(temperature, r, 1.0), int(at(top_k, r, 0)), at(top_p, r, 1.0), at(min_p, r, 0.0)
        greedy = not T > 0 or not T < np.inf
        p, mp = (1.0 if math.isnan(p) else p), (0.0 if math.isnan(mp) else mp)
        k = k if 0 < k < V else V
        rep[r] = greedy or k < V or p < 1 or mp > 0
        M = z[r].max()
        if M == -np.inf:
            ids.append(np.zeros(0, int))
            slq.append(np.zeros(0))
            continue
        if greedy:
            S = np.array([int(np.argmax(z[r]))])
            q = np.zeros(1)
            c = np.ones(1)
        else:
            x = (z[r] - M) / T
            w = np.exp(x)
            S = np.flatnonzero(x >= math.log(min(max(mp, 2.0 ** -100), 1.0)))
            S = S[np.lexsort((S, -x[S]))][:k]
            if p < 1:
                c = np.cumsum(w[S])
                n = 1 + int(np.count_nonzero(c[:-1] < p * c[-1]))
                if len(S) > 1 and np.any(w[S] != 1.0):
                    margin[r] = np.min(np.abs(c - p * c[-1])) / c[-1]
                S = S[:n]
            S = np.sort(S)
            c = np.cumsum(w[S])
            q = x[S] - math.log(c[-1])
        d = np.minimum(np.searchsorted(c, u[r] * c[-1], side="right"), len(S) - 1)
        if len(S) > 1 and np.any(w[S] != 1.0):      # sums of ones are exact: no margin is needed
            margin[r] = min(margin[r], min(np.min(np.abs(c - t * c[-1])) for t in u[r]) / c[-1])
        tok[r], lq[r] = S[d], q[d]
        keep = np.arange(len(S)) if rep[r] else np.sort(d[1:])
        ids.append(S[keep])
        slq.append(q[keep])
    return dict(tokens=tok, logq=lq, ids=ids, support_logq=slq, replayed=rep, margin=margin)

"""The definition of include/rlhead.h (rl_verify) in 64 bits, request by request (no tests here)."""
import math

import numpy as np


class Side:
    """Distributions of rows: z [n, V] with temperatures, or support rows, by replayed; rows maps the step's rows."""

    def __init__(self, V, z=None, temp=None, rows_ids=None, rows_logq=None, replayed=None, rows=None):
        self.V, self.z, self.temp, self.ids, self.lq, self.rep, self.rows = V, z, temp, rows_ids, rows_logq, replayed, rows
        self.kept = {}

    def log_probs(self, t):
        """ln of the row's probabilities [V] (-inf: none)."""
        r = t if self.rows is None else int(self.rows[t])
        if r not in self.kept:
            self.kept[r] = self._row(r)
        return self.kept[r]

    def _row(self, r):
        out = np.full(self.V, -np.inf)
        n = len(self.ids) if self.z is None else len(self.z)
        if not 0 <= r < n:
            return out
        if self.ids is not None and (self.z is None or self.rep[r]):
            ids, lq = np.asarray(self.ids[r], int), np.asarray(self.lq[r], np.float64)
            ok = (ids >= 0) & (ids < self.V) & (lq < np.inf)
            out[ids[ok]] = lq[ok]
            return out
        z = np.asarray(self.z[r], np.float64).copy()
        z[np.isnan(z) | (z == np.inf)] = -np.inf
        M = z.max()
        if M == -np.inf:
            return out
        T = 1.0 if self.temp is None else float(self.temp[r])
        if not T > 0 or not T < np.inf:
            out[int(np.argmax(z))] = 0
            return out
        x = (z - M) / T
        return x - math.log(np.exp(x).sum())


def verify_reference(step, cu, u, u_next, target, draft, ctx=None):
    """tokens, logq, accepted, keep_lens, and each request's margin: how near (relative) a random number came to a border."""
    R, T, V = len(cu) - 1, len(step), target.V
    tokens, logq = np.full(T, -1), np.zeros(T)
    acc, keep, margin = np.zeros(R, int), np.zeros(R, int), np.full(R, np.inf)
    for r in range(R):
        c = 0 if ctx is None else int(ctx[r])
        keep[r] = c
        t0, t1 = int(cu[r]), int(cu[r + 1])
        if t0 < 0 or t1 < t0 or t1 > T or t0 == t1:
            continue
        t = t0
        while t + 1 < t1:
            x = int(step[t + 1])
            if not 0 <= x < V:
                break
            lp = target.log_probs(t)[x]
            lq = 0.0 if draft is None else draft.log_probs(t)[x]
            p, q = math.exp(lp), math.exp(lq)
            a = float(u[t]) * q
            if p > 0 or a > 0:
                margin[r] = min(margin[r], abs(a - p) / max(a, p))
            if not a < p:
                break
            tokens[t], logq[t] = x, lp
            t += 1
        acc[r] = t - t0
        keep[r] = c + acc[r] + 1
        lp = target.log_probs(t)
        p = np.exp(lp)
        left = p
        if t + 1 < t1:
            if draft is None:
                q = np.zeros(V)
                if 0 <= step[t + 1] < V:
                    q[int(step[t + 1])] = 1
            else:
                q = np.exp(draft.log_probs(t))
            over = np.maximum(p - q, 0)
            # (differences below the rounding of this reference are no borders: both sides call them equal)
            if over.sum() > 0:
                left = over
        if p.sum() == 0:
            logq[t] = -np.inf
            continue
        s = np.cumsum(left)
        y = min(int(np.searchsorted(s, float(u_next[r]) * s[-1], side="right")), V - 1)
        # a border matters as far as it is from the number, in units of the whole distribution
        d = np.abs(s - float(u_next[r]) * s[-1])
        d = d[left > 0]
        if len(d) > 1 or u_next[r] == 0:
            margin[r] = min(margin[r], float(d.min()) if u_next[r] > 0 else np.inf)
        tokens[t], logq[t] = y, lp[y]
    return dict(tokens=tokens, logq=logq, accepted=acc, keep_lens=keep, margin=margin)

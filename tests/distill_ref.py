"""The definition of include/rlhead.h (distillation) in 64 bits, a row at a time, with what an error of
the rest's sum does to the results (no tests here)."""
import numpy as np


def distill_reference(z, offsets, ids, logq, dloss, kind, tail, T, beta):
    """loss [N], grad [N, V], mass [N], and the bounds of their errors for a relative error of 1 in the
    rest's exponentials (first order): to be multiplied by that error."""
    z = np.asarray(z, np.float64)
    N, V = z.shape
    loss, mass, grad = np.zeros(N), np.zeros(N), np.zeros((N, V))
    e_loss, e_grad = np.zeros(N), np.zeros((N, V))
    T = float(np.float32(T))
    beta = float(np.float32(beta))
    with np.errstate(all="ignore"):
        for r in range(N):
            a, b = int(offsets[r]), int(offsets[r + 1])
            S, y = np.asarray(ids[a:b], int), np.asarray(logq[a:b], np.float64)
            S, y = S[y > -np.inf], y[y > -np.inf]
            if len(S) == 0:
                continue
            x = z[r] / T
            x = x - x.max()
            lP = x - np.log(np.exp(x).sum())
            P = np.exp(lP)
            out = np.ones(V, bool)
            out[S] = False
            P0 = P[out].sum()
            if tail:
                t, lt = np.exp(y), y
                if P0 > 0:
                    t0 = max(1 - t.sum(), 2.0 ** -20)
                    t, lt = np.append(t, t0), np.append(lt, np.log(t0))
                    p, lp = np.append(P[S], P0), np.append(lP[S], np.log(P0))
                else:
                    p, lp = P[S], lP[S]
            else:
                y = y / T
                lt = y - y.max()
                lt = lt - np.log(np.exp(lt).sum())
                t, p, lp = np.exp(lt), P[S], lP[S]
            zero = p == 0
            if kind == "forward":
                f, pg = np.where(t > 0, t * (lt - lp), 0), -t
            elif kind == "reverse":
                f = np.where(zero, 0, p * (lp - lt))
                pg = f
            else:
                lm = np.log(beta * t + (1 - beta) * p)
                pg = np.where(zero, 0, (1 - beta) * p * (lp - lm))
                f = np.where(t > 0, beta * t * (lt - lm), 0) + pg
            A = pg.sum()
            loss[r], mass[r] = f.sum(), P[S].sum()
            g0 = pg[-1] / P0 if tail and P0 > 0 else 0.0
            w = float(dloss[r]) / T
            d = P * (g0 - A)
            d[S] = pg[:len(S)] - P[S] * A
            if w != 0:
                grad[r] = w * d
            # d(rest) moves the loss by P0 (g0 - A); a gradient's parts each by at most themselves, and A by its terms' sizes
            e_loss[r] = P0 * abs(g0 - A)
            size = np.abs(pg).sum() + p.sum()
            part = P * (abs(g0) + size)
            part[S] = np.abs(pg[:len(S)]) + P[S] * (1 + size)
            e_grad[r] = abs(w) * part
    return dict(loss=loss, mass=mass, grad=grad, e_loss=e_loss, e_grad=e_grad, terms=None)


def rest_error(T, V, spread):
    """Relative error of an exponential of the rest and of their sum: ex2.approx 2^-22, two roundings of an argument up to
    `spread` / T log2(e) (2^-24 each, times ln 2), the factor's own 2^-24, and up to V / 1024 + 16 additions."""
    arg = min(spread / T * 1.4427, 130.0)
    return 2.0 ** -22 + 3 * 2.0 ** -24 * arg * 0.6932 + (V / 1024 + 16) * 2.0 ** -24

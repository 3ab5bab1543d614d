"""Plain float64 forms of sampling under filters, a row's record and distillation from it, row by
row and without the library: what the GPU tests compare with."""
import numpy as np


def places(x):
    """Tokens in the order of their place: larger first, equal ones by index."""
    return np.argsort(-x, kind="stable")


def whole_numbers(w):
    """Weights in units of 2^-60, so that sums are exact and equal weights add up to what they are."""
    return [int(round(v * 2.0 ** 60)) for v in w.tolist()]


def keep(x, T, k=0, p=1.0, m=0.0):
    """Which tokens of a row x (float64) the filters keep, and their weights (0 for the others)."""
    x = np.asarray(x, dtype=np.float64)
    order = places(x)
    order = order[x[order] > -np.inf]
    if T == 0:
        order = order[:1]
        w = np.ones(1)
    else:
        w = np.exp((x[order] - x[order[0]]) / T)
        n = len(order) if k == 0 else min(k, len(order))
        if p < 1:
            ints = whole_numbers(w[:n])
            num, den = float(p).as_integer_ratio()
            want, run = num * sum(ints), 0
            for i, v in enumerate(ints):
                run += v
                if run * den >= want:
                    n = i + 1
                    break
        # exp(z) >= m as z >= ln m: a z of -1e-40 is below ln 1, where its exp rounds to 1
        while n > 1 and m > 0 and (x[order[n - 1]] - x[order[0]]) / T < np.log(m):
            n -= 1
        order, w = order[:n], w[:n]
    kept = np.zeros(len(x))
    kept[order] = w
    mask = np.zeros(len(x), dtype=bool)
    mask[order] = True
    return mask, kept


def draw(kept, us):
    """The first tokens, by index, whose cumulative weight is above u times the whole."""
    at = np.flatnonzero(kept)
    run = np.array(whole_numbers(kept[at]), dtype=object).cumsum()
    tokens = []
    for u in us:
        num, den = float(u).as_integer_ratio()
        lo, hi = 0, len(at) - 1
        while lo < hi:
            mid = (lo + hi) // 2
            if run[mid] * den > num * run[-1]:
                hi = mid
            else:
                lo = mid + 1
        tokens.append(int(at[lo]))
    return tokens


def sample(x, T, us, k=0, p=1.0, m=0.0):
    mask, kept = keep(x, T, k, p, m)
    return draw(kept, us), kept / kept.sum(), mask


def record(x, K, T):
    x = np.asarray(x, dtype=np.float64)
    order = places(x)[:K]
    top = x.max()
    return x[order], order, top / T + np.log(np.exp((x - top) / T).sum())


def distill(x, ids, z, lse=None, T=1.0):
    """One row's loss and gradient."""
    x, z = np.asarray(x, dtype=np.float64) / T, np.asarray(z, dtype=np.float64) / T
    some = np.asarray(ids) >= 0
    ids, z = np.asarray(ids)[some], z[some]
    if not len(ids):
        return 0.0, np.zeros(len(x))
    assert len(set(ids.tolist())) == len(ids)
    top = x.max()
    log_s = x - top - np.log(np.exp(x - top).sum())
    if lse is None:
        log_p = z - z.max() - np.log(np.exp(z - z.max()).sum())
    else:
        log_p = z - float(lse)
    p = np.exp(log_p)
    loss = float(sum(a * (b - c) for a, b, c in zip(p, log_p, log_s[ids]) if a > 0))
    target, whole = np.zeros(len(x)), p.sum()
    target[ids] = p
    if lse is not None:
        rest = np.ones(len(x), dtype=bool)
        rest[ids] = False
        r, s = max(0.0, 1.0 - p.sum()), np.exp(log_s[rest]).sum()
        if s < 2.0 ** -126:  # none, and r is what a float32 log-sum-exp leaves over
            s = 0.0
            if r < 2.0 ** -17 + 2.0 ** -22 * abs(float(lse)):
                r = 0.0
        if r > 0:
            loss += r * (np.log(r) - np.log(s))
            target[rest] = r * np.exp(log_s[rest]) / s
            whole += r
    return loss, (whole * np.exp(log_s) - target) / T

"""The training operators' formulas in 64 bits (numpy), one row at a time, and how far fp32 results may lie from them.

Bounds.  An exponential 2^a is off by 2^-22 (the approximate instruction) and, through its argument's three roundings, by
|a| ln 2 times 3 2^-24, of itself.  A sum s of them passes at most 13 batches of 32 columns a thread at V = 201088 (or 200 at
2^20), ten merges of lanes and warps and eight of CTAs, each with one exponential and two additions; a term's weight times |a|
is at most log2 V <= 20 in the mean.  Together below 2^-17 of s: 20 ln 2 3 2^-24 = 2.5e-6 of arguments, 30 2^-24 = 1.8e-6 of
additions along a term's way, 2^-22 (1 + 3) = 1e-6 of exponentials that do not cancel out: 5.3e-6 < 2^-17 = 7.6e-6.
So with s the sum without the maximum: log(1 + s) is off by 2^-17 s / (1 + s) + 2^-22, relative to log(1 + s)
where that is small; p by 2^-16 of itself; a log-probability by 2^-17 min(1, s) + 2^-22 |l|.
"""
import numpy as np

EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a step, relative
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}  # what may be lost below the normal numbers


def row(z, T):
    """(p, log p, lse, H, s) of a row; s: the sum of the others relative to the maximum.  None: no distribution."""
    y = np.asarray(z, np.float64) / T
    if y.size == 0 or not np.any(y > -np.inf):
        return None
    at = int(np.argmax(y))
    e = np.exp(y - y[at])
    e[at] = 0.0
    s = float(e.sum())
    e[at] = 1.0
    ln = np.log1p(s)
    l = (y - y[at]) - ln
    p = e / (1.0 + s)
    with np.errstate(invalid="ignore"):
        H = -float(np.where(p > 0, p * l, 0.0).sum())
    return p, l, y[at] + ln, H, s


def comp(p, s, z, t):
    """1 - p of column t."""
    return s / (1.0 + s) if z[t] == np.max(z) else 1.0 - p[t]


def lp_tol(l, s):
    return 2.0 ** -17 * min(1.0, s) + 2.0 ** -22 * abs(l)


def logprob(z, t, T):
    """(l, lse, H) and their tolerances, of a row whose token may be outside it."""
    z = np.asarray(z, np.float64)
    if not 0 <= t < z.size:
        return (0.0, 0.0, 0.0), (0.0, 0.0, 0.0)
    r = row(z, T)
    if r is None:
        return (-np.inf, -np.inf, 0.0), (0.0, 0.0, 0.0)
    p, l, lse, H, s = r
    return (l[t], lse, H), (0.0 if l[t] == -np.inf else lp_tol(l[t], s),
                            2.0 ** -17 * min(1.0, s) + 2.0 ** -22 * (abs(lse) + abs(np.max(z)) / T), 2.0 ** -16 * H)


def spread(z, t, T, c, f, dt, p=None, l=None, H=None, s=None, ctol=0.0):
    """(gradient, tolerance) of c l(t) + f H over the row's columns: (c (1[v = t] - p) - f p (l + H)) / T.
    ctol: how far c may be off."""
    p_, l_, _, H_, s_ = row(z, T)
    p = p_ if p is None else p
    l = l_ if l is None else l
    H = H_ if H is None else H
    with np.errstate(invalid="ignore"):
        ent = np.where(p > 0, p * (l + H), 0.0)
    mag = np.where(p > 0, p * (np.where(p > 0, np.abs(l), 0.0) + abs(H)), 0.0)
    g = -c * p - f * ent
    one = comp(p, s_, z, t)
    g[t] = c * one - f * ent[t]
    tol = 2.0 ** -16 * (abs(c) * p + abs(f) * mag) + ctol * p
    tol[t] = 2.0 ** -16 * (abs(c) * one + abs(f) * mag[t]) + ctol * one
    g, tol = g / T, tol / T
    return g, tol + EPS[dt] * np.abs(g) * (1 + 2.0 ** -10) + TINY[dt]


def policy(z, t, T, old, adv, ref, lo, hi, kl, ent, w, dt):
    """(loss, l, H, gradient), tolerances."""
    z = np.asarray(z, np.float64)
    zero = np.zeros(z.size)
    if not 0 <= t < z.size or w == 0:
        return (0.0, 0.0, 0.0, zero), (0.0, 0.0, 0.0, zero)
    r = row(z, T)
    if r is None:
        return (0.0, -np.inf, 0.0, zero), (0.0, 0.0, 0.0, zero)
    p, l, lse, H, s = r
    dl = lp_tol(l[t], s) if l[t] > -np.inf else 0.0
    R = np.exp(l[t] - old)
    a, b = -adv * R, -adv * min(max(R, 1 - lo), 1 + hi)
    loss, c = max(a, b), a if a >= b else 0.0
    lt = abs(adv) * R * (dl + 2.0 ** -21)
    ct = lt
    if kl:
        k = np.expm1(ref - l[t])
        loss += kl * (k - (ref - l[t]))
        c -= kl * k
        ct += abs(kl) * ((k + 1) * dl + 2.0 ** -22 * abs(k))
        lt += abs(kl) * (abs(k) * dl + 2.0 ** -22 * (abs(k) + abs(ref - l[t])))
    loss -= ent * H
    lt += abs(ent) * 2.0 ** -16 * H + 2.0 ** -22 * abs(loss)
    g, gt = spread(z, t, T, w * c, -w * ent, dt, ctol=abs(w) * ct)
    return (w * loss, l[t], H, g), (abs(w) * lt, dl, 2.0 ** -16 * H, gt)


def preference(z, t, cu, T, ref, beta, eps, margin, average, w, dt):
    """(loss [pairs], L [nseq], gradient [rows, V]), tolerances, of whole arrays."""
    z = np.asarray(z, np.float64)
    rows, V = z.shape
    n = len(cu) - 1
    L, Lt, mine = np.zeros(n), np.zeros(n), []
    for q in range(n):
        a = min(max(cu[q], 0), rows)
        b = min(max(cu[q + 1], a), rows)
        m = []
        for r in range(a, b):
            if 0 <= t[r] < V and cu[0] <= r < cu[n] and row(z[r], T) is not None:
                (l, _, _), (tol, _, _) = logprob(z[r], t[r], T)
                L[q] += l
                Lt[q] += tol  # (0 for a token of probability 0)
                m.append(r)
        each = max(1, len(m)) if average else 1
        L[q], Lt[q] = L[q] / each, Lt[q] / each + (2.0 ** -24 * abs(L[q] / each) if L[q] > -np.inf else 0.0)
        mine.append((m, each))
    loss, lt = np.zeros(n // 2), np.zeros(n // 2)
    g, gt = np.zeros((rows, V)), np.zeros((rows, V))
    for i in range(n // 2):
        a, b = 2 * i, 2 * i + 1
        ra, rb = (ref[a], ref[b]) if ref is not None else (0.0, 0.0)
        h = beta * ((L[a] - ra) - (L[b] - rb)) - margin
        ht = abs(beta) * (Lt[a] + Lt[b]) + 2.0 ** -23 * abs(h)
        wi = 1.0 if w is None else w[i]
        if wi == 0:
            continue
        soft = ((1 - eps) * np.logaddexp(0, -h) if eps < 1 else 0.0) + (eps * np.logaddexp(0, h) if eps > 0 else 0.0)
        loss[i] = wi * soft
        with np.errstate(over="ignore"):
            sp, sn = 1 / (1 + np.exp(-h)), 1 / (1 + np.exp(h))
        if not np.isfinite(h):
            ht = 0.0
        lt[i] = abs(wi) * (((1 - eps) * sn + eps * sp) * ht + 2.0 ** -21 * soft)
        d = wi * beta * (eps * sp - (1 - eps) * sn)
        dt_ = abs(wi * beta) * (sp * sn * ht + 2.0 ** -21 * (eps * sp + (1 - eps) * sn))
        for q, sign in ((a, 1), (b, -1)):
            for r in mine[q][0]:
                g[r], gt[r] = spread(z[r], t[r], T, sign * d / mine[q][1], 0.0, dt, ctol=dt_ / mine[q][1])
    return (loss, L, g), (lt, Lt, gt)


def distill(z, vals, idx, rest, T, w, dt):
    """(loss, gradient), tolerances.  rest: None or the log of the others' weight."""
    z = np.asarray(z, np.float64)
    V = z.size
    zero = np.zeros(V)
    ok = (idx >= 0) & (idx < V)
    ids, u = idx[ok].astype(np.int64), vals[ok].astype(np.float64) / T
    r = row(z, T)
    if ids.size == 0 or w == 0 or r is None:
        return (0.0, zero), (0.0, zero)
    u = np.append(u, -np.inf if rest is None else rest)
    top = u.max()
    if top == -np.inf:
        return (0.0, zero), (0.0, zero)
    e = np.exp(u - top)
    q = e / e.sum()
    at = int(np.argmax(e))
    others = np.delete(e, at).sum()
    lq = (u - top) - np.log1p(others)
    p, l, lse, H, s = r
    qt = 2.0 ** -16 * q
    lt = 0.0
    loss = 0.0
    target, ttol = np.zeros(V), np.zeros(V)
    for i, v in enumerate(ids):
        if q[i] > 0:
            loss += q[i] * (lq[i] - l[v])
            if l[v] > -np.inf:
                lt += qt[i] * abs(lq[i] - l[v]) + q[i] * (lp_tol(l[v], s) + lp_tol(lq[i], others))
        target[v] += q[i]
        ttol[v] += qt[i]
    listed = np.zeros(V, bool)
    listed[ids] = True
    out = np.where(listed, 0.0, p)
    if q[-1] > 0:
        m, li = out.sum(), p[listed].sum()
        lm = -np.inf if m == 0 else -np.log1p(li / m) if m > li else np.log(m)
        loss += q[-1] * (lq[-1] - lm)
        if m > 0:
            lt += qt[-1] * abs(lq[-1] - lm) + q[-1] * (lp_tol(lm, min(s, li / m)) + lp_tol(lq[-1], others)
                                                       + 2.0 ** -17 * min(1.0, li / m))
            target += q[-1] * out / m
            ttol += 2.0 ** -16 * q[-1] * out / m
    g = p - target
    tol = 2.0 ** -16 * p + ttol
    # where both lie near 1 the kernel takes 1 - q and 1 - p, each to 2^-16 of itself
    for v in np.nonzero((p > 0.5) & (target > 0.5) & listed)[0]:
        if np.count_nonzero(ids == v) == 1:
            near = others / (1 + others) if at < ids.size and ids[at] == v else 1 - target[v]
            g[v] = near - comp(p, s, z, v)
            tol[v] = 2.0 ** -16 * (near + comp(p, s, z, v)) + 2.0 ** -23 * (0.0 if z[v] == z.max() and ids[at % ids.size] == v else 1.0)
    g, tol = w * g / T, abs(w) * tol / T
    return (w * loss, g), (abs(w) * (lt + 2.0 ** -22 * abs(loss)), tol + EPS[dt] * np.abs(g) * (1 + 2.0 ** -10) + TINY[dt])


def near(got, want, tol, what=""):
    """Whether got lies within tol of want everywhere (equal where either is not finite)."""
    got, want = (np.atleast_1d(np.asarray(x, np.float64)) for x in (got, want))
    tol = np.broadcast_to(np.asarray(tol, np.float64), want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN elsewhere"
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), what + ": infinities"
    if fin.any():
        d = np.abs(got[fin] - want[fin])
        bad = d > tol[fin]
        if bad.any():
            at = tuple(int(x[bad][0]) for x in np.nonzero(fin))
            raise AssertionError(f"{what}: {int(bad.sum())} of {d.size} too far; first at {at}: got {got[at]!r}, want "
                                 f"{want[at]!r}, tolerance {tol[at]!r}")

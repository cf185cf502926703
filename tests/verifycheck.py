"""Draft verification in 64 bits on the CPU, sequence by sequence: the rule of tail_verify and
tail_verify_logits, with the smallest margin of every decision, so that a test can tell a wrong
token from one whose uniform lies on a boundary (the kernels' weights carry 2^-36)."""
from __future__ import annotations

import numpy as np

EDGE = 1e-9  # relative margins below this decide nothing


def sampler_target(vals, idx, prm):
    """The tail's sampler over one row's sorted candidates: (probabilities, ids); None when every one is -inf."""
    v = np.asarray(vals, np.float64)
    if v[0] == -np.inf:
        return None, 1.0
    k = v.size
    top_k, top_p, temp = (float(t) for t in prm[:3])
    kk = int(top_k) if 1 <= top_k < k + 1 else k
    margin = 1.0
    if not temp > 0 or kk == 1:
        e = np.array([1.0])
    else:
        e = _exp(v[:kk], v[0], temp)
        if top_p < 1:
            c = np.cumsum(e)
            cut = np.abs(c / c[-1] - top_p)
            margin = float(cut[:-1].min()) if kk > 1 else 1.0
            e = e[: int(np.nonzero(c >= top_p * c[-1])[0][0]) + 1]
    return (e / e.sum(), np.asarray(idx[: e.size], np.int64)), margin


def softmax_target(logits, temp):
    z = np.asarray(logits, np.float64)
    m = z.max()
    if m == -np.inf:
        return None
    if not temp > 0:
        p = np.zeros(z.size)
        p[int(np.argmax(z))] = 1.0
    else:
        p = _exp(z, m, float(temp))
        p /= p.sum()
    return p, np.arange(z.size)


def _exp(z, m, temp):
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp((z - m) / temp)
    return np.where(z == m, 1.0, np.where(z == -np.inf, 0.0, np.nan_to_num(e)))


def settle(cu, drafts, accept, u, target, draft, rows, fill=-7):
    """tokens [rows] (``fill`` behind the last sequence), counts [nseq] and the smallest margin of each sequence.

    target(row) -> ((p, ids) or None, margin); draft(row, ids) -> q at ids, or None for certain drafts."""
    nseq = len(cu) - 1
    tokens = np.full(rows, fill, np.int32)
    counts = np.zeros(nseq, np.int32)
    margins = np.ones(nseq)
    for s in range(nseq):
        lo, hi = int(cu[s]), int(cu[s + 1])
        tokens[lo:hi] = -1
        for j in range(lo, hi):
            t, margin = target(j)
            margins[s] = min(margins[s], margin)
            r = None
            if j < hi - 1:
                if t is not None:
                    p, ids = t
                    x = int(drafts[j])
                    at = np.nonzero(ids == x)[0]
                    px = float(p[at[0]]) if at.size else 0.0
                    qx = draft(j, np.array([x]))
                    qx = 1.0 if qx is None else float(qx[0])
                    if px > 0:
                        margins[s] = min(margins[s], abs(float(accept[j]) * qx - px) / px)
                    if float(accept[j]) * qx < px:
                        tokens[j] = x
                        continue
                    q = draft(j, ids)
                    q = (ids == x).astype(np.float64) if q is None else q
                    rest = np.maximum(p - q, 0.0)
                    r = rest if rest.sum() > 0 else p
            elif t is not None:
                p, ids = t
                r = p
            counts[s] = j - lo + 1
            if t is not None:
                c = np.cumsum(r)
                hit = np.nonzero((c > float(u[j]) * c[-1]) & (r > 0))[0]
                tokens[j] = ids[hit[0] if hit.size else np.nonzero(r > 0)[0][-1]]
                if np.count_nonzero(r) > 1:
                    last = np.nonzero(r > 0)[0][-1]
                    margins[s] = min(margins[s], float(np.abs(c[:last] / c[-1] - float(u[j])).min()))
            break
    return tokens, counts, margins


def compare(tokens, counts, want, cu):
    """Every sequence away from its boundaries equals the 64-bit result; rows behind the last one are untouched.
    Returns the number of sequences compared."""
    wt, wc, margins = want
    n = 0
    for s in range(len(cu) - 1):
        if margins[s] < EDGE:
            continue
        lo, hi = int(cu[s]), int(cu[s + 1])
        assert counts[s] == wc[s], f"sequence {s}: count {counts[s]} != {wc[s]}"
        assert np.array_equal(tokens[lo:hi], wt[lo:hi]), f"sequence {s}: {tokens[lo:hi]} != {wt[lo:hi]}"
        n += 1
    assert np.array_equal(tokens[int(cu[-1]):], wt[int(cu[-1]):]), "rows behind the last sequence changed"
    return n

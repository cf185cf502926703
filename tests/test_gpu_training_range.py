"""The training operators over the whole range that they document, on the GPU against the 64-bit formulas of
tests/traincheck.py: rests and lists far apart, NaN in a list, temperatures whose inverse is large or small, sums of very
unlike terms."""
import math

import numpy as np
import pytest

from tests import traincheck as tc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import decode_sampling_tail_gb300 as dst  # noqa: E402
from tests.test_gpu_training import DEV, DT, INF, _dev, _lists, _logits, _np, f32  # noqa: E402


# ------------------------------------------------------------------ a rest that outweighs its list, or is nothing beside it

ABOVE = [-120.0, -30.0, 0.5, 5.0, 10.0, 17.0, 18.0, 20.0, 25.0, 40.0, 60.0, 69.0, 75.0, 85.0, 100.0, 130.0]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 60000])  # a CTA a row, and a cluster
@pytest.mark.parametrize("T", [1.0, f32(0.7)])
def test_distill_with_a_rest_far_from_its_list(V, dt, T):
    rng = np.random.default_rng(V)
    k, kinds = 12, 6
    rows = kinds * len(ABOVE)
    z = rng.standard_normal((rows, V)).astype(np.float32)
    idx = np.stack([rng.permutation(V)[:k] for _ in range(rows)]).astype(np.int32)
    vals = rng.standard_normal((rows, k)).astype(np.float32)
    for r in range(rows):
        kind = r % kinds
        if kind == 0:
            z[r, np.setdiff1d(np.arange(40), idx[r])[0]] = 24.0  # a student sure of a token outside the list
        if kind == 1:
            z[r, idx[r, 3]] = 24.0                               # of one in it
        if kind == 2:
            z[r] = 0.25                                          # of none
        if kind == 3:
            idx[r, :3], vals[r, :3] = -1, 30.0                   # the teacher's likely tokens are none of the student's
        if kind == 4:
            z[r, idx[r]] -= 20.0                                 # the student knows as little of the list
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    top = np.where(idx >= 0, vals, -INF).max(1).astype(np.float64) / T
    rest = (top + np.repeat(ABOVE, kinds)).astype(np.float32)
    w = rng.uniform(0.5, 2.0, rows).astype(np.float32)
    loss, g = (_np(x) for x in dst.distill_topk(_dev(z, DT[dt]), _dev(vals), _dev(idx), teacher_rest=_dev(rest),
                                                temperature=T, weight=_dev(w)))
    alone = _np(dst.distill_topk(_dev(z, DT[dt]), _dev(vals), _dev(idx), teacher_rest=_dev(rest), temperature=T,
                                 weight=_dev(w), grad=False)[0])
    for r in range(rows):
        v, tol = tc.distill(z[r], vals[r], idx[r], float(rest[r]), T, float(w[r]), dt)
        what = f"row {r} (student {r % kinds}, rest {ABOVE[r // kinds]} above the list)"
        tc.near(loss[r], v[0], tol[0], "loss of " + what)
        tc.near(alone[r], v[0], tol[0], "loss alone of " + what)
        tc.near(g[r], v[1], tol[1], "gradient of " + what)


# ------------------------------------------------------------------ extreme temperatures

EXTREME = [2.0 ** -60, 1e-6, 1e-3, 1e6, 2.0 ** 60]


def _extreme(dt, seed=6, V=700):
    rng = np.random.default_rng(seed)
    z = _logits(rng, 4, V, dt)
    z[3] = 1e30 * np.sign(z[3])  # logits / T beyond fp32
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    return rng, z, z.argmax(1).astype(np.int32)


def _lost(T, size=1.0):
    """What exponentials below the smallest normal number leave out of a gradient (2^-126, times at most 2^6 for the
    entropy's logarithm)."""
    return size * 2.0 ** -120 / T


def _distill_by_logarithms(z, vals, ids, rest, T):
    """(loss, gradient, target) of one row, its ids valid and different, by logarithms alone: what lies outside the list
    may have any probability.  The rest is taken from the list's maximum exactly before it is divided by T."""
    def lse(x):
        return x.max() + math.log(np.exp(x - x.max()).sum())
    z, v = z.astype(np.float64), vals.astype(np.float64)
    top = v.max()
    u = (v - top) / T
    if rest is not None:
        from fractions import Fraction
        u = np.append(u, float((Fraction(rest) * Fraction(T) - Fraction(top)) / Fraction(T)))
    lq = u - lse(u)
    y = (z - z.max()) / T
    l = y - lse(y)
    target = np.zeros(z.size)
    target[ids] = np.exp(lq[:len(ids)])
    loss = sum(math.exp(a) * (a - b) for a, b in zip(lq, l[ids]) if a > -700)
    if rest is not None:
        out = np.delete(l, ids)
        if lq[-1] > -700:
            loss += math.exp(lq[-1]) * (lq[-1] - lse(out))
        target[np.setdiff1d(np.arange(z.size), ids)] = np.exp(lq[-1] + (out - lse(out)))  # (out alone may be of 1e18)
    return loss, (np.exp(l) - target) / T, target


@pytest.mark.parametrize("T", EXTREME)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("above", [None, -3.0, 0.0, 0.5, 20.0])
def test_distill_at_extreme_temperatures(T, dt, above):
    rng, z, _ = _extreme(dt)
    z = z[:3]
    vals, idx, _ = _lists(rng, z, 9, "f32", False, 1.0)
    rs = None if above is None else (vals.max(1).astype(np.float64) / T + above).astype(np.float32)  # (its step may be > 1)
    loss, g = dst.distill_topk(_dev(z, DT[dt]), _dev(vals), _dev(idx), temperature=T,
                               teacher_rest=None if rs is None else _dev(rs))
    for r in range(3):
        want, grad, target = _distill_by_logarithms(z[r], vals[r], idx[r], None if rs is None else float(rs[r]), T)
        # the loss: differences of numbers of |t| / T and |z| / T, fewer than 8 roundings of 2^-24 each, and logarithms
        # of sums, 2^-16 each
        big = max(abs(vals[r]).max(), abs(z[r][np.isfinite(z[r])]).max()) / T
        if abs(want) < 1e37:
            tc.near(_np(loss)[r], want, 2.0 ** -20 * big + 2.0 ** -15, f"loss of row {r}")
        # the gradient: p and q by 2^-16 of themselves, q also by its rest's exponent (three roundings of the number)
        p = grad * T + target
        tol = (2.0 ** -16 * (p + target) + 2.0 ** -22 * (0.0 if rs is None else abs(above) + 1) * target) / T
        tc.near(_np(g)[r], grad, tol + tc.EPS[dt] * np.abs(grad) * (1 + 2.0 ** -10) + _lost(T), f"gradient of row {r}")


@pytest.mark.parametrize("T", EXTREME)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ent,kl", [(0.0, 0.0), (0.01, 0.05)])
def test_policy_at_extreme_temperatures(T, dt, ent, kl):
    rng, z, t = _extreme(dt)
    l = np.array([tc.logprob(z[r], t[r], T)[0][0] for r in range(4)])
    old, ref = (l - 0.1).astype(np.float32), (l + 0.3).astype(np.float32)
    adv = np.array([1.0, -1.0, 0.5, -2.0], np.float32)
    H = torch.empty(4, device=DEV)
    loss, lp, g = dst.policy_loss(_dev(z, DT[dt]), _dev(t), _dev(old), _dev(adv), ref_logprob=_dev(ref), temperature=T,
                                  kl_coef=kl, entropy_coef=ent, out_entropy=H)
    c = f32(0.2)
    for r in range(4):
        v, tol = tc.policy(z[r], t[r], T, float(old[r]), float(adv[r]), float(ref[r]), c, c, f32(kl), f32(ent), 1.0, dt)
        for name, a, b, e in zip(("loss", "l", "H", "gradient"), (loss, lp, H, g), v, tol):
            # (terms below 2^-126 count as 0)
            low = _lost(T, 4.0) if name == "gradient" else 2.0 ** -100
            tc.near(_np(a)[r], b, e + low, f"{name} of row {r}")


@pytest.mark.parametrize("T", EXTREME)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_at_extreme_temperatures(T, dt, average):
    rng, z, t = _extreme(dt)
    cu = np.array([0, 1, 4], np.int32)
    L = [tc.logprob(z[r], t[r], T)[0][0] for r in range(4)]
    ref = np.array([L[0] + 1, sum(L[1:]) / (3 if average else 1)], np.float32)
    loss, seq, g = dst.preference_loss(_dev(z, DT[dt]), _dev(t), _dev(cu), ref_logprob=_dev(ref), beta=0.5,
                                       average=average, temperature=T)
    (wl, wL, wg), (tl, tL, tg) = tc.preference(z, t, cu, T, ref, 0.5, 0.0, 0.0, average, None, dt)
    tc.near(_np(loss), wl, tl, "loss")
    tc.near(_np(seq), wL, tL + 4 * z.shape[1] * 2.0 ** -126, "L")  # (terms below 2^-126 count as 0)
    tc.near(_np(g), wg, tg + _lost(T), "gradient")


@pytest.mark.parametrize("V", [300, 60000])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_keeps_nan_of_a_list(V, rest):
    rng = np.random.default_rng(V)
    z = _logits(rng, 3, V, "f32")
    vals, idx, rs = _lists(rng, z, 9, "f32", rest, 1.0)
    args = dict(teacher_rest=_dev(rs) if rest else None)
    clean = dst.distill_topk(_dev(z), _dev(vals), _dev(idx), **args)
    vals[1, 4] = np.nan
    loss, g = dst.distill_topk(_dev(z), _dev(vals), _dev(idx), **args)
    assert torch.isnan(loss[1]) and torch.isnan(g[1]).all()  # its own row, and all of that
    assert torch.equal(loss[[0, 2]], clean[0][[0, 2]]) and torch.equal(g[[0, 2]], clean[1][[0, 2]])
    alone = dst.distill_topk(_dev(z), _dev(vals), _dev(idx), grad=False, **args)[0]
    assert torch.isnan(alone).tolist() == [False, True, False]


# ------------------------------------------------------------------ what a log-sum-exp keeps

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1.0, f32(0.7), 0.05, 1.3])
def test_lse_is_rounded_once(T, dt):
    # rows whose likely token is e^20 times the others: log(1 + s) adds less than 2^-28 of error, and what is left is the
    # rounding of lse itself, half a step
    rng = np.random.default_rng(5)
    rows, V = 400, 500
    z = rng.standard_normal((rows, V)).astype(np.float32) * min(1.0, T)
    at = rng.integers(0, V, rows).astype(np.int32)
    z[np.arange(rows), at] = rng.uniform(26 * max(1.0, T), 60, rows).astype(np.float32)
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    lse = _np(dst.token_logprobs(_dev(z, DT[dt]), _dev(at), T)[1])
    for r in range(rows):
        (_, want, _), _ = tc.logprob(z[r], at[r], T)
        tc.near(lse[r], want, 2.0 ** -24 * abs(want) * (1 + 2.0 ** -10) + 2.0 ** -28, f"lse of row {r}")


# ------------------------------------------------------------------ the gradient of likely tokens, forward and back

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [300, 60000])
@pytest.mark.parametrize("T", [1.0, f32(0.7), 0.05])
@pytest.mark.parametrize("with_entropy", [False, True])
def test_gradient_from_the_statistics(V, dt, T, with_entropy):
    # 1 - p from 1 / 2 down to 1e-11, and tokens that are not the likely one
    rng = np.random.default_rng(V)
    rows = 12
    z = rng.standard_normal((rows, V)).astype(np.float32) * min(1.0, 2 * T)
    t = rng.integers(0, V, rows).astype(np.int32)
    z[np.arange(rows), t] = T * (math.log(V) + np.linspace(0.0, 25.0, rows))
    z[3, :V // 3] = -INF
    z[3, t[3]] = 8.0
    t[1] = (t[1] + 1) % V
    t[6], t[7] = -1, V
    z[8] = -INF
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    zt = _dev(z, DT[dt])
    stats = torch.empty((rows, 2), device=DEV)
    lp, lse, H = dst.token_logprobs(zt, _dev(t), T, entropy=True, out_stats=stats)
    for r in range(rows):
        if 0 <= t[r] < V and r != 8:
            s = tc.row(z[r], T)[4]  # (of its V terms those below 2^-126, which fp32 does not hold, count as 0)
            tc.near(_np(stats[r]), [z[r].max(), math.log1p(s)],
                    [0.0, 2.0 ** -17 * min(1.0, s) + 2.0 ** -22 * math.log1p(s) + V * 2.0 ** -126], f"statistics of row {r}")
    assert stats[6].tolist() == [0, 0] and stats[7].tolist() == [0, 0] and stats[8].tolist() == [-INF, 0]
    a, b = rng.standard_normal(rows).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    a[9] = b[9] = 0
    more = dict(d_entropy=_dev(b), entropy=H) if with_entropy else {}
    g = dst.token_logprobs_grad(zt, _dev(t), None, _dev(a), T, stats=stats, **more)
    for r in range(rows):
        if r in (6, 7, 8, 9):
            assert torch.count_nonzero(g[r]).item() == 0
            continue
        want, tol = tc.spread(z[r], t[r], T, float(a[r]), float(b[r]) if with_entropy else 0.0, dt)
        tc.near(_np(g[r]), want, tol, f"gradient of row {r}")
    # a lse beside them is not read; in place the same
    nan = torch.full((rows,), math.nan, device=DEV)
    assert torch.equal(dst.token_logprobs_grad(zt, _dev(t), nan, _dev(a), T, stats=stats, **more), g)
    assert torch.equal(dst.token_logprobs_grad(zt, _dev(t), None, _dev(a), T, stats=stats, out_grad=zt, **more), g)
    for bad in (stats[:, 0], None):
        with pytest.raises(ValueError):
            dst.token_logprobs_grad(zt, _dev(t), None, _dev(a), T, stats=bad)
    with pytest.raises(dst.TailError):
        dst.token_logprobs(zt, _dev(t), T, out_logprob=stats.view(-1)[:rows], out_stats=stats)


@pytest.mark.parametrize("T", EXTREME)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_from_the_statistics_at_extreme_temperatures(T, dt):
    rng, z, t = _extreme(dt)
    t[1] = 5  # not the likely one
    stats = torch.empty((4, 2), device=DEV)
    H = dst.token_logprobs(_dev(z, DT[dt]), _dev(t), T, entropy=True, out_stats=stats)[2]
    a, b = rng.standard_normal(4).astype(np.float32), rng.standard_normal(4).astype(np.float32)
    g = dst.token_logprobs_grad(_dev(z, DT[dt]), _dev(t), None, _dev(a), T, stats=stats, d_entropy=_dev(b), entropy=H)
    for r in range(4):
        want, tol = tc.spread(z[r], t[r], T, float(a[r]), float(b[r]), dt)
        tc.near(_np(g[r]), want, tol + _lost(T, 4.0), f"gradient of row {r}")


# ------------------------------------------------------------------ sums of very unlike terms

@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_small_terms_reach_a_sum_that_began_large(dt):
    # 608 rows, a CTA of 512 threads each.  Every thread's first vectors hold five zeros a lane, everything behind them
    # exp(-15.25), just below half a step of the 4 that the zeros make: added one after another they leave no trace, and s
    # loses 9e-6 of itself.  Bound: a term passes 16 additions in its batch, 25 batches and 10 merges, each 2^-24, and the
    # logarithm's rounding.
    rows, V = 608, 201088
    n = 16 // DT[dt].itemsize  # columns a vector
    z = torch.full((V,), -15.25, device=DEV)
    full = 8 // n  # vectors of zeros; behind them a pair
    z[:512 * n * full] = 0
    z[512 * n * full:512 * n * (full + 1)].view(512, n)[:, :2] = 0
    zeros = int((z == 0).sum())
    assert zeros == 512 * 10
    want = -math.log(zeros + (V - zeros) * math.exp(-15.25))
    z = z.to(DT[dt]).expand(rows, V).contiguous()
    lp, lse, H = dst.token_logprobs(z, torch.zeros(rows, dtype=torch.int32, device=DEV), entropy=True)
    tol = 51 * 2.0 ** -24 + 2.0 ** -22 * abs(want)
    tc.near(_np(lp), np.full(rows, want), tol, "l")
    tc.near(_np(lse), np.full(rows, -want), tol, "lse")
    p = math.exp(-15.25 + want)
    entropy = -want + (V - zeros) * p * 15.25  # H = lse - sum p z
    tc.near(_np(H), np.full(rows, entropy), tol + 51 * 2.0 ** -24, "H")


# ------------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("grad", [True, False])
def test_rows_whose_wait_runs_out_are_nan(grad):
    rng = np.random.default_rng(1)
    rows, V = 5, 60000  # a cluster a row
    z = _logits(rng, rows, V, "bf16")
    vals, idx, rs = _lists(rng, z, 20, "f32", True, 1.0)
    zt, t = _dev(z, DT["bf16"]), _dev(np.array([7, -1, V - 1, 30, 9], np.int32))
    old, adv = torch.full((rows,), -9.0, device=DEV), torch.ones(rows, device=DEV)
    cu = torch.tensor([0, 2, rows], dtype=torch.int32, device=DEV)
    v, i, r = _dev(vals), _dev(idx), _dev(rs)

    def calls():
        out = [*dst.token_logprobs(zt, t, entropy=True), *dst.policy_loss(zt, t, old, adv, grad=grad),
               *dst.preference_loss(zt, t, cu, grad=grad), *dst.distill_topk(zt, v, i, teacher_rest=r, grad=grad)]
        return [x for x in out if x is not None]

    want, late = calls(), 0
    try:
        dst.set_training_wait_limit(0)
        got = [calls() for _ in range(100)]
        torch.cuda.synchronize()  # every launch has ended
    finally:
        dst.set_training_wait_limit(1_000_000_000)
    for one in got:
        for x, y in zip(one, want):
            assert ((x == y) | torch.isnan(x)).all()
            late += int(torch.isnan(x).any())
        assert one[0][1].item() == 0  # an ignored row waits for nobody
    assert late  # (about three outputs of four)
    assert all(torch.equal(x, y) for x, y in zip(calls(), want))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 60000])
@pytest.mark.parametrize("twice", ["others", "likely", "both"])
@pytest.mark.parametrize("with_rest", [False, True])
def test_distill_of_likely_tokens_from_lists_with_an_id_twice(V, dt, twice, with_rest):
    # student and teacher both sure of one token: the gradient there is a difference of 1 - q and 1 - p, down to 1e-9
    rng = np.random.default_rng(V)
    rows, k = 10, 40
    z = rng.standard_normal((rows, V)).astype(np.float32)
    idx = np.stack([rng.permutation(V)[:k] for _ in range(rows)]).astype(np.int32)
    vals = rng.standard_normal((rows, k)).astype(np.float32)
    z[np.arange(rows), idx[:, 5]] = math.log(V) + np.linspace(0.0, 21.0, rows)
    vals[:, 5] = math.log(k) + np.linspace(1.0, 21.0, rows)
    if twice != "likely":
        idx[:, 9] = idx[:, 30]
    if twice != "others":
        idx[:, 17], vals[:, 17] = idx[:, 5], vals[:, 5] - 0.5
    rest = np.linspace(1.0, -3.0, rows).astype(np.float32) if with_rest else None
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    loss, g = (_np(x) for x in dst.distill_topk(_dev(z, DT[dt]), _dev(vals), _dev(idx),
                                                teacher_rest=_dev(rest) if with_rest else None))
    for r in range(rows):
        v, tol = tc.distill(z[r], vals[r], idx[r], float(rest[r]) if with_rest else None, 1.0, 1.0, dt)
        tc.near(loss[r], v[0], tol[0], f"loss of row {r}")
        tc.near(g[r], v[1], tol[1], f"gradient of row {r}")



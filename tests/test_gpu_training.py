"""The training operators on the GPU against the 64-bit formulas of tests/traincheck.py, within its bounds."""
import math

import numpy as np
import pytest

from tests import traincheck as tc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import decode_sampling_tail_gb300 as dst  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf

# rows, columns: single ones, odd ones, rows inside 16-byte vectors, one CTA a row and several
SHAPES = [(1, 1), (3, 2), (5, 7), (4, 33), (6, 300), (9, 1001), (2, 50021), (400, 515), (700, 515), (1, 201088)]


def f32(x):
    return float(np.float32(x))  # as the library takes it


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _matrix(a, dt, pad=0, offset=0):
    """a [rows, V] on the device as rows of V + pad columns that start `offset` elements into their buffer."""
    rows, V = a.shape
    buf = torch.full((rows * (V + pad) + offset + 16,), 7.0, dtype=DT[dt], device=DEV)
    view = buf[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    view.copy_(_dev(a, DT[dt]))
    return view, buf


def _logits(rng, rows, V, dt, scale=2.5):
    z = (scale * rng.standard_normal((rows, V))).astype(np.float32)
    for r in range(rows):
        z[r, rng.integers(0, V, 3)] += rng.uniform(2, 7, 3).astype(np.float32)
    if rows > 2 and V > 4:
        z[2, : V // 3] = -INF
    return _np(_dev(z, DT[dt])).astype(np.float32)


def _tokens(rng, rows, V):
    t = rng.integers(0, V, rows).astype(np.int32)
    if rows > 3:
        t[1], t[3] = -1, V
    return t


def _rows(rng, rows):
    """The rows that are compared: all of a few, some of many."""
    return range(rows) if rows <= 12 else sorted(rng.choice(rows, 12, replace=False).tolist() + [0, 1, 2, 3, rows - 1])


def _check_rows(rng, want, got, names, rows):
    """want(r) gives (values, tolerances) of a row; got: arrays by name."""
    for r in _rows(rng, rows):
        values, tols = want(r)
        for name, v, tol, g in zip(names, values, tols, got):
            if g is not None:
                tc.near(g[r], v, tol, f"{name} of row {r}")


# ------------------------------------------------------------------ token log-probabilities

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("T,pad", [(1.0, 0), (f32(0.7), 3)])
def test_logprobs_and_their_gradient(rows, V, dt, T, pad):
    rng = np.random.default_rng(rows * 7 + V)
    z, t = _logits(rng, rows, V, dt), _tokens(rng, rows, V)
    zt, _ = _matrix(z, dt, pad, offset=pad)
    lp, lse, H = dst.token_logprobs(zt, _dev(t), T, entropy=True)
    _check_rows(rng, lambda r: tc.logprob(z[r], t[r], T), [_np(x) for x in (lp, lse, H)], ("l", "lse", "H"), rows)
    plain = dst.token_logprobs(zt, _dev(t), T)
    assert plain[2] is None and torch.allclose(plain[0], lp, rtol=1e-5, atol=1e-5)

    a, b = rng.standard_normal(rows).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    if rows > 4:
        a[4] = b[4] = 0.0
    for with_b in (False, True):
        out, whole = _matrix(np.full((rows, V), 3.0), dt, pad, offset=pad)
        kept = whole.clone()
        dst.token_logprobs_grad(zt, _dev(t), lse, _dev(a), T, d_entropy=_dev(b) if with_b else None,
                                entropy=H if with_b else None, out_grad=out)
        # between and around the rows nothing is written
        kept[pad:pad + rows * (V + pad)].view(rows, V + pad)[:, :V] = out
        assert torch.equal(kept, whole)
        lse_n, H_n = _np(lse), _np(H)

        def want(r):
            if not 0 <= t[r] < V or (a[r] == 0 and (not with_b or b[r] == 0)):
                return [np.zeros(V)], [np.zeros(V)]
            l = z[r].astype(np.float64) / T - lse_n[r]  # the formula on the given lse and H
            g, tol = tc.spread(z[r].astype(np.float64), t[r], T, float(a[r]), float(b[r]) if with_b else 0.0, dt,
                               p=np.exp(l), l=l, H=H_n[r])
            c, f = float(a[r]), float(b[r]) if with_b else 0.0
            one = -np.expm1(l[t[r]])
            ent = np.exp(l[t[r]]) * (l[t[r]] + H_n[r]) if l[t[r]] > -INF else 0.0
            g[t[r]] = (c * one - f * ent) / T
            tol[t[r]] = (2.0 ** -16 * (abs(c * one) + abs(f) * (abs(ent) + np.exp(l[t[r]]) * abs(H_n[r])))) / T \
                + tc.EPS[dt] * abs(g[t[r]]) * 1.001 + tc.TINY[dt]
            return [g], [tol]

        _check_rows(rng, want, [_np(out)], ("gradient",), rows)
    # in place: the parts of a row are written by themselves
    dst.token_logprobs_grad(zt, _dev(t), lse, _dev(a), T, d_entropy=_dev(b), entropy=H, out_grad=zt)
    assert torch.equal(zt, out)


# ------------------------------------------------------------------ policy loss

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("T,kl,ent,pad", [(1.0, 0.0, 0.0, 0), (f32(0.7), 0.05, 0.01, 5),
                                             (f32(1.3), 0.1, 0.0, 8)])
def test_policy(rows, V, dt, T, kl, ent, pad):
    rng = np.random.default_rng(rows + 3 * V)
    z, t = _logits(rng, rows, V, dt), _tokens(rng, rows, V)
    if rows > 2:
        t[2] = V - 1  # not of probability 0
    l = np.array([tc.logprob(z[r], t[r], T)[0][0] if r in set(_rows(np.random.default_rng(1), rows)) or rows < 20
                  else 0.0 for r in range(rows)])
    l = np.where(np.isfinite(l), l, -5.0)
    d = rng.choice([-0.6, -0.3, -0.1, 0.0, 0.1, 0.2, 0.5], rows)  # both sides of both borders, and the ratio 1
    old = (l - d).astype(np.float32)
    ref = (l + 0.4 * rng.standard_normal(rows)).astype(np.float32)
    adv, w = rng.standard_normal(rows).astype(np.float32), rng.uniform(0.2, 2, rows).astype(np.float32)
    if rows > 4:
        w[4] = 0.0
    zt, _ = _matrix(z, dt, pad)
    out, whole = _matrix(np.full((rows, V), 3.0), dt, pad)
    kept = whole.clone()
    H = torch.empty(rows, device=DEV)
    loss, lp, g = dst.policy_loss(zt, _dev(t), _dev(old), _dev(adv), ref_logprob=_dev(ref) if kl else None,
                                  temperature=T, clip_low=0.2, clip_high=0.3, kl_coef=kl, entropy_coef=ent,
                                  weight=_dev(w), out_entropy=H, out_grad=out)
    kept[:rows * (V + pad)].view(rows, V + pad)[:, :V] = out
    assert g is out and torch.equal(kept, whole)
    lo, hi = f32(0.2), f32(0.3)
    _check_rows(np.random.default_rng(1),
                lambda r: tc.policy(z[r], t[r], T, float(old[r]), float(adv[r]), float(ref[r]), lo, hi, f32(kl), f32(ent),
                                    float(w[r]), dt),
                [_np(x) for x in (loss, lp, H, g)], ("loss", "l", "H", "gradient"), rows)
    # the loss alone, and the gradient in place
    alone, lp2, none = dst.policy_loss(zt, _dev(t), _dev(old), _dev(adv), ref_logprob=_dev(ref) if kl else None,
                                       temperature=T, clip_low=0.2, clip_high=0.3, kl_coef=kl, entropy_coef=ent,
                                       weight=_dev(w), grad=False)
    assert none is None and torch.allclose(alone, loss, rtol=1e-4, atol=1e-5)
    args = dict(ref_logprob=_dev(ref) if kl else None, temperature=T, clip_low=0.2, clip_high=0.3, kl_coef=kl,
                entropy_coef=ent, weight=_dev(w), out_entropy=H)
    dst.policy_loss(zt, _dev(t), _dev(old), _dev(adv), out_grad=zt, **args)
    assert torch.equal(zt, out)


# ------------------------------------------------------------------ preference loss

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,V,pad", [([1, 1], 5, 0), ([3, 7, 0, 2], 300, 3), ([5, 0, 1, 9, 4, 4], 1001, 0),
                                        ([2, 3], 50021, 1), ([300, 280], 97, 0)])
@pytest.mark.parametrize("average,eps,margin,with_ref", [(False, 0.0, 0.0, True), (True, 0.1, 0.3, False),
                                                         (False, 1.0, -0.2, True)])
def test_preference(lens, V, pad, dt, average, eps, margin, with_ref):
    rng = np.random.default_rng(sum(lens) + V)
    before, behind = 2, 3  # rows of no sequence
    cu = (before + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    rows, n = int(cu[-1]) + behind, len(lens)
    z, t = _logits(rng, rows, V, dt), rng.integers(0, V, rows).astype(np.int32)
    t[rng.random(rows) < 0.2] = -1
    if rows > 4:
        z[3] = -INF  # counted for nothing
    z[0], z[-1] = np.nan, np.nan  # not read
    T, beta = f32(0.9), 2.0 if average else 0.1
    ref = (-np.array(lens) * (1.0 if average else 5.0) + rng.standard_normal(n)).astype(np.float32)
    if average:
        ref = (-5.0 + rng.standard_normal(n)).astype(np.float32)
    w = rng.uniform(0.5, 2.0, n // 2).astype(np.float32)
    if n > 2:
        w[1] = 0.0
    zt, _ = _matrix(z, dt, pad)
    out, whole = _matrix(np.full((rows, V), 3.0), dt, pad)
    kept = whole.clone()
    loss, L, g = dst.preference_loss(zt, _dev(t), _dev(cu), ref_logprob=_dev(ref) if with_ref else None, beta=beta,
                                     label_smoothing=eps, margin=margin, average=average, temperature=T, weight=_dev(w),
                                     out_grad=out)
    kept[:rows * (V + pad)].view(rows, V + pad)[:, :V] = out
    assert torch.equal(kept, whole)
    z[0], z[-1] = 0, 0
    (wl, wL, wg), (tl, tL, tg) = tc.preference(z, t, cu, T, ref if with_ref else None, f32(beta), f32(eps), f32(margin),
                                               average, w, dt)
    tc.near(_np(loss), wl, tl, "loss")
    tc.near(_np(L), wL, tL, "L")
    tc.near(_np(g), wg, tg, "gradient")
    alone = dst.preference_loss(zt, _dev(t), _dev(cu), ref_logprob=_dev(ref) if with_ref else None, beta=beta,
                                label_smoothing=eps, margin=margin, average=average, temperature=T, weight=_dev(w),
                                grad=False)
    assert alone[2] is None and torch.equal(alone[0], loss) and torch.equal(alone[1], L)
    dst.preference_loss(zt, _dev(t), _dev(cu), ref_logprob=_dev(ref) if with_ref else None, beta=beta,
                        label_smoothing=eps, margin=margin, average=average, temperature=T, weight=_dev(w), out_grad=zt)
    assert torch.equal(zt, out)


def test_preference_bounds_outside_the_rows_are_cut():
    rng = np.random.default_rng(8)
    z, t = _logits(rng, 6, 40, "f32"), rng.integers(0, 40, 6).astype(np.int32)
    cu = np.array([-3, 2, 90], np.int32)
    loss, L, g = dst.preference_loss(_dev(z), _dev(t), _dev(cu))
    (wl, wL, wg), (tl, tL, tg) = tc.preference(z, t, cu, 1.0, None, f32(0.1), 0.0, 0.0, 0, None, "f32")
    tc.near(_np(loss), wl, tl, "loss")
    tc.near(_np(L), wL, tL, "L")
    tc.near(_np(g), wg, tg, "gradient")


def test_no_rows_and_no_sequences():
    z = torch.zeros((0, 10), device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    f = torch.zeros(0, device=DEV)
    assert dst.token_logprobs(z, i)[0].shape == (0,) and dst.policy_loss(z, i, f, f)[2].shape == (0, 10)
    assert dst.distill_topk(z, z[:, :3], torch.zeros((0, 3), dtype=torch.int32, device=DEV))[0].shape == (0,)
    loss, L, g = dst.preference_loss(z, i, torch.zeros(3, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert abs(loss.item() - math.log(2)) < 1e-6 and L.tolist() == [0, 0]  # two empty sequences
    g = dst.preference_loss(torch.ones((2, 10), device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV),
                            torch.zeros(1, dtype=torch.int32, device=DEV))[2]
    assert torch.count_nonzero(g).item() == 0


# ------------------------------------------------------------------ distillation

def _lists(rng, z, k, vdt, rest, T, twice=False):
    rows, V = z.shape
    teacher = np.where(np.isfinite(z), z, -3.0) + 0.7 * rng.standard_normal(z.shape)
    idx = np.argsort(-teacher, 1, kind="stable")[:, :k].astype(np.int32)
    vals = _np(_dev(np.take_along_axis(teacher, idx.astype(np.int64), 1).astype(np.float32), DT[vdt])).astype(np.float32)
    others = teacher.copy()
    np.put_along_axis(others, idx.astype(np.int64), -INF, 1)
    with np.errstate(divide="ignore"):
        rs = np.log(np.exp(others / T).sum(1)).astype(np.float32) if rest else None
    if rows > 5:
        idx[3] = -1            # no entry
        idx[4, k // 2:] = V    # a short list
        if k > 1:
            vals[5, 1:] = -INF  # one entry has it all
    if twice and k > 3:
        idx[:, 2] = np.where(idx[:, 2] >= 0, idx[:, 0], idx[:, 2])
        idx[0, 3] = idx[0, 1]
    return vals, idx, rs


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V,k,pad", [(1, 1, 1, 0), (7, 5, 5, 0), (7, 300, 17, 3), (9, 1001, 256, 0),
                                          (8, 1200, 1024, 1), (7, 50021, 77, 0), (400, 515, 4, 0), (700, 515, 200, 0), (1, 201088, 256, 0)])
@pytest.mark.parametrize("rest,T,vdt,twice", [(False, 1.0, "f32", False), (True, f32(0.7), "f32", False),
                                              (True, f32(1.6), "bf16", True)])
def test_distill(rows, V, k, pad, dt, rest, T, vdt, twice):
    rng = np.random.default_rng(rows + V + k)
    z = _logits(rng, rows, V, dt)
    vals, idx, rs = _lists(rng, z, k, vdt, rest, T, twice)
    w = rng.uniform(0.5, 2.0, rows).astype(np.float32)
    if rows > 6:
        w[6] = 0.0
    zt, _ = _matrix(z, dt, pad)
    vt, _ = _matrix(vals, vdt, 2)
    it = torch.full((rows, k + 3), -1, dtype=torch.int32, device=DEV)[:, :k].copy_(_dev(idx))
    it = it if rows > 1 else it.contiguous()
    out, whole = _matrix(np.full((rows, V), 3.0), dt, pad)
    kept = whole.clone()
    args = dict(teacher_rest=None if rs is None else _dev(rs), temperature=T, weight=_dev(w))
    loss, g = dst.distill_topk(zt, vt, it, out_grad=out, **args)
    kept[:rows * (V + pad)].view(rows, V + pad)[:, :V] = out
    assert torch.equal(kept, whole)
    _check_rows(rng, lambda r: tc.distill(z[r], vals[r], idx[r], None if rs is None else float(rs[r]), T, float(w[r]),
                                          dt), [_np(loss), _np(g)], ("loss", "gradient"), rows)
    alone, none = dst.distill_topk(zt, vt, it, grad=False, **args)
    assert none is None and torch.allclose(alone, loss, rtol=1e-4, atol=1e-6)
    dst.distill_topk(zt, vt, it, out_grad=zt, **args)
    assert torch.equal(zt, out)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_more_rows_than_shared_memory_holds(dt):
    # rows that pass twice through L2 instead
    rng = np.random.default_rng(12)
    rows, V = 330, 50021
    z = np.tile(_logits(rng, 30, V, dt), (11, 1))
    z[:, 0] = rng.standard_normal(rows)
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    t = rng.integers(0, V, rows).astype(np.int32)
    t[2::30] = V - 1
    t[7::11] = -1
    f = np.float32
    old, adv = np.full(rows, -11.0, f), rng.standard_normal(rows).astype(f)
    zt = _dev(z, DT[dt])
    loss, lp, g = (_np(x) for x in dst.policy_loss(zt, _dev(t), _dev(old), _dev(adv)))
    c = f32(0.2)
    _check_rows(rng, lambda r: [x[:2] + x[3:] for x in tc.policy(z[r], t[r], 1.0, -11.0, float(adv[r]), 0.0, c, c, 0.0, 0.0,
                                                                1.0, dt)], (loss, lp, g), ("loss", "l", "gradient"), rows)
    vals, idx, rs = _lists(rng, z, 20, "f32", True, 1.0)
    loss, g = (_np(x) for x in dst.distill_topk(zt, _dev(vals), _dev(idx), teacher_rest=_dev(rs)))
    _check_rows(rng, lambda r: tc.distill(z[r], vals[r], idx[r], float(rs[r]), 1.0, 1.0, dt), (loss, g),
                ("loss", "gradient"), rows)


# ------------------------------------------------------------------ rows that go wrong

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [100, 5003])
def test_masked_and_extreme_rows(dt, V):
    rng = np.random.default_rng(V)
    z = _logits(rng, 9, V, dt)
    low = float(torch.finfo(DT[dt]).min)
    z[0] = -INF                       # no distribution
    z[1], z[1, V // 2] = -INF, 1.5    # one column left
    z[2], z[2, 7] = low, 3.0          # masked by the type's lowest value
    z[3] = low                        # every column at it: uniform
    z[4, 3] = np.nan                  # its own row alone
    z[5] = 2.0                        # ties
    z[6, 11] = 60.0                   # one likely token
    z[7, 1:] = -INF
    t = np.array([3, V // 2, 7, 5, 9, 50, 11, 1, 20], np.int32)
    zt = _dev(z, DT[dt])
    got = [_np(x) for x in dst.token_logprobs(zt, _dev(t), 1.0, entropy=True)]
    f = np.float32
    old, adv, w = np.full(9, -2.0, f), rng.standard_normal(9).astype(f), np.ones(9, f)
    loss, lp, g = (_np(x) for x in dst.policy_loss(zt, _dev(t), _dev(old), _dev(adv), clip_low=0.5, entropy_coef=0.01))
    vals, idx = rng.standard_normal((9, 6)).astype(f), np.stack([rng.permutation(V)[:6] for _ in range(9)]).astype(np.int32)
    idx[6, 0], vals[6, 0] = 11, 50.0
    idx[7, 0] = 0
    vals[2, 5] = np.nan
    idx[2, 5] = -1
    dl, dg = (_np(x) for x in dst.distill_topk(zt, _dev(vals), _dev(idx), teacher_rest=_dev(np.zeros(9, f))))
    for r in range(9):
        if r == 4:
            assert all(np.isnan(x[r]) for x in (*got, loss, lp, dl)) and np.isnan(g[r]).all()
            continue
        v, tol = tc.logprob(z[r], t[r], 1.0)
        for a, b, c in zip(got, v, tol):
            tc.near(a[r], b, c, f"row {r}")
        v, tol = tc.policy(z[r], t[r], 1.0, -2.0, float(adv[r]), 0.0, 0.5, f32(0.2), 0.0, f32(0.01), 1.0, dt)
        tc.near(loss[r], v[0], tol[0], f"policy loss of row {r}")
        tc.near(g[r], v[3], tol[3], f"policy gradient of row {r}")
        v, tol = tc.distill(z[r], vals[r], idx[r], 0.0, 1.0, 1.0, dt)
        tc.near(dl[r], v[0], tol[0], f"distillation loss of row {r}")
        tc.near(dg[r], v[1], tol[1], f"distillation gradient of row {r}")
    assert abs(got[0][6] / tc.logprob(z[6], 11, 1.0)[0][0] - 1) < 2.0 ** -15  # log(1 - 1e-20) and the like keep their bits


@pytest.mark.parametrize("T", [2.0 ** -60, 1e-6, 1e6, 2.0 ** 60])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_extreme_temperatures(T, dt):
    rng = np.random.default_rng(6)
    V = 700
    z = _logits(rng, 4, V, dt)
    z[3] = 1e30 * np.sign(z[3])  # logits / T beyond fp32
    z = _np(_dev(z, DT[dt])).astype(np.float32)
    t = np.array([int(z[0].argmax()), 5, V - 1, int(z[3].argmax())], np.int32)
    zt = _dev(z, DT[dt])
    got = [_np(x) for x in dst.token_logprobs(zt, _dev(t), T, entropy=True)]
    f = np.float32
    vals, idx, rs = _lists(rng, z[:3], 9, "f32", False, 1.0)
    dl, dg = (_np(x) for x in dst.distill_topk(zt[:3], _dev(vals), _dev(idx), temperature=T))
    old = np.where(got[0] > -1e30, got[0], 0.0).astype(f)
    loss, lp, g = (_np(x) for x in dst.policy_loss(zt, _dev(t), _dev(old), _dev(np.ones(4, f)), temperature=T,
                                                   out_entropy=torch.empty(4, device=DEV)))
    assert np.isfinite(g).all() and np.isfinite(dg).all() and np.isfinite(got[2]).all()
    for r in range(4):
        (l, lse, H), (tl, ts, tH) = tc.logprob(z[r].astype(np.float64), t[r], T)
        if abs(l) < 1e37:
            tc.near(got[0][r], l, tl, f"l of row {r}")
        else:
            assert got[0][r] == -INF or abs(got[0][r] / l - 1) < 1e-6
        tc.near(got[2][r], H, tH + 1e-30, f"H of row {r}")
        if abs(lse) < 1e37:
            tc.near(got[1][r], lse, ts, f"lse of row {r}")
    for r in range(3):
        v, tol = tc.distill(z[r], vals[r], idx[r], None, T, 1.0, dt)
        if abs(v[0]) < 1e37:
            # its terms are differences of numbers of |t| / T, rounded a few times each
            tc.near(dl[r], v[0], tol[0] + 2.0 ** -20 * abs(vals[r]).max() / T, f"distillation loss of row {r}")


def test_tokens_of_probability_zero():
    z = torch.zeros((3, 50), device=DEV)
    z[:, :20] = -INF
    t = torch.tensor([3, 3, 30], dtype=torch.int32, device=DEV)
    old, adv = torch.full((3,), -4.0, device=DEV), torch.tensor([1.0, -1.0, 1.0], device=DEV)
    lp, lse, _ = dst.token_logprobs(z, t)
    assert lp.tolist()[:2] == [-INF, -INF] and abs(lp[2].item() + math.log(30)) < 1e-5
    loss, _, g = dst.policy_loss(z, t, old, adv)  # the ratio is 0: nothing to gain, or the clipped loss; no slope
    assert loss.tolist()[0] == 0 and abs(loss[1].item() - 0.8) < 1e-6 and torch.count_nonzero(g[:2]).item() == 0
    loss, _, g = dst.policy_loss(z, t, old, adv, ref_logprob=old, kl_coef=0.1)
    assert loss.tolist()[:2] == [INF, INF] and torch.isfinite(g[2]).all()
    cu = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    loss, L, g = dst.preference_loss(z, t, cu)
    assert L[0].item() == -INF and math.isnan(loss[0].item())  # -inf less -inf
    loss, L, g = dst.preference_loss(z[1:], t[1:], torch.arange(3, dtype=torch.int32, device=DEV))
    assert loss[0].item() == INF and abs(g[0, 3].item() + 0.1) < 1e-6 and torch.isfinite(g).all()


def test_ignored_rows_are_not_read():
    z = torch.full((4, 1000), math.nan, device=DEV)
    t = torch.tensor([-1, 1000, -7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    nan = torch.full((4,), math.nan, device=DEV)
    assert all(torch.equal(x, torch.zeros(4, device=DEV)) for x in dst.token_logprobs(z, t, entropy=True))
    zero = torch.zeros_like(z)
    assert torch.equal(dst.token_logprobs_grad(z, t, nan, nan), zero)
    loss, lp, g = dst.policy_loss(z, t, nan, nan, ref_logprob=nan, kl_coef=0.1)
    assert torch.equal(loss, zero[:, 0]) and torch.equal(lp, zero[:, 0]) and torch.equal(g, zero)
    loss, g = dst.distill_topk(z, z[:, :1].contiguous(), t[:, None].contiguous(), teacher_rest=nan)
    assert torch.equal(loss, zero[:, 0]) and torch.equal(g, zero)


@pytest.mark.parametrize("V", [300, 60000])
def test_distill_from_lists_of_minus_infinity(V):
    z = torch.randn((4, V), generator=torch.Generator(device=DEV).manual_seed(9), device=DEV)
    z[0, 9], z[1, 10] = math.nan, INF
    idx = torch.arange(3, dtype=torch.int32, device=DEV).repeat(4, 1) * 7
    vals = torch.full((4, 3), -INF, device=DEV)
    for rest in (None, torch.full((4,), -INF, device=DEV)):  # nothing to aim at: ignored, whatever the logits hold
        loss, g = dst.distill_topk(z, vals, idx, teacher_rest=rest)
        assert torch.equal(loss, torch.zeros(4, device=DEV)) and torch.equal(g, torch.zeros_like(z))
    rest = torch.tensor([0.0, 0.0, math.nan, 0.0], device=DEV)
    vals[1] = 1.0
    loss, g = dst.distill_topk(z, vals, idx, teacher_rest=rest)
    assert torch.isnan(loss[[0, 2]]).all() and torch.isnan(g[[0, 2]]).all()
    v, tol = tc.distill(_np(z[3]), _np(vals[3]).astype(np.float32), idx[3].cpu().numpy(), 0.0, 1.0, 1.0, "f32")
    tc.near(_np(loss[3]), v[0], tol[0], "loss")
    tc.near(_np(g[3]), v[1], tol[1], "gradient")


@pytest.mark.parametrize("terms", [dict(), dict(entropy_coef=0.01), dict(kl_coef=0.1)])
def test_policy_keeps_nan_and_takes_nothing_of_an_advantage_of_0(terms):
    z = torch.zeros((6, 300), device=DEV)
    z[0, 7] = math.nan
    t = torch.full((6,), 5, dtype=torch.int32, device=DEV)
    l = -math.log(300)
    old = torch.full((6,), l, device=DEV)
    adv = torch.ones(6, device=DEV)
    old[1], adv[2] = math.nan, math.nan  # their rows' losses, without a term that has one of itself too
    old[3], adv[3] = -200.0, 0.0         # a ratio behind fp32's range, times nothing
    adv[4] = 0.0
    for hi in (0.2, INF):
        loss, lp, g = dst.policy_loss(z, t, old, adv, ref_logprob=torch.full((6,), l, device=DEV), clip_high=hi, **terms)
        assert torch.isnan(loss[:3]).all() and torch.isnan(g[:3]).all()
        assert math.isnan(lp[0].item()) and torch.isfinite(lp[1:]).all()
        assert torch.isfinite(loss[3:]).all() and torch.isfinite(g[3:]).all()
        want = terms.get("entropy_coef", 0.0) * l  # -coef H
        assert (loss[3:5] - want).abs().max().item() < 1e-6 and abs(loss[5].item() - (want - 1)) < 1e-5


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_longer_than_shared_memory(dt):
    # 2^20 columns: a part of a row that its CTA does not hold is read twice
    rng = np.random.default_rng(3)
    V = 1 << 20
    z = _logits(rng, 2, V, dt)
    t = np.array([V - 1, 17], np.int32)
    zt = _dev(z, DT[dt])
    f = np.float32
    old, adv = np.array([-14.0, -13.0], f), np.array([1.0, -1.0], f)
    loss, lp, g = (_np(x) for x in dst.policy_loss(zt, _dev(t), _dev(old), _dev(adv)))
    vals, idx, rs = _lists(rng, z, 1000, "f32", True, 1.0)
    dl, dg = (_np(x) for x in dst.distill_topk(zt, _dev(vals), _dev(idx), teacher_rest=_dev(rs)))
    c = f32(0.2)
    for r in range(2):
        v, tol = tc.policy(z[r], t[r], 1.0, float(old[r]), float(adv[r]), 0.0, c, c, 0.0, 0.0, 1.0, dt)
        for a, b, e in zip((loss, lp, g), (v[0], v[1], v[3]), (tol[0], tol[1], tol[3])):
            tc.near(a[r], b, e, f"row {r}")
        v, tol = tc.distill(z[r], vals[r], idx[r], float(rs[r]), 1.0, 1.0, dt)
        tc.near(dl[r], v[0], tol[0], f"loss of row {r}")
        tc.near(dg[r], v[1], tol[1], f"gradient of row {r}")
    with pytest.raises(dst.TailError):
        dst.token_logprobs(torch.zeros((1, V + 1), device=DEV), _dev(t[:1]))


@pytest.mark.parametrize("V", [8 * 8 * 12416, 8 * 8 * 12417, 811000])
def test_distill_parts_that_just_fill_shared_memory(V):
    # the longest part beside the longest list that is kept, the shortest that is not, and between
    rng = np.random.default_rng(13)
    z = _logits(rng, 2, V, "bf16")
    vals, idx, rs = _lists(rng, z, 1024, "f32", True, 1.0)
    loss, g = (_np(x) for x in dst.distill_topk(_dev(z, DT["bf16"]), _dev(vals), _dev(idx), teacher_rest=_dev(rs)))
    for r in range(2):
        v, tol = tc.distill(z[r], vals[r], idx[r], float(rs[r]), 1.0, 1.0, "bf16")
        tc.near(loss[r], v[0], tol[0], f"loss of row {r}")
        tc.near(g[r], v[1], tol[1], f"gradient of row {r}")


def test_many_short_rows():
    g = torch.Generator(device=DEV).manual_seed(4)
    rows, V = 70001, 37
    z = 3 * torch.randn((rows, V), generator=g, device=DEV)
    t = torch.randint(-1, V, (rows,), generator=g, device=DEV, dtype=torch.int32)
    old, adv = torch.full((rows,), -3.0, device=DEV), torch.randn(rows, generator=g, device=DEV)
    loss, lp, grad = dst.policy_loss(z, t, old, adv)
    l = torch.log_softmax(z.double(), -1)
    live = t >= 0
    want = torch.where(live, l.gather(1, t.clamp(min=0).long()[:, None])[:, 0], 0.0)
    assert (lp.double() - want).abs().max().item() < 2.0 ** -17 + 2.0 ** -22 * 30
    R = torch.exp(want + 3.0)
    c = torch.where(live & (-adv * R >= -adv * R.clamp(1 - f32(0.2), 1 + f32(0.2))), -adv * R, 0.0)
    one = torch.zeros_like(l).scatter_(1, t.clamp(min=0).long()[:, None], 1.0)
    exact = c[:, None] * (one - l.exp())
    near = ((R - 1 + f32(0.2)).abs() > 1e-4) & ((R - 1 - f32(0.2)).abs() > 1e-4)  # the slope jumps at the clip's borders
    # of c 2^-16 (l's error, R's) and of p 2^-16
    assert ((grad.double() - exact).abs() <= 2.0 ** -15 * c.abs()[:, None] + 1e-30)[near].all()
    vals, idx = z.topk(5, dim=-1)
    kl, d = dst.distill_topk(z, vals, idx.to(torch.int32), temperature=2.0)
    q = torch.softmax(vals.double() / 2, -1)
    p = torch.softmax(z.double() / 2, -1)
    exact = (p - torch.zeros_like(p).scatter_(1, idx, q)) / 2
    assert (d.double() - exact).abs().max().item() < 2.0 ** -16
    assert (kl.double() - (q * (q.log() - p.gather(1, idx).log())).sum(-1)).abs().max().item() < 2.0 ** -15


def test_offsets_behind_32_bits():
    rng = np.random.default_rng(9)
    rows, V, ld = 3, 1000, 3 << 29  # rows of 3 GB each apart in 16 bits
    z = _logits(rng, rows, V, "bf16")
    buf = torch.zeros(2 * ld + V, dtype=torch.bfloat16, device=DEV)
    zt = torch.as_strided(buf, (rows, V), (ld, 1))
    zt.copy_(_dev(z, torch.bfloat16))
    t = _dev(np.array([1, 2, 3], np.int32))
    near = zt.contiguous()
    f = torch.ones(rows, device=DEV)
    old = torch.full((rows,), -3.0, device=DEV)
    a, b = dst.policy_loss(zt, t, old, f), dst.policy_loss(near, t, old, f)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    vals, idx, _ = _lists(rng, z, 9, "f32", False, 1.0)
    a, b = (dst.distill_topk(x, _dev(vals), _dev(idx)) for x in (zt, near))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    lse = dst.token_logprobs(zt, t)[1]
    a = dst.token_logprobs_grad(zt, t, lse, f, out_grad=zt)
    assert torch.equal(a, dst.token_logprobs_grad(near, t, lse, f)) and torch.count_nonzero(buf[V:ld]).item() == 0


@pytest.mark.parametrize("shift", [1, 4])
@pytest.mark.parametrize("V", [1003, 40000])
def test_gradients_that_lie_otherwise_than_their_logits(shift, V):
    rng = np.random.default_rng(V)
    z, t = _logits(rng, 5, V, "bf16"), _tokens(rng, 5, V)
    zt, _ = _matrix(z, "bf16")
    apart, whole = _matrix(np.full((5, V), 3.0), "bf16", 2, offset=shift)
    kept = whole.clone()
    f, old = torch.ones(5, device=DEV), torch.full((5,), -6.0, device=DEV)
    a = dst.policy_loss(zt, _dev(t), old, f, entropy_coef=0.1)[2]
    dst.policy_loss(zt, _dev(t), old, f, entropy_coef=0.1, out_grad=apart)
    assert torch.equal(a, apart)
    kept[shift:shift + 5 * (V + 2)].view(5, V + 2)[:, :V] = a
    assert torch.equal(kept, whole)
    vals, idx, rs = _lists(rng, z, 30, "f32", True, 1.0)
    a = dst.distill_topk(zt, _dev(vals), _dev(idx), teacher_rest=_dev(rs))[1]
    assert torch.equal(a, dst.distill_topk(zt, _dev(vals), _dev(idx), teacher_rest=_dev(rs), out_grad=apart)[1])


def test_rows_interleaved_with_their_gradient():
    rng = np.random.default_rng(2)
    both = torch.zeros((6, 2 * 256), dtype=torch.bfloat16, device=DEV)
    z, t = _logits(rng, 6, 256, "bf16"), rng.integers(0, 256, 6).astype(np.int32)
    both[:, :256] = _dev(z, torch.bfloat16)
    f, old = torch.ones(6, device=DEV), torch.full((6,), -4.0, device=DEV)
    want = dst.policy_loss(both[:, :256].contiguous(), _dev(t), old, f)[2]
    dst.policy_loss(both[:, :256], _dev(t), old, f, out_grad=both[:, 256:])
    assert torch.equal(both[:, 256:], want)
    with pytest.raises(dst.TailError):
        dst.policy_loss(both[:, :256], _dev(t), old, f, out_grad=both[:, 128:384])


# ------------------------------------------------------------------ arguments

def test_wrappers_check_their_tensors():
    z = torch.zeros((4, 10), device=DEV)
    i, f = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, device=DEV)
    for call in (lambda: dst.token_logprobs(z.double(), i), lambda: dst.token_logprobs(z, i.long()),
                 lambda: dst.token_logprobs(z.t(), i), lambda: dst.token_logprobs(z, i[:3]),
                 lambda: dst.token_logprobs(z[:1].expand(4, 10), i),
                 lambda: dst.policy_loss(z, i, f, f[:2]), lambda: dst.policy_loss(z, i, f, f.double()),
                 lambda: dst.policy_loss(z, i, f, f, out_grad=z.half()),
                 lambda: dst.policy_loss(z, i, f, f, out_grad=z[:, :9]),
                 lambda: dst.policy_loss(z, i, f, f, weight=f[::2]),
                 lambda: dst.preference_loss(z, i, i[:2]), lambda: dst.preference_loss(z, i, i[:3], ref_logprob=f),
                 lambda: dst.preference_loss(z, i, i[:3], workspace=f),
                 lambda: dst.distill_topk(z, z[:, :3], i[:, None].expand(4, 3)),
                 lambda: dst.distill_topk(z, z[:, :3], torch.zeros((4, 2), dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dst.token_logprobs(z, i, 0.0), lambda: dst.policy_loss(z, i, f, f, kl_coef=0.1),
                 lambda: dst.policy_loss(z, i, f, f, clip_low=2.0), lambda: dst.policy_loss(z, i, f, f, out_loss=f),
                 lambda: dst.token_logprobs_grad(z, i, f, f, d_entropy=f),
                 lambda: dst.preference_loss(z, i, i[:3], workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
                 lambda: dst.distill_topk(torch.zeros((1, 2000), device=DEV), torch.zeros((1, 1500), device=DEV),
                                          torch.zeros((1, 1500), dtype=torch.int32, device=DEV))):
        with pytest.raises(dst.TailError):
            call()


# ------------------------------------------------------------------ streams, graphs, runs together

def _everything(z, t, cu, old, adv, vals, idx, outs, stream=None):
    dst.token_logprobs(z, t, entropy=True, out_logprob=outs["lp"], out_lse=outs["lse"], out_entropy=outs["H"],
                       stream=stream)
    dst.token_logprobs_grad(z, t, outs["lse"], adv, out_grad=outs["g0"], stream=stream)
    dst.policy_loss(z, t, old, adv, out_loss=outs["l1"], out_logprob=outs["lp1"], out_grad=outs["g1"], stream=stream)
    dst.preference_loss(z, t, cu, out_loss=outs["l2"], out_seq_logprob=outs["L2"], out_grad=outs["g2"],
                        workspace=outs["ws"], stream=stream)
    dst.distill_topk(z, vals, idx, out_loss=outs["l3"], out_grad=outs["g3"], stream=stream)


def _outs(rows, V, nseq, dtype):
    e = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    o = dict(lp=e(rows), lse=e(rows), H=e(rows), l1=e(rows), lp1=e(rows), l2=e(nseq // 2), L2=e(nseq), l3=e(rows),
             ws=torch.zeros(dst.preference_loss_workspace(rows), dtype=torch.uint8, device=DEV))
    o.update({n: torch.zeros((rows, V), dtype=dtype, device=DEV) for n in ("g0", "g1", "g2", "g3")})
    return o


def _inputs(seed, rows, V):
    rng = np.random.default_rng(seed)
    z = _logits(rng, rows, V, "bf16")
    vals, idx, _ = _lists(rng, z, 16, "f32", False, 1.0)
    return [_dev(z, torch.bfloat16), _dev(rng.integers(-1, V, rows).astype(np.int32)),
            _dev(np.array([0, rows // 3, rows], np.int32)), _dev(-5 * rng.random(rows).astype(np.float32)),
            _dev(rng.standard_normal(rows).astype(np.float32)), _dev(vals), _dev(idx)]


@pytest.mark.parametrize("rows,V", [(12, 3001), (3, 60000)])
def test_captured_replayed_and_on_two_streams(rows, V):
    a, b = _inputs(1, rows, V), _inputs(2, rows, V)
    wa, wb = _outs(rows, V, 2, torch.bfloat16), _outs(rows, V, 2, torch.bfloat16)
    _everything(*a, wa)
    _everything(*b, wb)
    torch.cuda.synchronize()
    # a graph over inputs that are filled before each replay
    x = [i.clone() for i in a]
    got = _outs(rows, V, 2, torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(*x, got)
    for src, want in ((a, wa), (b, wb), (a, wa)):
        for i, s in zip(x, src):
            i.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            if n != "ws":
                assert torch.equal(got[n], want[n]), n
    # two at once, each on a stream and with a workspace of its own; by object and by number
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    g1, g2 = _outs(rows, V, 2, torch.bfloat16), _outs(rows, V, 2, torch.bfloat16)
    torch.cuda.synchronize()
    for _ in range(5):
        _everything(*a, g1, stream=s1)
        _everything(*b, g2, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for n in wa:
        if n != "ws":
            assert torch.equal(g1[n], wa[n]) and torch.equal(g2[n], wb[n]), n


def test_results_do_not_change_from_call_to_call():
    x = _inputs(5, 40, 20011)
    first = _outs(40, 20011, 2, torch.bfloat16)
    _everything(*x, first)
    for _ in range(3):
        again = _outs(40, 20011, 2, torch.bfloat16)
        _everything(*x, again)
        for n in first:
            if n != "ws":
                assert torch.equal(first[n], again[n]), n


def test_tail_scores_policy_and_distillation_together():
    """A rollout's tokens from the tail, scored, and a policy step on the same logits: the ratio is 1.  The tail's
    top-k as the teacher of a draft model: its steps bring the draft's log-probabilities to the teacher's."""
    g = torch.Generator(device=DEV).manual_seed(3)
    H, V, k, n = 256, 8192, 64, 4
    w = (torch.randn((H, V), generator=g, device=DEV) * 0.15).to(torch.bfloat16)
    hidden = torch.randn((n, H), generator=g, device=DEV).to(torch.bfloat16)
    params = torch.tensor([[0, 1.0, 0.8, 0.1 + 0.2 * i] for i in range(n)], device=DEV)
    tokens = torch.empty(n, dtype=torch.int32, device=DEV)
    logits = torch.empty((n, V), device=DEV)
    vals, idx = torch.empty((n, k), device=DEV), torch.empty((n, k), dtype=torch.int32, device=DEV)
    with dst.Tail(H, V, k, n, hidden_dtype="bf16") as tail:
        tail.run(hidden, torch.ones(H, device=DEV), w, params, out_tokens=tokens, out_logits=logits, out_topk_vals=vals,
                 out_topk_idx=idx)
        tail.check()
    old, lse, _ = dst.token_logprobs(logits, tokens, 0.8)
    assert torch.isfinite(old).all() and (old < 0).all()
    adv = torch.randn(n, generator=g, device=DEV)
    loss, lp, grad = dst.policy_loss(logits, tokens, old, adv, ref_logprob=old, kl_coef=0.1, temperature=0.8)
    assert torch.allclose(lp, old, rtol=1e-6, atol=1e-6) and torch.allclose(loss, -adv, rtol=1e-5)
    assert torch.allclose(grad, dst.token_logprobs_grad(logits, tokens, lse, -adv, 0.8), rtol=1e-4, atol=1e-7)

    rest = (dst.token_logprobs(logits, idx[:, 0].contiguous())[1].double())
    rest = (rest + torch.log1p(-torch.exp(vals.double() - rest[:, None]).sum(-1))).float()
    full = torch.log_softmax(logits.double(), -1)
    student = (logits + 0.5 * torch.randn((n, V), generator=g, device=DEV)).contiguous()
    before = (torch.exp(full) * (full - torch.log_softmax(student.double(), -1))).sum(-1)
    leaf = student.clone().requires_grad_()
    kl, d = dst.distill_topk(leaf.detach(), vals, idx, teacher_rest=rest)
    (leaf * 1.0).backward(d)  # the gradient is handed on to whatever formed the logits
    assert torch.equal(leaf.grad, d)
    assert (kl.double() <= before + 1e-6).all()  # merging the others loses their part of the divergence
    step = student - 1e-2 * d
    after = dst.distill_topk(step, vals, idx, teacher_rest=rest, grad=False)[0]
    want = -1e-2 * (d.double() ** 2).sum(-1)  # to first order
    assert torch.allclose((after - kl).double(), want, rtol=0.1, atol=1e-5)


def test_outputs_of_a_call_on_the_default_stream_by_its_number():
    from decode_sampling_tail_gb300._args import allocating_on
    zero = torch.cuda.default_stream(DEV).cuda_stream
    assert zero == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        with allocating_on(zero, 0):
            assert torch.cuda.current_stream().cuda_stream == zero
        assert torch.cuda.current_stream().cuda_stream != zero
    z = torch.randn((4, 500), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    t = torch.arange(4, dtype=torch.int32, device=DEV)
    want = dst.token_logprobs(z, t)
    torch.cuda.synchronize()
    got = dst.token_logprobs(z, t, stream=zero)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_rest_of_confident_teachers():
    """The tail's top-k of rows that hold all but 10^-1 to 10^-12 of the weight, their rests both ways that distill_topk
    documents, and a student's loss against 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(7)
    H, V, k, n, T = 256, 8192, 64, 8, f32(0.9)
    x = torch.randn((n, H), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((H, V), generator=g, device=DEV) * 0.15
    unit = x.float() / x.float().pow(2).mean(-1, keepdim=True).sqrt()
    for r in range(n):  # logit of column 100 + r in row r
        w[:, 100 + r] = unit[r] * (13.0 + 3.5 * r) / H
    logits, tokens = torch.empty((n, V), device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
    vals, idx = torch.empty((n, k), device=DEV), torch.empty((n, k), dtype=torch.int32, device=DEV)
    with dst.Tail(H, V, k, n, hidden_dtype="bf16") as tail:
        tail.run(x, torch.ones(H, device=DEV), w.to(torch.bfloat16), torch.tensor([[0, 1.0, T, 0.5]] * n, device=DEV),
                 out_tokens=tokens, out_logits=logits, out_topk_vals=vals, out_topk_idx=idx)
        tail.check()
    y = logits.double() / T
    exact = torch.logsumexp(y.scatter(1, idx.long(), -INF), -1)
    left = (exact - torch.logsumexp(y, -1)).exp()
    assert left.max().item() > 1e-3 and 0 < left.min().item() < 1e-8

    others = logits.scatter(1, idx.long(), -INF)
    rest = dst.token_logprobs(others, idx[:, 0].contiguous(), T)[1]
    # 2^-17 of the sum, and half a step
    assert ((rest.double() - exact).abs() <= 2.0 ** -17 + 2.0 ** -22 * exact.abs()).all()
    lse = dst.token_logprobs(logits, tokens, T)[1]
    listed = torch.exp(vals.double() / T - lse.double()[:, None]).sum(-1)
    rough = (lse.double() + torch.log(torch.clamp(1 - listed, min=0))).float()
    # what is left, by lse's error of the whole weight: 2^-17 min(1, s) of its sum, and its rounding
    off = (torch.exp(rough.double() - torch.logsumexp(y, -1)) - left).abs()
    s = torch.expm1(torch.logsumexp(y, -1) - y.amax(-1)).clamp(max=1)
    assert (off <= 2.0 ** -17 * s + 2.0 ** -22 * (lse.abs().double() + 1)).all()

    student = logits + 0.5 * torch.randn((n, V), generator=g, device=DEV)
    for some in (rest, rough):
        loss, d = (_np(a) for a in dst.distill_topk(student, vals, idx, teacher_rest=some, temperature=T))
        assert np.isfinite(loss).all() and np.isfinite(d).all()
        for r in range(n):
            v, tol = tc.distill(_np(student[r]), _np(vals[r]).astype(np.float32), idx[r].cpu().numpy(), float(some[r]), T,
                                1.0, "f32")
            tc.near(loss[r], v[0], tol[0], f"loss of row {r}")
            tc.near(d[r], v[1], tol[1], f"gradient of row {r}")

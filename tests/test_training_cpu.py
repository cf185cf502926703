"""The training operators without a GPU: refusals of the C entry points and of their wrappers, and the 64-bit formulas
of tests/traincheck.py against differences and cases worked by hand."""
import ctypes
import math

import numpy as np
import pytest

import decode_sampling_tail_gb300 as dst
from decode_sampling_tail_gb300 import build as dbuild
from tests import traincheck as tc

P = 1 << 20           # stands for an aligned device pointer; refused calls never read it
O1, O2, O3, G, WS = 1 << 24, 1 << 25, 1 << 26, 1 << 30, 1 << 27
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def L():
    dbuild.build()
    return dst.lib()


def logprobs(L, **kw):
    a = dict(rows=4, V=100, z=P, dt=0, ld=100, t=P, T=1.0, lp=O1, lse=O2, ent=O3)
    a.update(kw)
    return L.tail_token_logprobs(a["rows"], a["V"], a["z"], a["dt"], a["ld"], a["t"], a["T"], a["lp"], a["lse"],
                                 a["ent"], None)


def logprobs_grad(L, **kw):
    a = dict(rows=4, V=100, z=P, dt=0, ld=100, t=P, T=1.0, lse=P, a=P, b=P, ent=P, g=G, gld=100)
    a.update(kw)
    return L.tail_token_logprobs_grad(a["rows"], a["V"], a["z"], a["dt"], a["ld"], a["t"], a["T"], a["lse"], a["a"],
                                      a["b"], a["ent"], a["g"], a["gld"], None)


def policy(L, **kw):
    a = dict(rows=4, V=100, z=P, dt=0, ld=100, t=P, T=1.0, old=P, adv=P, ref=P, lo=0.2, hi=0.2, kl=0.1, e=0.0, w=None,
             loss=O1, lp=O2, ent=O3, g=G, gld=100)
    a.update(kw)
    return L.tail_policy_loss(a["rows"], a["V"], a["z"], a["dt"], a["ld"], a["t"], a["T"], a["old"], a["adv"], a["ref"],
                              a["lo"], a["hi"], a["kl"], a["e"], a["w"], a["loss"], a["lp"], a["ent"], a["g"], a["gld"],
                              None)


def preference(L, **kw):
    a = dict(rows=4, V=100, nseq=2, z=P, dt=0, ld=100, t=P, cu=P, T=1.0, ref=P, beta=0.1, eps=0.0, m=0.0, avg=0, w=P,
             ws=WS, wb=1 << 20, loss=O1, seq=O2, g=G, gld=100)
    a.update(kw)
    return L.tail_preference_loss(a["rows"], a["V"], a["nseq"], a["z"], a["dt"], a["ld"], a["t"], a["cu"], a["T"],
                                  a["ref"], a["beta"], a["eps"], a["m"], a["avg"], a["w"], a["ws"], a["wb"], a["loss"],
                                  a["seq"], a["g"], a["gld"], None)


def distill(L, **kw):
    a = dict(rows=4, V=100, k=8, z=P, dt=0, ld=100, v=P, vdt=0, vld=8, i=P, ild=8, T=1.0, rest=P, w=P, loss=O1, g=G,
             gld=100)
    a.update(kw)
    return L.tail_distill_topk(a["rows"], a["V"], a["k"], a["z"], a["dt"], a["ld"], a["v"], a["vdt"], a["vld"], a["i"],
                               a["ild"], a["T"], a["rest"], a["w"], a["loss"], a["g"], a["gld"], None)


CALLS = dict(logprobs=logprobs, logprobs_grad=logprobs_grad, policy=policy, preference=preference, distill=distill)
BAD = [dict(rows=-1), dict(V=0), dict(V=-5), dict(z=None), dict(z=P + 2), dict(z=P + 1, dt=2), dict(dt=3), dict(dt=-1),
       dict(ld=99), dict(T=0.0), dict(T=-1.0), dict(T=NAN), dict(T=INF), dict(T=1e-30)]
GRAD = [dict(gld=99), dict(g=G + 2), dict(g=P + 4), dict(g=P, gld=104), dict(g=P + 400, ld=150, gld=150)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", BAD)
def test_all_refuse(L, call, kw):
    assert CALLS[call](L, **kw) == dst.TAIL_ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["logprobs_grad", "policy", "preference", "distill"])
@pytest.mark.parametrize("kw", GRAD)
def test_gradients_over_the_logits_are_refused(L, call, kw):
    assert CALLS[call](L, **kw) == dst.TAIL_ERR_INVALID_ARG


@pytest.mark.parametrize("call,kw", [
    ("logprobs", dict(t=None)), ("logprobs", dict(t=P + 1)), ("logprobs", dict(lp=None, lse=None, ent=None)),
    ("logprobs", dict(lp=O1 + 2)), ("logprobs", dict(lp=P)), ("logprobs", dict(lp=O1, lse=O1 + 8)),
    ("logprobs", dict(lse=P + 1596)), ("logprobs_grad", dict(lse=None)), ("logprobs_grad", dict(a=None)),
    ("logprobs_grad", dict(b=None)), ("logprobs_grad", dict(ent=None)), ("logprobs_grad", dict(g=None)),
    ("logprobs_grad", dict(a=G + 16)), ("policy", dict(t=None)), ("policy", dict(old=None)), ("policy", dict(adv=None)),
    ("policy", dict(ref=None)), ("policy", dict(loss=None)), ("policy", dict(lo=-0.1)), ("policy", dict(lo=1.5)),
    ("policy", dict(lo=NAN)), ("policy", dict(hi=-0.1)), ("policy", dict(hi=NAN)), ("policy", dict(kl=INF)),
    ("policy", dict(e=NAN)), ("policy", dict(w=P + 2)), ("policy", dict(loss=P)), ("policy", dict(lp=O1)),
    ("policy", dict(old=G + 400)), ("policy", dict(loss=G)), ("preference", dict(nseq=-2)), ("preference", dict(nseq=3)),
    ("preference", dict(cu=None)), ("preference", dict(cu=P + 2)), ("preference", dict(t=None)),
    ("preference", dict(beta=INF)), ("preference", dict(m=NAN)), ("preference", dict(eps=-0.1)),
    ("preference", dict(eps=1.1)), ("preference", dict(avg=2)), ("preference", dict(ws=None)),
    ("preference", dict(ws=WS + 8)), ("preference", dict(wb=100)), ("preference", dict(loss=None)),
    ("preference", dict(seq=O1)), ("preference", dict(loss=WS)), ("preference", dict(ws=P)),
    ("distill", dict(k=0)), ("distill", dict(k=1025, vld=1025, ild=1025)), ("distill", dict(v=None)),
    ("distill", dict(vdt=3)), ("distill", dict(vld=7)), ("distill", dict(v=P + 2)), ("distill", dict(i=None)),
    ("distill", dict(ild=7)), ("distill", dict(i=P + 2)), ("distill", dict(loss=None)), ("distill", dict(loss=P)),
    ("distill", dict(rest=O1)), ("distill", dict(v=G))])
def test_refusals_of_its_own(L, call, kw):
    assert CALLS[call](L, **kw) == dst.TAIL_ERR_INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [dict(V=(1 << 20) + 1, ld=1 << 21, gld=1 << 21), dict(rows=(1 << 24) + 1)])
def test_limits(L, call, kw):
    if call == "logprobs":
        kw = {k: v for k, v in kw.items() if k != "gld"}
    assert CALLS[call](L, **kw) == dst.TAIL_ERR_UNSUPPORTED
    assert L.tail_last_error()


def test_no_rows_is_a_no_op(L):
    for name, call in CALLS.items():
        kw = dict(rows=0, z=None, t=None)
        if name == "distill":
            kw.pop("t")
        if name == "preference":
            kw["nseq"] = 0
        assert call(L, **kw) == dst.TAIL_OK, name


def test_workspace(L):
    n = ctypes.c_int64()
    sizes = []
    for rows in (0, 1, 1000, 1 << 24):
        assert L.tail_preference_loss_workspace(rows, ctypes.byref(n)) == dst.TAIL_OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] == 0 and sizes[2] >= 20 * 1000
    assert dst.preference_loss_workspace(1000) == sizes[2]
    assert L.tail_preference_loss_workspace(1, None) == dst.TAIL_ERR_INVALID_ARG
    assert L.tail_preference_loss_workspace(-1, ctypes.byref(n)) == dst.TAIL_ERR_INVALID_ARG
    with pytest.raises(dst.TailError):
        dst.preference_loss_workspace((1 << 24) + 1)


def test_wrappers_want_cuda_tensors():
    torch = pytest.importorskip("torch")
    z, i, f = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for call in (lambda: dst.token_logprobs(z, i), lambda: dst.token_logprobs_grad(z, i, f, f),
                 lambda: dst.policy_loss(z, i, f, f), lambda: dst.preference_loss(z, i, i[:3]),
                 lambda: dst.distill_topk(z, z, i[:, None])):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the formulas

def _grad_by_differences(f, z, h=1e-6):
    g = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        a, b = z.copy(), z.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_log_probability_by_hand():
    z = np.log([1.0, 2.0, 5.0])
    (l, lse, H), _ = tc.logprob(z, 1, 1.0)
    assert math.isclose(l, math.log(0.25)) and math.isclose(lse, math.log(8.0))
    assert math.isclose(H, -sum(p * math.log(p) for p in (0.125, 0.25, 0.625)))
    assert tc.logprob(z, 3, 1.0)[0] == (0.0, 0.0, 0.0)
    assert tc.logprob([-INF, -INF], 0, 1.0)[0] == (-INF, -INF, 0.0)
    assert math.isclose(tc.logprob([50.0, 0.0], 0, 1.0)[0][0], -math.exp(-50.0), rel_tol=1e-12)


@pytest.mark.parametrize("T", [1.0, 0.6])
def test_spread_is_the_gradient(T):
    z = np.random.default_rng(1).standard_normal(9) * 2
    f = lambda x: 0.7 * tc.logprob(x, 4, T)[0][0] + 0.3 * tc.logprob(x, 4, T)[0][2]  # noqa: E731
    g, _ = tc.spread(z, 4, T, 0.7, 0.3, "f32")
    assert np.allclose(g, _grad_by_differences(f, z), atol=1e-8)


@pytest.mark.parametrize("old,adv", [(-1.0, 0.8), (-1.0, -0.8), (-3.0, 0.8), (-3.0, -0.8), (-0.2, 1.0), (-0.2, -1.0)])
def test_policy_is_its_gradient(old, adv):
    z = np.random.default_rng(2).standard_normal(7)
    args = (3, 0.9, old, adv, -1.4, 0.2, 0.3, 0.05, 0.02, 1.7, "f32")
    (loss, l, H, g), _ = tc.policy(z, *args)
    R = math.exp(l - old)
    want = -min(adv * R, adv * min(max(R, 0.8), 1.3)) + 0.05 * (math.exp(-1.4 - l) - (-1.4 - l) - 1) - 0.02 * H
    assert math.isclose(loss, 1.7 * want, rel_tol=1e-12)
    assert np.allclose(g, _grad_by_differences(lambda x: tc.policy(x, *args)[0][0], z), atol=1e-8)


@pytest.mark.parametrize("average", [0, 1])
def test_preference_is_its_gradient(average):
    rng = np.random.default_rng(3)
    z, t, cu = rng.standard_normal((9, 5)), np.array([0, 4, -1, 2, 2, 1, 9, 3, 0]), [1, 4, 6, 6, 8]
    args = (t, cu, 1.1, np.array([-3.0, -2.5, -0.5, -1.0]), 0.7, 0.1, 0.2, average, np.array([1.0, 0.4]), "f32")
    (loss, L, g), _ = tc.preference(z, *args)
    assert L[2] == 0.0 and np.all(g[[0, 2, 6, 8]] == 0) and loss.shape == (2,)
    assert np.allclose(g, _grad_by_differences(lambda x: tc.preference(x, *args)[0][0].sum(), z), atol=1e-8)


@pytest.mark.parametrize("rest", [None, 0.3, -INF, 4.0])
@pytest.mark.parametrize("idx", [[4, 0, 2], [4, -1, 2], [3, 3, 1], [9, -1, 11]])
def test_distill_is_its_gradient(rest, idx):
    z = np.random.default_rng(4).standard_normal(6)
    args = (np.array([1.0, 0.2, -0.4]), np.array(idx), rest, 0.8, 1.3, "f32")
    (loss, g), _ = tc.distill(z, *args)
    assert np.allclose(g, _grad_by_differences(lambda x: tc.distill(x, *args)[0][0], z), atol=1e-8)
    assert abs(g.sum()) < 1e-12  # adding a number to every logit changes nothing
    assert (loss == 0) == (idx[0] == 9)


def test_distill_is_zero_where_student_and_teacher_agree():
    z = np.array([1.0, 2.0, 0.5, -1.0])
    (loss, g), _ = tc.distill(z, z[[1, 0]], np.array([1, 0]), float(np.logaddexp(0.5, -1.0)), 1.0, 1.0, "f32")
    assert abs(loss) < 1e-15 and np.allclose(g, 0, atol=1e-15)


def test_sizes_behind_32_bits_are_refused(L):
    torch = pytest.importorskip("torch")
    from decode_sampling_tail_gb300._args import need_matrix
    for shape in ((2 ** 31, 1), (1, 2 ** 32 + 5), (2 ** 32 + 1, 7)):
        t = torch.empty(shape, dtype=torch.bfloat16, device="meta")
        with pytest.raises(ValueError, match="2\\^31"):
            need_matrix(t, "logits", shape[0], t.get_device())
    for rows in (2 ** 31, 2 ** 32, 2 ** 32 + 1, -1):
        with pytest.raises(ValueError, match="rows"):
            dst.preference_loss_workspace(rows)
    assert dst.preference_loss_workspace(0) == 0 and dst.preference_loss_workspace(1) == 512


def test_allocations_on_the_default_stream_by_its_number(monkeypatch):
    torch = pytest.importorskip("torch")
    from decode_sampling_tail_gb300._args import allocating_on
    used = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: used.append(s))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda pointer, device=None: ("other", pointer, device))
    for number in (0, 1, 0x7f0012340000):  # what a default stream's cuda_stream is; cudaStreamLegacy; any other
        allocating_on(number, 3)
    assert used == [("default", 3), ("default", 3), ("other", 0x7f0012340000, 3)]


def test_statistics_refusals(L):
    S = 1 << 28  # [rows][2]
    scores = lambda **k: (lambda a: L.tail_token_logprobs_ex(4, 100, P, 0, 100, P, 1.0, a["lp"], a["lse"], a["H"],  # noqa: E731
                                                             a["s"], None))({**dict(lp=O1, lse=O2, H=O3, s=S), **k})
    for bad in (dict(s=S + 2), dict(s=P), dict(s=P + 1592), dict(lp=S + 28), dict(lp=None, lse=None, H=None, s=None)):
        assert scores(**bad) == dst.TAIL_ERR_INVALID_ARG
    grad = lambda **k: (lambda a: L.tail_token_logprobs_grad_ex(4, 100, P, 0, 100, P, a["T"], a["lse"], a["s"], a["a"],  # noqa: E731
                                                                None, None, G, 100, None))(
        {**dict(T=1.0, lse=None, s=S, a=P), **k})
    for bad in (dict(s=None), dict(s=S + 1), dict(s=G - 28), dict(a=None), dict(T=0.0), dict(lse=P + 2)):
        assert grad(**bad) == dst.TAIL_ERR_INVALID_ARG


def test_wait_limit(L):
    for ns in (-1, 1 << 64):
        with pytest.raises(ValueError):
            dst.set_training_wait_limit(ns)

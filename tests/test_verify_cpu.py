"""Refusals of tail_verify and tail_verify_logits (host side, no GPU), the argument checks of their wrappers, and
the 64-bit rule of tests/verifycheck.py against cases worked by hand."""
import ctypes

import numpy as np
import pytest

import decode_sampling_tail_gb300 as dst
from decode_sampling_tail_gb300 import build as dbuild
from tests import verifycheck as vc

P = 4096  # stands for an aligned device pointer; refused calls never read it
OT, OC, WS = 1 << 24, 1 << 25, 1 << 26  # outputs and workspace, apart from it


@pytest.fixture(scope="module")
def L():
    dbuild.build()
    return dst.lib()


def verify(L, **kw):
    a = dict(rows=4, nseq=1, k=8, vals=P, idx=P, params=P, cols=4, cu=P, drafts=P, accept=P, q=None, qd=0, ld=0, V=0,
             tokens=OT, count=OC)
    a.update(kw)
    return L.tail_verify(a["rows"], a["nseq"], a["k"], a["vals"], a["idx"], a["params"], a["cols"], a["cu"],
                         a["drafts"], a["accept"], a["q"], a["qd"], a["ld"], a["V"], a["tokens"], a["count"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(nseq=-1), dict(k=0), dict(k=1025), dict(cols=2), dict(cols=5), dict(vals=None),
    dict(idx=None), dict(params=None), dict(cu=None), dict(drafts=None), dict(accept=None), dict(tokens=None),
    dict(count=None), dict(vals=P + 2), dict(idx=P + 1), dict(cu=P + 2), dict(tokens=P + 2), dict(count=P + 1),
    dict(q=P, qd=3, ld=64, V=64), dict(q=P, qd=0, ld=63, V=64), dict(q=P, qd=0, ld=64, V=0),
    dict(q=P + 2, qd=0, ld=64, V=64), dict(q=P + 1, qd=2, ld=64, V=64)])
def test_verify_refuses(L, kw):
    assert verify(L, **kw) == dst.TAIL_ERR_INVALID_ARG


@pytest.mark.parametrize("call,names", [
    ("verify", ["cu", "drafts", "accept", "vals", "idx", "params"]),
    ("logits", ["cu", "drafts", "accept", "u", "temp", "ws"])])
@pytest.mark.parametrize("out", ["tokens", "count"])
def test_outputs_over_inputs_are_refused(L, call, names, out):
    run = verify if call == "verify" else logits
    for name in names:
        # one sequence of 4 rows: 16 bytes of tokens, 4 of counts
        for by in ((0, -16) if name == "ws" else (0, 4, -4) if out == "tokens" else (0, -4)):
            kw = {out: 1 << 28, name: (1 << 28) + by}
            assert run(L, **kw) == dst.TAIL_ERR_INVALID_ARG, (name, by)
    assert run(L, tokens=OT, count=OT + 12) == dst.TAIL_ERR_INVALID_ARG


def test_no_sequences_is_a_no_op(L):
    assert verify(L, nseq=0, cu=None, count=None) == dst.TAIL_OK


def logits(L, **kw):
    a = dict(rows=4, nseq=1, V=100, logits=P, ld_t=0, ld=100, temp=P, cu=P, drafts=P, accept=P, u=P, q=None, qd=0,
             qld=0, ws=WS, wb=1 << 20, tokens=OT, count=OC)
    a.update(kw)
    return L.tail_verify_logits(a["rows"], a["nseq"], a["V"], a["logits"], a["ld_t"], a["ld"], a["temp"], a["cu"],
                                a["drafts"], a["accept"], a["u"], a["q"], a["qd"], a["qld"], a["ws"], a["wb"],
                                a["tokens"], a["count"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(nseq=-1), dict(V=0), dict(logits=None), dict(temp=None), dict(cu=None), dict(drafts=None),
    dict(accept=None), dict(u=None), dict(tokens=None), dict(count=None), dict(ld_t=3), dict(ld_t=-1), dict(ld=99),
    dict(logits=P + 2), dict(logits=P + 1, ld_t=2), dict(temp=P + 2), dict(ws=None), dict(ws=WS + 8), dict(wb=100),
    dict(q=P, qd=3, qld=100), dict(q=P, qld=99), dict(q=P + 2, qld=100)])
def test_verify_logits_refuses(L, kw):
    assert logits(L, **kw) == dst.TAIL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(V=(1 << 20) + 1, ld=1 << 21), dict(rows=65536), dict(nseq=65536)])
def test_verify_logits_limits(L, kw):
    assert logits(L, wb=1 << 40, **kw) == dst.TAIL_ERR_UNSUPPORTED
    assert L.tail_last_error()


def test_workspace_grows_with_the_call(L):
    n = ctypes.c_int64()
    sizes = []
    for rows, nseq, V in ((0, 1, 1), (1, 1, 1), (8, 2, 201088), (65535, 65535, 1 << 20)):
        assert L.tail_verify_logits_workspace(rows, nseq, V, ctypes.byref(n)) == dst.TAIL_OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[2] >= 8 * 25 * 16
    assert dst.verify_logits_workspace(8, 2, 201088) == sizes[2]
    assert L.tail_verify_logits_workspace(1, 1, 1, None) == dst.TAIL_ERR_INVALID_ARG
    with pytest.raises(dst.TailError):
        dst.verify_logits_workspace(1, 1, 1 << 21)


def test_wrappers_want_cuda_tensors():
    torch = pytest.importorskip("torch")
    i = torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(3)
    with pytest.raises(ValueError):
        dst.verify(torch.zeros(3, 4), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4), i[:2], i, f)
    with pytest.raises(ValueError):
        dst.verify_logits(torch.zeros(3, 10), f, i[:2], i, f, f)


def test_probabilities_without_columns_are_refused():
    # their pointer is null, which would stand for certain drafts
    torch = pytest.importorskip("torch")
    from decode_sampling_tail_gb300 import _args
    assert _args.need_matrix(torch.zeros(3, 5), "q", 3, -1)[2:] == (5, 5)
    with pytest.raises(ValueError):
        _args.need_matrix(torch.zeros(3, 0), "q", 3, -1)


# ------------------------------------------------------------------ the rule by hand

def _one(target, draft, drafts, accept, u):
    n = len(drafts)
    t, c, _ = vc.settle([0, n], drafts, accept, u, lambda r: ((np.array(target), np.arange(len(target))), 1.0), draft, n)
    return t.tolist(), int(c[0])


def test_rule_accepts_below_the_ratio_and_draws_the_rest():
    p, q = [0.5, 0.3, 0.2], np.array([0.2, 0.6, 0.2])
    draft = lambda row, ids: q[ids]  # noqa: E731
    # draft 1 has p / q = 0.5: a = 0.49 stands, a = 0.5 does not; the residual is (0.3, 0, 0): token 0
    assert _one(p, draft, [1, 0], [0.49, 0], [0, 0.85]) == ([1, 2], 2)
    assert _one(p, draft, [1, 0], [0.5, 0], [0.99, 0.85]) == ([0, -1], 1)


def test_rule_certain_drafts_and_absent_tokens():
    none = lambda row, ids: None  # noqa: E731
    p = [0.5, 0.3, 0.2]
    assert _one(p, none, [1, 0], [0.29, 0], [0, 0.6]) == ([1, 1], 2)
    # refused: drawn from (0.5, 0, 0.2) / 0.7
    assert _one(p, none, [1, 0], [0.31, 0], [0.7, 0]) == ([0, -1], 1)
    assert _one(p, none, [1, 0], [0.31, 0], [0.72, 0]) == ([2, -1], 1)
    assert _one(p, none, [-1, 0], [0.0, 0], [0.1, 0]) == ([0, -1], 1)


def test_rule_emits_the_target_distribution():
    # the exact law of the first token over the two uniforms: accepted mass + refused mass x residual
    p, q = np.array([0.5, 0.2, 0.3]), np.array([0.1, 0.6, 0.3])
    rest = np.maximum(p - q, 0) / np.maximum(p - q, 0).sum()
    law = np.minimum(p, q) + (q - np.minimum(p, q)).sum() * rest
    assert np.allclose(law, p)
    n, grid = np.zeros(3), 400
    for x in range(3):
        for i in range(grid):
            a = (i + 0.5) / grid
            t, _ = _one(p, lambda row, ids: q[ids], [x, 0], [a, 0], [(i * 7 % grid + 0.5) / grid, 0])
            n[t[0]] += q[x] / grid
    assert np.abs(n - p).max() < 0.01


def test_sampler_target_cuts_like_the_sampler():
    v, i = [2.0, 1.0, 0.0, -np.inf], [7, 3, 9, 1]
    (p, ids), _ = vc.sampler_target(v, i, [0, 0.7, 1.0])
    e = np.exp([0.0, -1.0])
    assert ids.tolist() == [7, 3] and np.allclose(p, e / e.sum())
    (p, ids), _ = vc.sampler_target(v, i, [2, 1.0, 1.0])
    assert ids.tolist() == [7, 3]
    (p, ids), _ = vc.sampler_target(v, i, [0, 1.0, 0.0])
    assert ids.tolist() == [7] and p.tolist() == [1.0]
    assert vc.sampler_target([-np.inf, -np.inf], [0, 1], [0, 1, 1])[0] is None

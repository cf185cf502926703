"""tail_verify and tail_verify_logits on the GPU against the 64-bit rule of tests/verifycheck.py."""
import numpy as np
import pytest

from tests import verifycheck as vc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import decode_sampling_tail_gb300 as dst  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _lens(rng, nseq, most, pad):
    n = rng.integers(1, most + 1, nseq)
    if nseq > 3:
        n[nseq // 2] = 0  # an empty sequence
        n[nseq // 3] = 11  # more rows than a CTA has warps
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return cu, int(cu[-1]) + pad


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


# ------------------------------------------------------------------ lists

def _lists_case(seed, nseq, k, V, q, most=6, pad=3, cols=4, params=None):
    rng = np.random.default_rng(seed)
    cu, R = _lens(rng, nseq, most, pad)
    vals = -np.sort(-(rng.standard_normal((R, k)) * 2.0).astype(np.float32), axis=1)
    idx = np.stack([rng.permutation(V)[:k] for _ in range(R)]).astype(np.int32)
    prm = np.empty((R, 4), np.float32)
    prm[:, 0] = rng.choice([0, 1, 2, 5, 1e6, max(1, k // 2)], R)
    prm[:, 1] = np.where(rng.random(R) < 0.4, 1.0, rng.uniform(0.2, 0.99, R))
    prm[:, 2] = np.where(rng.random(R) < 0.15, 0.0, rng.uniform(0.3, 1.6, R))
    prm[:, 3] = rng.random(R)
    if params is not None:
        params(prm, vals, idx)
    full = rng.standard_normal((R, V)).astype(np.float32) - 4
    np.put_along_axis(full, idx.astype(np.int64), vals + 0.5 * rng.standard_normal((R, k)).astype(np.float32), 1)
    Q = _softmax(np.where(np.isfinite(full), full, -50.0)).astype(np.float32)
    drafts = np.array([rng.choice(V, p=p / p.sum()) for p in Q.astype(np.float64)], np.int32)
    drafts[rng.random(R) < 0.1] = -1
    accept = rng.random(R, dtype=np.float32)
    qt = None if q == "none" else _dev(Q, DT[q])
    return dict(cu=cu, R=R, vals=vals, idx=idx, prm=np.ascontiguousarray(prm[:, :cols]), drafts=drafts, accept=accept,
                q=qt, V=V, cols=cols)


def _lists_want(c):
    qn = None if c["q"] is None else c["q"].double().cpu().numpy()
    u = c["prm"][:, 3] if c["cols"] == 4 else np.full(c["R"], 0.5)

    def draft(row, ids):
        if qn is None:
            return None
        ids = np.asarray(ids)
        ok = (ids >= 0) & (ids < c["V"])
        return np.where(ok, np.clip(qn[row][np.where(ok, ids, 0)], 0, 1), 0.0)

    return vc.settle(c["cu"], c["drafts"], c["accept"], u,
                     lambda r: vc.sampler_target(c["vals"][r], c["idx"][r], c["prm"][r]), draft, c["R"])


def _lists_run(c, **kw):
    tokens = torch.full((c["R"],), -7, dtype=torch.int32, device=DEV)
    t, n = dst.verify(_dev(c["vals"]), _dev(c["idx"]), _dev(c["prm"]), _dev(c["cu"]), _dev(c["drafts"]),
                      _dev(c["accept"]), draft_probs=c["q"], out_tokens=tokens, **kw)
    torch.cuda.synchronize()
    return t.cpu().numpy(), n.cpu().numpy()


@pytest.mark.parametrize("q", ["none", "f32", "f16", "bf16"])
@pytest.mark.parametrize("nseq,k,V,cols", [(1, 1, 16, 4), (5, 2, 40, 3), (33, 37, 1001, 4), (64, 256, 4096, 4),
                                           (9, 1000, 1024, 4), (7, 1024, 5000, 3)])
def test_lists_match_the_rule(nseq, k, V, cols, q):
    c = _lists_case(11 + k, nseq, k, V, q, cols=cols)
    tokens, counts = _lists_run(c)
    assert vc.compare(tokens, counts, _lists_want(c), c["cu"]) >= 0.9 * nseq


def test_lists_without_drafts_draw_the_tails_tokens():
    # a sequence of one row is a plain draw: the token of tail_merge_shards on the same candidates
    rng = np.random.default_rng(5)
    R, k = 300, 200
    c = _lists_case(6, R, k, 3000, "none", most=1, pad=0)
    c["cu"] = np.arange(R + 1, dtype=np.int32)
    for name in ("vals", "idx", "prm", "drafts", "accept"):
        reps = -(-R // c[name].shape[0])
        c[name] = np.concatenate([c[name]] * reps)[:R]
    c["prm"][:, 3] = rng.random(R)
    c["R"] = R
    tokens, counts = _lists_run(c)
    drawn = torch.empty(R, dtype=torch.int32, device=DEV)
    dst.merge_shards(_dev(c["vals"])[None], _dev(c["idx"])[None], [0], k, params=_dev(c["prm"]), out_tokens=drawn)
    want, drawn = _lists_want(c), drawn.cpu().numpy()
    away = want[2] > 1e-5  # the sampler's own sums are fp32
    assert away.sum() > 250 and np.array_equal(tokens[away], drawn[away])
    assert np.all(counts == 1)


@pytest.mark.parametrize("q", ["none", "f32"])
def test_lists_masked_and_extreme_rows(q):
    def edit(prm, vals, idx):
        vals[0::9] = -np.inf                      # nothing left
        vals[1::9, 1:] = -np.inf                  # one candidate left
        vals[2::9, 20:] = np.finfo(np.float32).min
        vals[3::9, :3] = np.inf                   # the mass is shared
        vals[4::9] = 2.5                          # ties: list order
        prm[5::9, 2] = 1e-30
        prm[6::9, 2] = 1e30
        prm[7::9, 1] = 0.0
        prm[8::9, :3] = [np.nan, np.nan, 0.7]
    c = _lists_case(21, 60, 48, 500, q, params=edit)
    tokens, counts = _lists_run(c)
    assert vc.compare(tokens, counts, _lists_want(c), c["cu"]) > 40


@pytest.mark.parametrize("q", ["none", "f32"])
def test_smallest_and_largest_temperatures(q):
    # below 2^-127 the reciprocal of a temperature is no fp32 number; at +inf it is 0
    def lists(prm, vals, idx):
        prm[0::4, 2] = 1e-40
        prm[1::4, 2] = 1.5e-45
        prm[2::4, 2] = np.inf
        vals[::2, 30:] = -np.inf
    c = _lists_case(23, 40, 48, 500, q, params=lists)
    tokens, counts = _lists_run(c)
    assert vc.compare(tokens, counts, _lists_want(c), c["cu"]) > 25

    def whole(z, temp):
        temp[0::4] = 1e-40
        temp[1::4] = 1.5e-45
        temp[2::4] = np.inf
        z[::2, 5000:] = -np.inf
    c = _logits_case(24, 40, 9001, "f32", q, edit=whole)
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) > 25


def test_lists_draft_covering_the_target_draws_from_it():
    # q is 1 at every id: the residual is zero, the draw is from P
    c = _lists_case(31, 40, 20, 100, "f32")
    c["q"] = torch.ones_like(c["q"])
    c["accept"][:] = 0.9999
    tokens, counts = _lists_run(c)
    assert vc.compare(tokens, counts, _lists_want(c), c["cu"]) > 30


def test_lists_ids_outside_the_draft_columns():
    c = _lists_case(33, 20, 30, 200, "f32")
    c["V"] = 150
    c["q"] = c["q"][:, :150]  # a strided view: its rows are 200 apart
    tokens, counts = _lists_run(c)
    assert vc.compare(tokens, counts, _lists_want(c), c["cu"]) > 15


# ------------------------------------------------------------------ whole vocabulary

def _logits_case(seed, nseq, V, l, q, most=5, pad=2, std=2.5, edit=None):
    rng = np.random.default_rng(seed)
    cu, R = _lens(rng, nseq, most, pad)
    z = (rng.standard_normal((R, V)) * std).astype(np.float32)
    temp = np.where(rng.random(R) < 0.15, 0.0, rng.uniform(0.4, 1.5, R)).astype(np.float32)
    if edit is not None:
        edit(z, temp)
    logits = _dev(z, DT[l])
    zl = logits.float().cpu().numpy()
    safe = np.where(np.isfinite(zl), zl, -30.0)
    Q = _softmax(safe + 0.6 * rng.standard_normal((R, V)).astype(np.float32)).astype(np.float32)
    drafts = np.array([rng.choice(V, p=p / p.sum()) for p in Q.astype(np.float64)], np.int32)
    drafts[rng.random(R) < 0.1] = rng.choice([-1, V, V + 5])
    return dict(cu=cu, R=R, V=V, logits=logits, temp=temp, drafts=drafts, accept=rng.random(R, dtype=np.float32),
                u=rng.random(R, dtype=np.float32), q=None if q == "none" else _dev(Q, DT[q]))


def _logits_want(c):
    z = c["logits"].double().cpu().numpy()
    qn = None if c["q"] is None else c["q"].double().cpu().numpy()

    def draft(row, ids):
        if qn is None:
            return None
        ids = np.asarray(ids)
        ok = (ids >= 0) & (ids < c["V"])
        return np.where(ok, np.clip(qn[row][np.where(ok, ids, 0)], 0, 1), 0.0)

    return vc.settle(c["cu"], c["drafts"], c["accept"], c["u"],
                     lambda r: (vc.softmax_target(z[r], c["temp"][r]), 1.0), draft, c["R"])


def _logits_run(c, **kw):
    tokens = torch.full((c["R"],), -7, dtype=torch.int32, device=DEV)
    t, n = dst.verify_logits(c["logits"], _dev(c["temp"]), _dev(c["cu"]), _dev(c["drafts"]), _dev(c["accept"]),
                             _dev(c["u"]), draft_probs=c["q"], out_tokens=tokens, **kw)
    torch.cuda.synchronize()
    return t.cpu().numpy(), n.cpu().numpy()


@pytest.mark.parametrize("l,q", [("f32", "none"), ("f32", "bf16"), ("f32", "f32"), ("f16", "f32"), ("f16", "none"),
                                 ("bf16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("nseq,V", [(1, 1), (6, 7), (5, 8189), (5, 8192), (12, 20011), (4, 50021)])
def test_logits_match_the_rule(nseq, V, l, q):
    c = _logits_case(100 + V, nseq, V, l, q)
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) >= 0.6 * nseq


@pytest.mark.parametrize("q", ["none", "bf16"])
def test_logits_whole_vocabulary(q):
    c = _logits_case(7, 6, 201088, "f32", q, most=3)
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) >= 3


@pytest.mark.parametrize("q", ["none", "f32"])
def test_logits_flat_distributions(q):
    # thousands of equal shares: a neighbour is one part in V away
    c = _logits_case(8, 40, 30011, "f32", q, std=0.01)
    c["temp"][:] = 1.0
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) >= 30


@pytest.mark.parametrize("l", ["f32", "bf16"])
@pytest.mark.parametrize("q", ["none", "f32"])
def test_logits_masked_and_extreme_rows(l, q):
    def edit(z, temp):
        z[0::9] = -np.inf
        z[1::9, 1:] = -np.inf
        z[2::9, 9000:] = -np.inf                     # whole chunks masked
        z[3::9, 5:9000:17] = np.inf
        z[4::9] = 1.25
        z[5::9, ::2] = -3.0e38
        temp[6::9] = 1e-20
        temp[7::9] = 1e20
        temp[8::9] = np.nan
    c = _logits_case(9, 60, 12007, l, q, edit=edit)
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) > 35


def test_logits_draft_covering_the_target_draws_from_it():
    c = _logits_case(10, 20, 9001, "f32", "f32")
    c["q"] = torch.ones_like(c["q"])
    c["accept"][:] = 0.9999
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) > 12


def test_logits_strided_rows_and_other_alignments():
    c = _logits_case(12, 10, 3001, "f32", "f16")
    wide = torch.full((c["R"], 3010), float("nan"), device=DEV)
    wide[:, 3:3004] = c["logits"]
    c["logits"] = wide[:, 3:3004]
    qw = torch.full((c["R"], 3013), float("nan"), dtype=torch.float16, device=DEV)
    qw[:, 1:3002] = c["q"]
    c["q"] = qw[:, 1:3002]
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) > 7


def test_logits_one_call_is_every_call():
    # results do not depend on the batch, on the stream, nor on what the workspace held
    c = _logits_case(13, 12, 20011, "f32", "bf16", pad=0)
    tokens, counts = _logits_run(c)
    R, nseq = c["R"], len(c["cu"]) - 1
    need = dst.verify_logits_workspace(R, nseq, c["V"])
    side = torch.cuda.Stream(DEV)
    dirty = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    t2, n2 = _logits_run(c, workspace=dirty, stream=side)
    t3, n3 = _logits_run(c, workspace=dirty)
    assert np.array_equal(tokens, t2) and np.array_equal(counts, n2)
    assert np.array_equal(tokens, t3) and np.array_equal(counts, n3)
    for s in range(nseq):
        lo, hi = int(c["cu"][s]), int(c["cu"][s + 1])
        if hi == lo:
            continue
        one = {**c, "cu": np.array([0, hi - lo], np.int32), "R": hi - lo, "logits": c["logits"][lo:hi],
               "q": c["q"][lo:hi], "temp": c["temp"][lo:hi], "drafts": c["drafts"][lo:hi],
               "accept": c["accept"][lo:hi], "u": c["u"][lo:hi]}
        t, n = _logits_run(one)
        assert np.array_equal(t, tokens[lo:hi]) and n[0] == counts[s]


def test_rows_behind_32_bit_offsets():
    # rows 2^30 elements apart: the fourth one's bytes and elements start past 2^32 and past 2^31
    far = 1 << 30
    room = torch.empty(5 * far, dtype=torch.bfloat16, device=DEV)

    def spread(t):
        view = room.as_strided(t.shape, (far, 1), 7)
        view.copy_(t)
        return view

    c = _logits_case(26, 2, 3001, "bf16", "f32", most=1, pad=0)
    c["cu"], c["R"] = np.array([0, 4, 5], np.int32), 5
    g = np.random.default_rng(27)
    for k in ("temp", "accept", "u"):
        c[k] = (0.4 + 0.5 * g.random(5)).astype(np.float32)
    z = torch.from_numpy(2.5 * g.standard_normal((5, 3001))).to(DEV, torch.bfloat16)
    q = torch.softmax(z.float() + 0.3, -1)
    c["logits"], c["q"], c["drafts"] = z, q, q.argmax(-1).int().cpu().numpy()
    for accept in (1e-6, 0.99):
        c["accept"][:] = accept
        want = _logits_want(c)
        tokens, counts = _logits_run({**c, "logits": spread(z)})
        assert vc.compare(tokens, counts, want, c["cu"]) >= 1
        c["q"] = q.to(torch.bfloat16)
        want = _logits_want(c)
        tokens, counts = _logits_run({**c, "q": spread(c["q"])})
        assert vc.compare(tokens, counts, want, c["cu"]) >= 1
        c["q"] = q


@pytest.mark.parametrize("l,q", [("f32", "none"), ("bf16", "f32")])
def test_logits_many_sequences(l, q):
    # enough of them that a chunk is cut into fewer parts; the same tokens as the first ones alone
    c = _logits_case(25, 110, 20011, l, q, most=3)
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) > 90
    n, R = 5, int(c["cu"][5])
    few = {**c, "cu": c["cu"][: n + 1], "R": R, "logits": c["logits"][:R], "q": None if c["q"] is None else c["q"][:R],
           **{k: c[k][:R] for k in ("temp", "drafts", "accept", "u")}}
    t, m = _logits_run(few)
    assert np.array_equal(t, tokens[:R]) and np.array_equal(m, counts[:n])


def test_captured_calls_replay():
    # both forms in one graph, two captured calls with a workspace each; inputs change between replays
    a, b = (_logits_case(s, 8, 9001, "f32", "bf16", pad=0) for s in (14, 15))
    lists = _lists_case(16, 8, 64, 500, "f32")
    want = [_logits_run(a), _logits_run(b), _lists_run(lists)]
    R, nseq, V = a["R"], len(a["cu"]) - 1, a["V"]
    keep = []

    def args(c):
        d = dict(logits=c["logits"].clone(), temperature=_dev(c["temp"]), cu_rows=_dev(c["cu"]), drafts=_dev(c["drafts"]),
                 u_accept=_dev(c["accept"]), u_draw=_dev(c["u"]), draft_probs=c["q"],
                 out_tokens=torch.full((c["R"],), -7, dtype=torch.int32, device=DEV),
                 out_count=torch.full((nseq,), -7, dtype=torch.int32, device=DEV),
                 workspace=torch.empty(dst.verify_logits_workspace(c["R"], nseq, V), dtype=torch.uint8, device=DEV))
        keep.append(d)
        return d

    da, db = args(a), args(b)
    la = [_dev(lists[n]) for n in ("vals", "idx", "prm", "cu", "drafts", "accept")]
    lt = torch.full((lists["R"],), -7, dtype=torch.int32, device=DEV)
    ln = torch.empty(8, dtype=torch.int32, device=DEV)

    def step():
        dst.verify_logits(**da)
        dst.verify_logits(**db)
        dst.verify(*la, draft_probs=lists["q"], out_tokens=lt, out_count=ln)

    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        for d in (da, db):
            d["out_tokens"].fill_(-7)
            d["out_count"].fill_(-7)
        lt.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [(d["out_tokens"].cpu().numpy(), d["out_count"].cpu().numpy()) for d in (da, db)]
        got.append((lt.cpu().numpy(), ln.cpu().numpy()))
        for (t, n), (wt, wn) in zip(got, want):
            assert np.array_equal(t, wt) and np.array_equal(n, wn)
    da["u_accept"].fill_(0.0)  # accepts every draft the target allows
    graph.replay()
    torch.cuda.synchronize()
    a["accept"] = np.zeros_like(a["accept"])
    assert vc.compare(da["out_tokens"].cpu().numpy(), da["out_count"].cpu().numpy(), _logits_want(a), a["cu"]) >= 5


def test_no_rows_and_no_sequences():
    e32, e = torch.empty(0, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    t, n = dst.verify(torch.empty((0, 5), device=DEV), torch.empty((0, 5), dtype=torch.int32, device=DEV),
                      torch.empty((0, 4), device=DEV), cu, e, e32)
    assert t.numel() == 0 and n.tolist() == [0, 0, 0]
    t, n = dst.verify_logits(torch.empty((0, 9), device=DEV), e32, cu, e, e32, e32)
    assert t.numel() == 0 and n.tolist() == [0, 0, 0]
    t, n = dst.verify_logits(torch.empty((0, 9), device=DEV), e32, cu[:1], e, e32, e32)
    assert n.numel() == 0


def test_wrappers_refuse_what_does_not_fit():
    c = _lists_case(40, 4, 8, 64, "f32")
    a = [_dev(c[n]) for n in ("vals", "idx", "prm", "cu", "drafts", "accept")]
    bad = [dict(zip(range(6), a)) for _ in range(7)]
    bad[0][0] = a[0].double()
    bad[1][1] = a[1].long()
    bad[2][2] = a[2][:, :2]
    bad[3][3] = a[3].cpu()
    bad[4][4] = a[4][:-1]
    bad[5][0] = a[0].t().contiguous().t()
    bad[6][5] = a[5].half()
    for b in bad:
        with pytest.raises(ValueError):
            dst.verify(*[b[i] for i in range(6)])
    with pytest.raises(ValueError):
        dst.verify(*a, draft_probs=c["q"].t())
    with pytest.raises(ValueError):
        dst.verify(*a, draft_probs=c["q"].double())
    g = _logits_case(41, 4, 100, "f32", "f32")
    b = [g["logits"], _dev(g["temp"]), _dev(g["cu"]), _dev(g["drafts"]), _dev(g["accept"]), _dev(g["u"])]
    with pytest.raises(ValueError):
        dst.verify_logits(b[0].double(), *b[1:])
    with pytest.raises(ValueError):
        dst.verify_logits(*b, draft_probs=g["q"][:, :50])
    with pytest.raises(dst.TailError):
        dst.verify_logits(*b, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        dst.verify_logits(*b, workspace=torch.empty(1 << 20, dtype=torch.float32, device=DEV))


# ------------------------------------------------------------------ far below the chunk's largest

def _deep(z, temp, most=1.0):
    # per row: columns at 0 and -1 binary orders, one 1024-column segment of the same chunk at -59.03 to -59.97, the
    # rest below -75: integer weights of nothing, on either side of where exponentials are formed at all
    rng = np.random.default_rng(50)
    R, V = z.shape
    temp[:] = np.geomspace(0.05, most, R).astype(np.float32)
    unit = (temp.astype(np.float64) * np.log(2.0))[:, None]
    y = rng.uniform(-120.0, -75.0, (R, V))
    y[:, 4096:5120] = rng.uniform(-59.97, -59.03, (R, 1024))
    y[:, 5], y[:, 9] = 0.0, -1.0
    z[:] = (y * unit).astype(np.float32)


@pytest.mark.parametrize("accept", [0.0, 0.9])
@pytest.mark.parametrize("q", ["none", "f32"])
def test_logits_segments_without_weight_take_no_draw(q, accept):
    c = _logits_case(51, 24, 20000, "f32", q, edit=_deep)
    c["accept"][:] = accept
    c["drafts"][::2] = 5
    c["drafts"][1::2] = 9
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) >= 20


@pytest.mark.parametrize("l,q", [("f32", "none"), ("f32", "f32"), ("bf16", "bf16")])
def test_logits_peaked_rows_at_low_temperatures(l, q):
    def edit(z, temp):
        rng = np.random.default_rng(52)
        R, V = z.shape
        temp[:] = np.geomspace(0.05, 1.0, R).astype(np.float32)
        z[np.arange(R), rng.integers(0, V, R)] += rng.uniform(12.0, 30.0, R)
    c = _logits_case(53, 40, 50021, l, q, most=3, edit=edit)
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) >= 30
    lo, hi = c["cu"][:-1], c["cu"][1:]
    assert all(tokens[a + n - 1] >= 0 for a, b, n in zip(lo, hi, counts) if b > a)


@pytest.mark.parametrize("accept,most", [(0.5, 57.0), (0.0, 140.0)])
def test_logits_unlikely_drafts_are_judged_by_their_own_probability(accept, most):
    # P(x) = 2^-y / (1 + ..), u q above or below it by 2^-19.5 or zero: the largest column holds all but 2^-25 of the
    # row, so that the fp32 sum over the columns is off by less than 2^-22 and the draft's weight decides
    rng = np.random.default_rng(60)
    nseq, V = 400, 64
    R = 2 * nseq
    temp = rng.uniform(0.3, 1.5, R).astype(np.float32)
    z = np.full((R, V), -np.inf, np.float32)
    z[:, 3] = rng.uniform(-30.0, 30.0, R)
    y = rng.uniform(26.0, most, R)
    z[:, 40] = (z[:, 3] - y * temp * np.log(2.0)).astype(np.float32)
    e = np.exp((z[:, 40].astype(np.float64) - z[:, 3]) / temp)
    p = e / (1.0 + e)
    q = np.zeros((R, V), np.float32)
    q[:, 40] = 2.0 * p * (1.0 + np.where(np.arange(R) % 4 < 2, 1.0, -1.0) * 2.0 ** -19.5)
    c = dict(cu=np.arange(0, R + 1, 2, dtype=np.int32), R=R, V=V, logits=_dev(z), temp=temp,
             drafts=np.full(R, 40, np.int32), accept=np.full(R, accept, np.float32), u=rng.random(R, dtype=np.float32),
             q=_dev(q))
    tokens, counts = _logits_run(c)
    assert vc.compare(tokens, counts, _logits_want(c), c["cu"]) == nseq

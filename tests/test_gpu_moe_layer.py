"""The mixture-of-experts layer (tail_moe_run) on the GPU against 64 bits (tests/moecheck.py), and the steps it
belongs to: its slots through tail_run_moe, and layer -> tail -> draft verification in one graph."""
import numpy as np
import pytest

import gen
import oracle
from tests import moecheck as mc
from tests import tailcheck as tc
from tests import verifycheck as vc
from tests.test_gpu_parity import make_tail

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import decode_sampling_tail_gb300 as dst  # noqa: E402

DEV = torch.device("cuda:0")
CLAMPED = dict(act="glu", act_alpha=1.702, act_beta=1.0, act_limit=7.0, interleaved=True)
SILU = dict(act="glu", act_alpha=1.0, act_beta=0.0, act_limit=0.0, interleaved=False)
RELU2 = dict(act="relu2")


class Case:
    def __init__(self, T, H, I, E, topk, *, w="bf16", shared=0, act=CLAMPED, score="softmax", seed=0, bias=True,
                 gamma=True, router_bias=True, route_scale=1.0, t_max=None):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.T, self.H, self.I, self.E, self.topk, self.shared, self.w = T, H, I, E, topk, shared, w
        self.act, self.score, self.route_scale, self.t_max = act, score, route_scale, t_max or T
        n, N1 = E + shared, (2 * I if act["act"] == "glu" else I)

        def rnd(*shape, s=1.0):
            return s * torch.randn(shape, generator=g, device=DEV)

        self.x = (1.5 * rnd(T, H)).to(torch.bfloat16)
        self.gamma = 0.5 + torch.rand(H, generator=g, device=DEV) if gamma else None
        self.router_w = rnd(E, H, s=1.5 * H ** -0.5).to(torch.bfloat16)
        self.router_bias = rnd(E, s=0.1) if router_bias else None
        self.b1 = rnd(n, N1, s=0.2) if bias else None
        self.b2 = rnd(n, H, s=0.2) if bias else None
        self.s1 = self.s2 = None
        if w == "bf16":
            self.w1 = rnd(n, N1, H, s=H ** -0.5).to(torch.bfloat16)
            self.w2 = rnd(n, H, I, s=I ** -0.5).to(torch.bfloat16)
        else:
            def blocks(rows, cols):
                e = round(float(np.log2(cols ** -0.5 / 3.0)))
                b = torch.randint(0, 256, (n, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
                return b, torch.randint(125 + e, 130 + e, (n, rows, cols // 32), generator=g, device=DEV,
                                        dtype=torch.uint8)
            self.w1, self.s1 = blocks(N1, H)
            self.w2, self.s2 = blocks(H, I)

    def handle(self):
        return dst.Moe(self.H, self.I, self.E, self.topk, self.t_max, n_shared=self.shared, weight_dtype=self.w,
                       score=self.score, route_scale=self.route_scale, **self.act)

    def outputs(self):
        S = self.topk + self.shared
        nan = float("nan")
        return dict(out_hidden=torch.full((self.T, self.H), nan, dtype=torch.bfloat16, device=DEV),
                    out_slots=torch.full((self.T, S, self.H), nan, device=DEV),
                    out_slot_w=torch.full((self.T, S), nan, device=DEV),
                    out_ids=torch.full((self.T, S), -7, dtype=torch.int32, device=DEV))

    def run(self, m, out, x=None, **kw):
        m.run(self.x if x is None else x, self.gamma, self.router_w, self.w1, self.w2, router_bias=self.router_bias,
              w1_scale=self.s1, w2_scale=self.s2, b1=self.b1, b2=self.b2, **out, **kw)

    def want(self, x=None):
        x = self.x if x is None else x
        t, ids, w, gap = mc.route(x, self.gamma, self.router_w, self.router_bias, self.topk, self.shared, self.score,
                                  self.route_scale, 1e-5)
        a = self.act
        y, bound = mc.experts(t, ids, self.w1, self.s1, self.b1, self.w2, self.s2, self.b2, self.w, a["act"],
                              a.get("act_alpha", 1.0), a.get("act_beta", 0.0), a.get("act_limit", 0.0),
                              a.get("interleaved", False))
        return ids, w, gap, y, bound


def check(c, out, x=None):
    x = c.x if x is None else x
    ids, w, gap, y, bound = c.want(x)
    sure = gap > 1e-5
    assert sure.sum() >= 0.9 * len(gap) - 1
    got = {k: v for k, v in out.items()}
    assert torch.equal(got["out_ids"][sure].long(), ids[sure])
    assert ((got["out_slot_w"].double() - w).abs()[sure] <= 1e-5 * w.abs()[sure] + 1e-7).all()
    err = (got["out_slots"].double() - y).abs()[sure]
    assert (err <= bound[sure]).all(), f"{(err / bound[sure]).max().item():.3f} of the bound"
    # as a whole: the parts left out are independent, so their norm is about 2^-17 of the output's
    ref = y[sure].norm().item()
    assert err.norm().item() <= 2.0 ** -14 * max(ref, 1e-30), err.norm().item() / max(ref, 1e-30)
    h = oracle.moe_combine(x.view(torch.int16).cpu().numpy().view(np.uint16), got["out_slots"].cpu().numpy(),
                           got["out_slot_w"].cpu().numpy(), n_routed=c.topk)
    assert np.array_equal(got["out_hidden"].view(torch.int16).cpu().numpy().view(np.uint16), h)


def run_check(c):
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
        torch.cuda.synchronize()
    check(c, out)
    return out


# tokens from one to the most; widths of one k-step to many; groups of 1-4, 5-8 and 9-16 tokens an expert
SHAPES = [(1, 32, 32, 1, 1), (1, 2880, 2880, 8, 4), (2, 64, 96, 5, 2), (3, 256, 352, 33, 4), (4, 2080, 160, 6, 3),
          (5, 160, 2080, 4, 4), (7, 512, 512, 16, 2), (8, 96, 64, 2, 1), (13, 384, 1120, 12, 4), (16, 736, 416, 3, 2),
          (33, 320, 288, 7, 3), (64, 288, 320, 128, 8), (64, 128, 160, 1, 1), (31, 64, 64, 500, 16)]


@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,H,I,E,topk", SHAPES)
def test_layer_matches_64_bits(T, H, I, E, topk, w):
    run_check(Case(T, H, I, E, topk, w=w, seed=T + H))


@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
@pytest.mark.parametrize("act", ["clamped", "silu", "relu2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_layer_forms(w, act, score):
    a = {"clamped": CLAMPED, "silu": SILU, "relu2": RELU2}[act]
    run_check(Case(6, 288, 416, 24, 6, w=w, shared=2, act=a, score=score, seed=3, route_scale=2.5))


@pytest.mark.parametrize("act", [CLAMPED, RELU2])
def test_layer_16_column_widths(act):
    # bf16 rows that are whole 32-byte pieces but not whole k-steps
    run_check(Case(9, 16, 16, 3, 2, act=act, seed=4))
    run_check(Case(5, 48, 112, 4, 2, act=act, seed=5))


@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
def test_layer_without_norm_and_biases(w):
    run_check(Case(3, 256, 160, 9, 3, w=w, seed=6, gamma=False, bias=False, router_bias=False))
    run_check(Case(3, 256, 160, 9, 3, w=w, seed=7, bias=False, router_bias=False, score="sigmoid"))


@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
def test_layer_widest_rows(w):
    # too wide for many activation rows in shared memory: experts are passed over once a few tokens
    run_check(Case(9, 16384, 64, 2, 1, w=w, seed=8))
    run_check(Case(9, 64, 16384, 2, 2, w=w, seed=9, act=RELU2))


@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
def test_layer_ties_go_to_the_lower_expert(w):
    c = Case(5, 64, 32, 40, 7, w=w, seed=10, router_bias=False)
    c.router_w[:] = c.router_w[:1]  # every score equal
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
    assert out["out_ids"].tolist() == [list(range(7))] * 5
    assert torch.allclose(out["out_slot_w"], torch.full((5, 7), 1 / 7, device=DEV), rtol=1e-6)


def test_layer_large_and_small_activations():
    # fp16 parts are scaled a row at a time: rows 2^40 apart, a zero row
    c = Case(4, 256, 128, 2, 2, w="mxfp4", seed=11, gamma=False, bias=False, act=RELU2)
    c.x[1] *= 2.0 ** 20
    c.x[2] *= 2.0 ** -20
    c.x[3] = 0.0
    out = run_check(c)
    _, _, _, y, _ = c.want()
    for t in range(3):  # each row to its own size
        assert (out["out_slots"][t].double() - y[t]).norm() <= 2.0 ** -14 * y[t].norm()
    assert out["out_slots"][3].abs().max() == 0


def test_layer_block_scales_far_apart():
    # neighbouring blocks 2^40 apart, the smallest and the largest exponents
    c = Case(3, 512, 64, 2, 1, w="mxfp4", seed=12, gamma=False, bias=False, act=RELU2)
    c.s1[:, :, ::2] -= 40
    run_check(c)
    for e in (30, 200, -60):  # rows that end inside a k-step, scales far from the usual ones or from row to row
        c = Case(3, 160, 96, 2, 1, w="mxfp4", seed=19, gamma=False, bias=False, act=SILU, router_bias=False)
        if e > 0:
            c.s1[:] = c.s1 % 3 + e
            c.b1 = None
        else:
            c.s1[:, ::3] -= 60
        if e == 200:  # keep the products finite
            c.x *= 2.0 ** -80
        run_check(c)
    c = Case(2, 256, 64, 1, 1, w="mxfp4", seed=13, gamma=False, bias=False, act=SILU)
    c.s2[:] = 0
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
    assert out["out_slots"].abs().max() < 1e-30
    c.s2[0, 5, :] = 255
    with c.handle() as m:
        c.run(m, out)
    bad = torch.isnan(out["out_slots"])
    assert bad[:, :, 5].all() and bad.sum() == bad[:, :, 5].sum()


def test_layer_non_finite_tokens_stay_in_their_rows():
    for w in ("bf16", "mxfp4"):
        c = Case(6, 128, 96, 3, 2, w=w, seed=14, gamma=False)
        clean = run_check(c)
        c.x[2, 7] = float("inf")
        c.x[4, 3] = float("nan")
        out = c.outputs()
        with c.handle() as m:
            c.run(m, out)
        for t in (0, 1, 3, 5):
            assert torch.isfinite(out["out_slots"][t]).all()
            assert (out["out_slots"][t] - clean["out_slots"][t]).norm() <= 2.0 ** -14 * clean["out_slots"][t].norm()
        for t in (2, 4):
            assert not torch.isfinite(out["out_slots"][t]).all()
            assert ((out["out_ids"][t] >= 0) & (out["out_ids"][t] < 3)).all()


def test_layer_runs_again_in_place_and_on_other_streams():
    c = Case(12, 416, 288, 10, 4, w="mxfp4", shared=1, seed=15, t_max=20)
    ref = run_check(c)
    with c.handle() as m:
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        for stream in (None, side):
            for T in (12, 1, 20, 5, 12):  # other batches leave nothing behind
                x = c.x[:T] if T <= 12 else torch.cat((c.x, c.x[:8]))
                o = dict(out_hidden=torch.empty_like(x))
                c.run(m, o, x=x.contiguous(), stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(o["out_hidden"], ref["out_hidden"])
        x = c.x.clone()  # h may replace x
        c.run(m, dict(out_hidden=x), x=x)
        assert torch.equal(x, ref["out_hidden"])
        slots = torch.empty_like(ref["out_slots"])
        assert m.run(c.x, c.gamma, c.router_w, c.w1, c.w2, router_bias=c.router_bias, w1_scale=c.s1, w2_scale=c.s2,
                     b1=c.b1, b2=c.b2, out_slots=slots) is None
        assert torch.equal(slots, ref["out_slots"])
        h = m.run(c.x, c.gamma, c.router_w, c.w1, c.w2, router_bias=c.router_bias, w1_scale=c.s1, w2_scale=c.s2,
                  b1=c.b1, b2=c.b2)
        assert torch.equal(h, ref["out_hidden"])
        none = torch.empty((0, c.H), dtype=torch.bfloat16, device=DEV)
        assert m.run(none, c.gamma, c.router_w, c.w1, c.w2, router_bias=c.router_bias, w1_scale=c.s1, w2_scale=c.s2,
                     b1=c.b1, b2=c.b2).shape == (0, c.H)


def test_two_handles_run_side_by_side():
    # every CTA of a run wants a whole SM; runs of two handles share the device in any mix, eager and replayed
    cases = [Case(12, 416, 288, 10, 4, w="mxfp4", shared=1, seed=15), Case(5, 512, 384, 9, 3, seed=16)]
    want = [run_check(c)["out_hidden"] for c in cases]
    streams = [torch.cuda.Stream(DEV) for _ in cases]
    handles = [c.handle() for c in cases]
    outs = [[torch.empty_like(w) for _ in range(6)] for w in want]
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    torch.cuda.synchronize()
    for c, m, s, g, o in zip(cases, handles, streams, graphs, outs):
        with torch.cuda.graph(g, stream=s):
            for y in o[:3]:
                c.run(m, dict(out_hidden=y), stream=s)
    for _ in range(20):
        for c, m, s, g, o in zip(cases, handles, streams, graphs, outs):
            with torch.cuda.stream(s):
                g.replay()
            for y in o[3:]:
                c.run(m, dict(out_hidden=y), stream=s)
    torch.cuda.synchronize()
    for m, o, w in zip(handles, outs, want):
        m.check()
        assert all(torch.equal(y, w) for y in o)
        m.close()


def test_layer_nan_router_bias_stays_within_the_experts():
    # a NaN score ranks somewhere; the slots still name experts of the layer
    c = Case(6, 96, 64, 5, 2, seed=17)
    bits = torch.tensor([-1, 0x7fc00000, -1, -1, -1], dtype=torch.int32, device=DEV)
    c.router_bias = bits.view(torch.float32)
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
        torch.cuda.synchronize()
        m.check()
    assert ((out["out_ids"] >= 0) & (out["out_ids"] < 5)).all()


def test_layer_slots_feed_the_tails_producer_step():
    # slots and weights through tail_run_moe give the h, the top-k and the tokens of out_hidden through the tail
    w = gen.custom(6, 256, 8192, 32, hidden_dtype="bf16", seed=330)
    c = Case(6, 256, 192, 16, 6, shared=2, act=RELU2, score="sigmoid", seed=16)
    out = c.outputs()
    x, gamma, w_t, p = tc.to_device(w, torch)
    with c.handle() as m, make_tail(w) as t:
        c.run(m, out)
        tok = [torch.full((6,), -7, dtype=torch.int32, device=DEV) for _ in range(2)]
        tv = [torch.empty((6, 32), device=DEV) for _ in range(2)]
        ti = [torch.empty((6, 32), dtype=torch.int32, device=DEV) for _ in range(2)]
        h = torch.empty((6, 256), dtype=torch.bfloat16, device=DEV)
        t.run_moe(c.x, out["out_slots"], out["out_slot_w"], gamma, w_t, p, out_tokens=tok[0], out_topk_vals=tv[0],
                  out_topk_idx=ti[0], out_hidden=h, n_routed=6)
        t.run(out["out_hidden"], gamma, w_t, p, out_tokens=tok[1], out_topk_vals=tv[1], out_topk_idx=ti[1])
        torch.cuda.synchronize()
        t.check()
    assert torch.equal(h, out["out_hidden"])
    assert torch.equal(tok[0], tok[1]) and torch.equal(tv[0], tv[1]) and torch.equal(ti[0], ti[1])


@pytest.mark.parametrize("path", ["gemv", "tensor"])
def test_speculative_step_layer_tail_and_verification_in_one_graph(path):
    # two sequences of drafted rows: MoE layer -> tail (top-k, logits) -> both verifications, captured and replayed
    B, H, V, k = 7, 256, 8192, 32
    w = gen.custom(B, H, V, k, hidden_dtype="bf16", seed=331)
    c = Case(B, H, 160, 12, 4, w="mxfp4", seed=17)
    _, gamma, w_t, p = tc.to_device(w, torch)
    rng = np.random.default_rng(9)
    cu = np.array([0, 4, 7], np.int32)
    accept, u = rng.random(B, dtype=np.float32), rng.random(B, dtype=np.float32)
    dev = dict(cu=torch.from_numpy(cu).to(DEV), accept=torch.from_numpy(accept).to(DEV),
               u=torch.from_numpy(u).to(DEV), temp=torch.full((B,), 0.8, device=DEV),
               drafts=torch.full((B,), -1, dtype=torch.int32, device=DEV))
    h = torch.empty((B, H), dtype=torch.bfloat16, device=DEV)
    logits = torch.empty((B, V), device=DEV)
    tv, ti = torch.empty((B, k), device=DEV), torch.empty((B, k), dtype=torch.int32, device=DEV)
    o = [torch.full((B,), -7, dtype=torch.int32, device=DEV) for _ in range(2)]
    n = [torch.empty(2, dtype=torch.int32, device=DEV) for _ in range(2)]
    ws = torch.empty(dst.verify_logits_workspace(B, 2, V), dtype=torch.uint8, device=DEV)
    with c.handle() as m, make_tail(w, path=path) as t:
        def step():
            c.run(m, dict(out_hidden=h))
            t.run(h, gamma, w_t, None, out_logits=logits, out_topk_vals=tv, out_topk_idx=ti)
            dst.verify(tv, ti, p, dev["cu"], dev["drafts"], dev["accept"], out_tokens=o[0], out_count=n[0])
            dst.verify_logits(logits, dev["temp"], dev["cu"], dev["drafts"], dev["accept"], dev["u"], out_tokens=o[1],
                              out_count=n[1], workspace=ws)
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        likely = ti[:, 0].clone()
        for drafts in (likely, ti[:, 1].clone(), torch.full_like(likely, -1)):
            dev["drafts"].copy_(drafts)
            h.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            t.check()
            d = drafts.cpu().numpy()
            v, i, prm, L = (a.cpu().numpy() for a in (tv, ti, p, logits))
            full = lambda row, ids: None  # noqa: E731
            want = vc.settle(cu, d, accept, prm[:, 3], lambda r: vc.sampler_target(v[r], i[r], prm[r]), full, B)
            vc.compare(o[0].cpu().numpy(), n[0].cpu().numpy(), want, cu)
            want = vc.settle(cu, d, accept, u, lambda r: (vc.softmax_target(L[r], np.float32(0.8)), 1.0), full, B)
            vc.compare(o[1].cpu().numpy(), n[1].cpu().numpy(), want, cu)
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
    check(c, out)
    assert torch.equal(h, out["out_hidden"])


def test_wrapper_refuses_what_does_not_fit():
    c = Case(3, 64, 32, 4, 2, w="mxfp4", seed=18)
    with c.handle() as m:
        good = dict(router_bias=c.router_bias, w1_scale=c.s1, w2_scale=c.s2, b1=c.b1, b2=c.b2)
        args = [c.x, c.gamma, c.router_w, c.w1, c.w2]
        for i, bad in ((0, c.x.float()), (0, c.x[:, :32]), (0, torch.cat((c.x, c.x))), (0, c.x.cpu()),
                       (1, c.gamma.double()), (2, c.router_w[:3]), (3, c.w1.view(torch.int8)), (4, c.w2[:, :, :8]),
                       (2, c.router_w.t().contiguous().t())):
            with pytest.raises(ValueError):
                m.run(*[bad if j == i else a for j, a in enumerate(args)], **good)
        for key, bad in (("w1_scale", None), ("w2_scale", c.s1), ("b1", c.b2[:, :32]), ("router_bias", c.gamma),
                         ("out_slots", torch.empty((3, 2, 32), device=DEV)),
                         ("out_ids", torch.empty((3, 2), dtype=torch.int64, device=DEV))):
            with pytest.raises(ValueError):
                m.run(*args, **{**good, key: bad})
    with pytest.raises(ValueError):
        m.run(*args, **good)  # closed
    b = Case(3, 64, 32, 4, 2, seed=18)
    with b.handle() as m, pytest.raises(ValueError):
        m.run(b.x, b.gamma, b.router_w, b.w1, b.w2, w1_scale=c.s1, w2_scale=c.s2)
    for kw in (dict(H=40), dict(H=16400), dict(E=600), dict(topk=17), dict(t_max=65), dict(n_shared=9)):
        with pytest.raises(dst.TailError):
            dst.Moe(**{**dict(H=64, I=64, E=32, topk=2, t_max=4), **kw})


@pytest.mark.parametrize("T,shared", [(2, 0), (3, 0), (4, 0), (13, 1)])
def test_layer_rows_whose_largest_value_is_a_power_of_two(T, shared):
    # 4-bit rows are scaled by a power of two of their largest |t|; neighbouring fp32 gammas carry that value over one
    for seed in range(4):
        c = Case(T, 2880, 32, 4, 2, w="mxfp4", shared=shared, act=RELU2, seed=100 + seed)
        c.gamma[:] = 1.0
        x = c.x.double()
        at = x.abs().argmax(-1)
        while len(set(at.tolist())) < T:  # a column of its own for each token
            c.x[torch.arange(T, device=DEV), at] = 0.0
            x = c.x.double()
            at = x.abs().argmax(-1)
        rms = torch.sqrt((x * x).mean(-1) + 1e-5)
        top = (16.0 * rms / x[torch.arange(T, device=DEV), at].abs()).float()
        m = c.handle()
        for step in range(-24, 25):
            c.gamma[at] = (top.view(torch.int32) + step).view(torch.float32)
            out = c.outputs()
            c.run(m, out)
            ids, _, gap, y, bound = c.want()
            sure = gap > 1e-5
            err = (out["out_slots"].double() - y).abs()
            assert (err <= bound)[sure].all(), (seed, step, ((err / bound).amax((1, 2)) > 1).tolist())
        m.close()


@pytest.mark.parametrize("T,H,I,E,topk,shared", [(1, 14368, 32, 2, 1, 0), (2, 16352, 32, 2, 1, 0), (9, 32, 16352, 3, 2, 0),
                                                (64, 11296, 32, 16, 16, 0), (64, 16352, 32, 17, 16, 8)])
def test_layer_widest_rows_of_an_odd_number_of_blocks(T, H, I, E, topk, shared):
    run_check(Case(T, H, I, E, topk, w="mxfp4", shared=shared, act=RELU2, seed=40))


@pytest.mark.parametrize("bias", [False, True])
def test_layer_sigmoid_weights_of_scores_that_underflow(bias):
    # z of about -96: sigmoid(z) is no fp32 number, its share of the sum is.  z is off by at most 13 half-steps of
    # 2^-18 (8 products a lane, 5 additions), so a share by twice that
    c = Case(5, 64, 32, 12, 4, act=RELU2, score="sigmoid", seed=43, gamma=False, router_bias=bias)
    c.x[:, 0], c.router_w[:, 0] = 16.0, -6.0
    if bias:
        c.router_bias = torch.linspace(0.1, 0.9, 12, device=DEV)
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
    ids, w, gap, _, _ = c.want()
    sure = gap > 1e-5
    assert sure.sum() >= 4 and torch.equal(out["out_ids"][sure].long(), ids[sure])
    assert ((out["out_slot_w"].double() - w).abs()[sure] <= 2 * 13 * 2.0 ** -18 * w[sure] + 2.0 ** -22).all()
    assert torch.isfinite(out["out_hidden"]).all()


@pytest.mark.parametrize("H", [512, 160])
@pytest.mark.parametrize("apart", [16, 23, 24, 26, 40, 100])
def test_layer_large_blocks_that_meet_zeros_hide_no_small_ones(H, apart):
    # every other block of W1 is 2^apart times its neighbours and meets activations of zero: the small ones are the sum
    c = Case(3, H, 64, 2, 1, w="mxfp4", seed=41, gamma=False, bias=False, act=SILU, router_bias=False)
    c.s1[:, ::2, ::2] -= apart
    c.s1[:, 1::2, 1::2] -= apart  # the up rows hold their small blocks elsewhere
    c.x.view(3, -1, 32)[0, 1::2] = 0.0
    c.x.view(3, -1, 32)[1, ::2] = 0.0
    run_check(c)
    # blocks of 4 sizes in one step of a row, the largest all zeros, and a block that holds no value
    c = Case(3, H, 64, 2, 1, w="mxfp4", seed=42, gamma=False, bias=False, act=RELU2, router_bias=False)
    for i in range(4):
        c.s1[:, :, i::4] -= (i * apart) // 3
    c.x.view(3, -1, 32)[:, 0::4] = 0.0
    c.w1.view(2, 64, -1, 16)[:, :, 1::4] = 0
    c.s1[:, ::3, 1::4] = 0
    run_check(c)


@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_layer_waits_that_run_out_are_reported_and_recoverable(T, w):
    # at a limit of 1 ns every wait that is not over at its first look runs out: each run reports it, ends, and leaves
    # the handle as it was
    c = Case(T, 512, 416, 12, 4, w=w, shared=1, seed=44)
    want = run_check(c)
    out = c.outputs()
    with c.handle() as m:
        c.run(m, out)
        m.check()
        for _ in range(3):
            m.set_wait_limit(1)
            c.run(m, out)
            c.run(m, out)
            with pytest.raises(dst.TailError) as e:
                m.check()
            assert e.value.args and dst.lib().tail_moe_check(m.h) == dst.TAIL_OK  # the word was cleared
            m.set_wait_limit(1_000_000_000)
            out = c.outputs()
            c.run(m, out)
            m.check()
            assert all(torch.equal(out[k], want[k]) for k in out)


def test_layer_refuses_outputs_over_inputs_and_each_other():
    c = Case(3, 64, 32, 4, 2, w="mxfp4", shared=1, seed=45)
    o = c.outputs()
    arena = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)

    def at(byte, like):
        return arena[byte:byte + like.numel() * like.element_size()].view(like.dtype).view(like.shape)

    def moved(**kw):  # a case with one input in the arena, at byte 4096
        d = Case(3, 64, 32, 4, 2, w="mxfp4", shared=1, seed=45)
        for k in kw:
            setattr(d, k, at(4096, getattr(d, k)).copy_(getattr(d, k)))
        return d

    with c.handle() as m:
        for name, like in o.items():
            size, step = like.numel() * like.element_size(), 16
            for k in ("x", "gamma", "router_w", "router_bias", "w1", "s1", "b1", "w2", "s2", "b2"):
                d = moved(**{k: 1})
                n = getattr(d, k).numel() * getattr(d, k).element_size()
                for byte in (4096 - size // step * step + step, 4096 + (n - 1) // step * step):
                    if not 4096 - size < byte < 4096 + n:
                        continue
                    with pytest.raises(dst.TailError) as e:
                        d.run(m, {**o, name: at(byte, like)})
                    assert e.value.status == dst.TAIL_ERR_INVALID_ARG
            for other in o:
                if other != name:
                    with pytest.raises(dst.TailError):
                        c.run(m, {**o, name: at(8192, like), other: at(8192, o[other])})
        d = moved(x=1)  # side by side, and h in place of x, are allowed
        x = d.x.clone()
        out = {k: at(16384 + 8192 * i, v) for i, (k, v) in enumerate(o.items()) if k != "out_hidden"}
        d.run(m, {**out, "out_hidden": d.x})
        torch.cuda.synchronize()
        check(c, {**{k: v.clone() for k, v in out.items()}, "out_hidden": d.x}, x=x)

"""Operators of a speculative decode step's end, measured: their cases, inputs, plain forms and exact values.

  verify          drafted tokens against the tail's sorted top-k and its sampler
  verify_logits   drafted tokens against the softmax of whole-vocabulary logits
  moe             a mixture-of-experts layer for a few tokens (norm, router, experts, combine, residual)

A speculative step runs the last MoE layer and the tail on the rows of the drafted positions (a sequence with d
drafts has d + 1 rows) and then verifies the drafts.  Formulas, for a sequence's rows j = 0 .. d with target
distributions P_j, draft distributions q_j (one-hot when absent), drafts x_j and uniforms a_j, u_j:

  draft j is accepted iff a_j q_j(x_j) < P_j(x_j) and every draft before it was;
  at the first refused row j the token is the smallest i with u_j R < sum_{i' <= i} r_i', r = max(P_j - q_j, 0),
  R = sum r (r = P_j when R = 0); with every draft accepted it is drawn from P_d the same way;
  the sequence's tokens are the accepted drafts, that token, then -1.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one chat session, three drafts by a lookup (no draft probabilities): the latency of the check itself
        dict(name="verify_one", op="verify", nseq=1, dmin=3, dmax=3, pad=0, V=201088, k=256, q="none", cols=4),
        # a full decode batch of a small draft model: 64 sequences with five drafts each
        dict(name="verify_batch", op="verify", nseq=64, dmin=5, dmax=5, pad=0, V=201088, k=256, q="bf16", cols=4),
        # a large ragged batch padded to a fixed number of rows, long lists
        dict(name="verify_ragged", op="verify", nseq=200, dmin=0, dmax=9, pad=24, V=32000, k=1000, q="f32", cols=4),
        # one session, the whole vocabulary, lookup drafts
        dict(name="logits_one", op="verify_logits", nseq=1, dmin=4, dmax=4, pad=0, V=201088, l="f32", q="none"),
        # a small batch with a draft model, on the tail's fp32 logits
        dict(name="logits_batch", op="verify_logits", nseq=16, dmin=3, dmax=3, pad=0, V=201088, l="f32", q="bf16"),
        # an odd vocabulary, 16-bit logits, ragged drafts, rows left over
        dict(name="logits_odd", op="verify_logits", nseq=37, dmin=0, dmax=7, pad=5, V=50021, l="bf16", q="f16"),
        # a large batch
        dict(name="logits_large", op="verify_logits", nseq=96, dmin=2, dmax=4, pad=0, V=201088, l="f32", q="f32"),
        # one token through a wide layer in 4-bit weights: the latency of a decode step
        dict(name="moe_one_mxfp4", op="moe", T=1, H=2880, I=2880, E=128, topk=4, shared=0, w="mxfp4", act="clamped",
             score="softmax"),
        # one sequence's drafted positions in 16 bits
        dict(name="moe_few_bf16", op="moe", T=5, H=2880, I=2880, E=32, topk=4, shared=0, w="bf16", act="clamped",
             score="softmax"),
        # a small batch in 4-bit weights
        dict(name="moe_batch_mxfp4", op="moe", T=16, H=2880, I=2880, E=128, topk=4, shared=0, w="mxfp4",
             act="clamped", score="softmax"),
        # sigmoid router, six routed and two shared experts without a gate
        dict(name="moe_shared_bf16", op="moe", T=8, H=2688, I=1856, E=64, topk=6, shared=2, w="bf16", act="relu2",
             score="sigmoid"),
        # the largest batch the operator is for: nearly every expert is read
        dict(name="moe_large_bf16", op="moe", T=64, H=2880, I=2880, E=128, topk=4, shared=0, w="bf16", act="silu",
             score="softmax"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["verify", "verify_logits", "moe", "moe"])
    if op == "verify":
        dmin = rng.randint(0, 3)
        V = 16 * _log_int(rng, 64, 12568)
        return dict(op=op, nseq=_log_int(rng, 1, 256), dmin=dmin, dmax=dmin + rng.randint(0, 6),
                    pad=rng.choice([0, 0, rng.randint(1, 30)]), V=V, k=_log_int(rng, 1, min(V, 1024)),
                    q=rng.choice(["none", "f32", "f16", "bf16"]), cols=rng.choice([3, 4, 4, 4]))
    if op == "verify_logits":
        dmin = rng.randint(0, 3)
        V = _log_int(rng, 300, 201088)
        return dict(op=op, nseq=_log_int(rng, 1, 64), dmin=dmin, dmax=dmin + rng.randint(0, 2),
                    pad=rng.choice([0, 0, rng.randint(1, 9)]), V=V, l=rng.choice(["f32", "f32", "f16", "bf16"]),
                    q=rng.choice(["none", "f32", "f16", "bf16"]))
    E = rng.choice([8, 16, 32, 48, 64, 96])
    topk = rng.randint(1, min(8, E))
    shared = rng.choice([0, 0, 1, 2])
    H, I = 32 * _log_int(rng, 8, 90), 32 * _log_int(rng, 8, 90)
    return dict(op=op, T=_log_int(rng, 1, 64), H=H, I=I, E=E, topk=topk, shared=shared,
                w=rng.choice(["bf16", "mxfp4"]), act=rng.choice(["clamped", "silu", "relu2"]),
                score=rng.choice(["softmax", "sigmoid"]))


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(case, seed):
    """Row starts of the sequences ([nseq + 1]) and the number of rows, some of them behind the last sequence.  The
    case fixes the drafts' numbers, the seed their order."""
    span = case["dmax"] - case["dmin"] + 1
    n = 1 + case["dmin"] + np.random.default_rng(seed).permutation(np.arange(case["nseq"]) * 5 % span)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return cu, int(cu[-1]) + case["pad"]


def _params(case, R, seed):
    """Sampling parameters as serving sees them: mostly drawn, some greedy, top_p and top_k on and off."""
    r = np.random.default_rng(seed + 1)
    p = np.empty((R, 4), np.float32)
    p[:, 0] = r.choice([0, 1, 20, 50, 10 ** 6], R, p=[0.25, 0.05, 0.25, 0.25, 0.2])
    p[:, 1] = np.where(r.random(R) < 0.4, 1.0, r.uniform(0.5, 0.99, R))
    p[:, 2] = np.where(r.random(R) < 0.15, 0.0, r.uniform(0.4, 1.4, R))
    p[:, 3] = r.random(R, dtype=np.float32)
    return p


def _draft_probs(logits, g, dtype):
    """A draft model's distribution: the target's logits with noise on them."""
    z = logits.float()
    return torch.softmax(z + 0.7 * torch.randn(z.shape, generator=g, device=DEV), dim=-1).to(DTYPES[dtype])


def _sample(p, g):
    """One token a row from the rows of p (exponential races)."""
    e = torch.empty(p.shape, device=DEV).exponential_(generator=g)
    return torch.argmax(p.float() / e, dim=-1).to(torch.int32)


def _prepare_verify(case, seed):
    g = _gen(seed)
    cu, R = _rows(case, seed)
    V, k = case["V"], case["k"]
    vals = torch.sort(2.5 * torch.randn((R, k), generator=g, device=DEV) + 6.0, dim=-1, descending=True).values
    step = next(s for s in (7919, 104729, 1009, 1) if math.gcd(s, V) == 1)
    start = torch.randint(0, V, (R, 1), generator=g, device=DEV)
    idx = ((start + step * torch.arange(k, device=DEV)) % V).to(torch.int32)
    q = None
    if case["q"] == "none":
        pick = _sample(torch.softmax(vals, dim=-1), g).long()
        drafts = torch.gather(idx, 1, pick[:, None])[:, 0]
    else:
        full = torch.randn((R, V), generator=g, device=DEV) - 8.0
        full.scatter_(1, idx.long(), vals)
        q = _draft_probs(full, g, case["q"])
        drafts = _sample(q, g)
    params = torch.from_numpy(_params(case, R, seed)).to(DEV)[:, :case["cols"]].contiguous()
    return dict(case=case, vals=vals, idx=idx, params=params, cu=torch.from_numpy(cu).to(DEV),
                drafts=drafts.contiguous(), q=q, accept=torch.rand(R, generator=g, device=DEV),
                tokens=torch.full((R,), -7, dtype=torch.int32, device=DEV),
                count=torch.full((case["nseq"],), -7, dtype=torch.int32, device=DEV))


def _prepare_logits(case, seed):
    g = _gen(seed)
    cu, R = _rows(case, seed)
    V = case["V"]
    logits = 2.2 * torch.randn((R, V), generator=g, device=DEV)
    peaks = torch.randint(0, V, (R, 24), generator=g, device=DEV)  # what the context makes likely
    logits.scatter_add_(1, peaks, 4.0 + 4.0 * torch.rand((R, 24), generator=g, device=DEV))
    logits = logits.to(DTYPES[case["l"]])
    if case["q"] == "none":
        q, drafts = None, _sample(torch.softmax(logits.float(), dim=-1), g)
    else:
        q = _draft_probs(logits, g, case["q"])
        drafts = _sample(q, g)
    p = torch.from_numpy(_params(case, R, seed)).to(DEV)
    s = dict(case=case, logits=logits, q=q, drafts=drafts, cu=torch.from_numpy(cu).to(DEV),
             temperature=p[:, 2].contiguous(), draw=p[:, 3].contiguous(),
             accept=torch.rand(R, generator=g, device=DEV),
             tokens=torch.full((R,), -7, dtype=torch.int32, device=DEV),
             count=torch.full((case["nseq"],), -7, dtype=torch.int32, device=DEV))
    if own:
        import decode_sampling_tail_gb300 as dst
        s["workspace"] = torch.empty(dst.verify_logits_workspace(R, case["nseq"], V), dtype=torch.uint8, device=DEV)
    return s


def _gated(case):
    return case["act"] != "relu2"


def _act_args(case):
    """(alpha, beta, limit) of glu * sigmoid(alpha glu) * (up + beta); limit 0: no clamp."""
    return (1.702, 1.0, 7.0) if case["act"] == "clamped" else (1.0, 0.0, 0.0)


def _weight(case, g, n, rows, cols):
    """n matrices [rows, cols] of entries of about 1 / sqrt(cols): bf16, or 4-bit blocks of 32 with their scales."""
    if case["w"] == "bf16":
        return torch.empty((n, rows, cols), dtype=torch.bfloat16, device=DEV).normal_(0, cols ** -0.5, generator=g), None
    blocks = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=DEV).random_(0, 256, generator=g)
    e = round(math.log2(cols ** -0.5 / 3.0))
    scales = torch.randint(127 + e - 1, 127 + e + 2, (n, rows, cols // 32), generator=g, device=DEV, dtype=torch.uint8)
    return blocks, scales


def _prepare_moe(case, seed):
    g = _gen(seed)
    T, H, I, E, n = case["T"], case["H"], case["I"], case["E"], case["E"] + case["shared"]
    N1 = 2 * I if _gated(case) else I
    s = dict(case=case)
    s["x"] = (1.5 * torch.randn((T, H), generator=g, device=DEV)).to(torch.bfloat16)
    s["gamma"] = 0.5 + torch.rand(H, generator=g, device=DEV)
    s["router_w"] = (torch.randn((E, H), generator=g, device=DEV) * (1.5 * H ** -0.5)).to(torch.bfloat16)
    s["router_b"] = 0.1 * torch.randn(E, generator=g, device=DEV)
    s["w1"], s["s1"] = _weight(case, g, n, N1, H)
    s["w2"], s["s2"] = _weight(case, g, n, H, I)
    s["b1"] = 0.1 * torch.randn((n, N1), generator=g, device=DEV)
    s["b2"] = 0.1 * torch.randn((n, H), generator=g, device=DEV)
    S = case["topk"] + case["shared"]
    s["hidden"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    s["ids"] = torch.empty((T, S), dtype=torch.int32, device=DEV)
    s["slot_w"] = torch.empty((T, S), dtype=torch.float32, device=DEV)
    if own:
        s["moe"] = _handle(case)
    return s


def _handle(case):
    import decode_sampling_tail_gb300 as dst
    alpha, beta, limit = _act_args(case)
    return dst.Moe(case["H"], case["I"], case["E"], case["topk"], t_max=case["T"], n_shared=case["shared"],
                   weight_dtype=case["w"], act="glu" if _gated(case) else "relu2", act_alpha=alpha, act_beta=beta,
                   act_limit=limit, interleaved=case["act"] == "clamped", score=case["score"],
                   route_scale=2.5 if case["score"] == "sigmoid" else 1.0)


def prepare(case, seed):
    return {"verify": _prepare_verify, "verify_logits": _prepare_logits, "moe": _prepare_moe}[case["op"]](case, seed)


# --------------------------------------------------------------------------- plain forms

def _settle(s, P, q, order_ids, accept, draw):
    """Tokens and counts from the target probabilities P [R, n] (64 bits; column c stands for token order_ids[:, c],
    or for token c where that is None), and the draft probabilities q of the same columns and of the drafts."""
    R, nseq = P.shape[0], s["count"].shape[0]
    q_cols, q_draft, p_draft = q
    row = torch.arange(R, device=DEV)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, row, right=True) - 1
    live = row < cu[-1]
    seq = torch.where(live, seq, 0).clamp_(max=nseq - 1)
    last = row == cu[seq + 1] - 1
    refused = ~(accept.double() * q_draft < p_draft) & ~last
    stop = (refused | last) & live
    sel = torch.full((nseq,), R, dtype=torch.int64, device=DEV)
    sel.scatter_reduce_(0, seq, torch.where(stop, row, R), "amin")
    has = sel < R
    at = torch.where(has, sel, 0)
    Ps = P[at]
    res = torch.clamp(Ps - q_cols(at), min=0.0)
    use = refused[at] & (res.sum(-1) > 0)
    r = torch.where(use[:, None], res, Ps)
    C = torch.cumsum(r, -1)
    hit = C > (draw[at].double() * C[:, -1])[:, None]
    n = P.shape[1]
    col = torch.arange(n, device=DEV)
    first = torch.where(hit & (r > 0), col, n).amin(-1)
    final = torch.where(r > 0, col, -1).amax(-1)
    pick = torch.where(first < n, first, final)
    token = pick if order_ids is None else torch.gather(order_ids[at].long(), 1, pick.clamp(min=0)[:, None])[:, 0]
    out = s["tokens"].long()
    mine = torch.where(live, sel[seq], R)
    out = torch.where(live, torch.where(row < mine, s["drafts"].long(), torch.where(row == mine, token[seq], -1)), out)
    count = torch.where(has, sel - cu[:-1] + 1, 0)
    return out.to(torch.int32), count.to(torch.int32)


def _plain_verify(s):
    case, vals, idx, prm = s["case"], s["vals"].double(), s["idx"].long(), s["params"].double()
    R, k = vals.shape
    top_k, top_p, temp = prm[:, 0], prm[:, 1], prm[:, 2]
    draw = prm[:, 3] if case["cols"] == 4 else torch.full_like(temp, 0.5)
    kk = torch.where((top_k >= 1) & (top_k < k + 1), torch.floor(top_k), float(k))
    col = torch.arange(k, device=DEV)
    greedy = ~(temp > 0) | (kk == 1)
    e = torch.exp((vals - vals[:, :1]) / torch.where(greedy, 1.0, temp)[:, None]) * (col < kk[:, None])
    e = torch.where(greedy[:, None], (col == 0).double(), e)
    C = torch.cumsum(e, -1)
    short = (C < top_p[:, None] * C[:, -1:]).sum(-1)  # candidates before the one that reaches top_p
    m = torch.where(top_p < 1, short + 1.0, kk)
    P = e * (col < m[:, None])
    P = P / P.sum(-1, keepdim=True)
    x = s["drafts"].long()
    hit = idx == x[:, None]
    p_draft = torch.where(hit, P, 0.0).sum(-1)
    if s["q"] is None:
        q = (lambda at: hit[at].double(), torch.ones_like(p_draft), p_draft)
    else:
        q = (lambda at: torch.gather(s["q"][at], 1, idx[at]).double(),
             torch.gather(s["q"], 1, x[:, None])[:, 0].double(), p_draft)
    return _settle(s, P, q, s["idx"], s["accept"], draw)


def _plain_logits(s):
    z = s["logits"].double()
    R, V = z.shape
    m = z.amax(-1, keepdim=True)
    temp = s["temperature"].double()
    greedy = ~(temp > 0)
    col = torch.arange(V, device=DEV)
    best = torch.where(z == m, col, V).amin(-1)
    e = torch.exp((z - m) / torch.where(greedy, 1.0, temp)[:, None])
    P = torch.where(greedy[:, None], (col == best[:, None]).double(), e / e.sum(-1, keepdim=True))
    x = s["drafts"].long()
    p_draft = torch.gather(P, 1, x[:, None])[:, 0]
    if s["q"] is None:
        q = (lambda at: (col == x[at][:, None]).double(), torch.ones_like(p_draft), p_draft)
    else:
        q = (lambda at: s["q"][at].double(), torch.gather(s["q"], 1, x[:, None])[:, 0].double(), p_draft)
    return _settle(s, P, q, None, s["accept"], s["draw"])


def _widen(w, scale, ids):
    """The matrices `ids` of a weight in 32 bits."""
    if scale is None:
        return w[ids].float()
    b = w[ids].int()
    lut = torch.tensor(FP4, device=DEV)
    v = lut[torch.stack((b & 15, b >> 4), -1).flatten(-2)]
    sc = torch.exp2(scale[ids].float() - 127.0)
    return (v.unflatten(-1, (-1, 32)) * sc[..., None]).flatten(-2)


def _plain_moe(s):
    case = s["case"]
    T, E, k, shared = case["T"], case["E"], case["topk"], case["shared"]
    x = s["x"].float()
    t = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * s["gamma"]
    # 64 bits: the selection compares logits that may lie close together
    xd = s["x"].double()
    td = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-5) * s["gamma"].double()
    logit = td @ s["router_w"].double().T
    rank = torch.sigmoid(logit) + s["router_b"].double() if case["score"] == "sigmoid" else logit + s["router_b"].double()
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :k]
    if case["score"] == "sigmoid":
        sc = torch.sigmoid(torch.gather(logit, 1, ids))
        wt = 2.5 * sc / sc.sum(-1, keepdim=True)
    else:
        wt = torch.softmax(torch.gather(rank, 1, ids), dim=-1)
    if shared:
        ids = torch.cat((ids, torch.arange(E, E + shared, device=DEV).expand(T, shared)), 1)
        wt = torch.cat((wt, torch.ones((T, shared), dtype=wt.dtype, device=DEV)), 1)
    wt = wt.float()
    alpha, beta, limit = _act_args(case)
    out = torch.empty_like(s["hidden"])
    for i in range(T):
        h = torch.matmul(_widen(s["w1"], s["s1"], ids[i]), t[i]) + s["b1"][ids[i]]
        if not _gated(case):
            a = torch.clamp(h, min=0.0) ** 2
        else:
            gate, up = (h[:, 0::2], h[:, 1::2]) if case["act"] == "clamped" else h.chunk(2, dim=-1)
            if limit > 0:
                gate, up = torch.clamp(gate, max=limit), torch.clamp(up, -limit, limit)
            a = gate * torch.sigmoid(alpha * gate) * (up + beta)
        y = torch.matmul(_widen(s["w2"], s["s2"], ids[i]), a[:, :, None])[:, :, 0] + s["b2"][ids[i]]
        out[i] = (x[i] + (wt[i][:, None] * y).sum(0)).to(torch.bfloat16)
    return out, ids.to(torch.int32), wt


# --------------------------------------------------------------------------- the framework's calls

def _own(s):
    import decode_sampling_tail_gb300 as dst
    case = s["case"]
    if case["op"] == "verify":
        return dst.verify(s["vals"], s["idx"], s["params"], s["cu"], s["drafts"], s["accept"], draft_probs=s["q"],
                          out_tokens=s["tokens"], out_count=s["count"])
    if case["op"] == "verify_logits":
        return dst.verify_logits(s["logits"], s["temperature"], s["cu"], s["drafts"], s["accept"], s["draw"],
                                 draft_probs=s["q"], out_tokens=s["tokens"], out_count=s["count"],
                                 workspace=s.get("workspace"))
    if "moe" not in s:
        s["moe"] = _handle(case)
    s["moe"].run(s["x"], s["gamma"], s["router_w"], s["w1"], s["w2"], router_bias=s["router_b"], w1_scale=s["s1"],
                 w2_scale=s["s2"], b1=s["b1"], b2=s["b2"], out_hidden=s["hidden"], out_ids=s["ids"],
                 out_slot_w=s["slot_w"])
    return s["hidden"], s["ids"], s["slot_w"]


def run(state):
    if own:
        return _own(state)
    return {"verify": _plain_verify, "verify_logits": _plain_logits, "moe": _plain_moe}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass.  Draft probabilities are read at the drafts and, for one row a sequence,
    at every candidate; an expert is read once when any token selects it (their expected number)."""
    size = {"none": 0, "f32": 4, "f16": 2, "bf16": 2}
    if case["op"] == "moe":
        T, H, I, E, k, sh = (case[n] for n in ("T", "H", "I", "E", "topk", "shared"))
        N1 = 2 * I if _gated(case) else I
        read = E * (1.0 - (1.0 - k / E) ** T) + sh
        per = (N1 * H + H * I) * (2.0 if case["w"] == "bf16" else 0.5 + 1 / 32) + 4 * (N1 + H)
        return {"bytes": read * per + 2 * E * H + 4 * H + 4 * E + 4 * T * H + 8 * T * (k + sh),
                "flops": 2.0 * T * ((k + sh) * (N1 * H + H * I) + E * H)}
    nseq = case["nseq"]
    rows = nseq * (1 + 0.5 * (case["dmin"] + case["dmax"]))
    small = rows * (4 + 4 + 4 + size[case["q"]]) + 8 * nseq
    if case["op"] == "verify":
        return {"bytes": small + rows * (8 * case["k"] + 4 * case["cols"]) + nseq * case["k"] * size[case["q"]],
                "flops": 8.0 * rows * case["k"]}
    return {"bytes": small + 8 * rows + rows * case["V"] * size[case["l"]] + nseq * case["V"] * size[case["q"]],
            "flops": 6.0 * rows * case["V"]}


# --------------------------------------------------------------------------- exact values

def _exact_tokens(case, s, target, ids):
    """Sequence by sequence: target(row) gives the row's probabilities, ids(row) the tokens they belong to."""
    cu, x, a = s["cu"].cpu().numpy(), s["drafts"].cpu().numpy(), s["accept"].cpu().numpy().astype(np.float64)
    tokens, count = s["tokens"].cpu().numpy().copy(), np.zeros(case["nseq"], np.int32)

    def draft(row, tok):
        if s["q"] is None:
            return (np.asarray(tok) == x[row]).astype(np.float64)
        return s["q"][row].double().cpu().numpy()[tok]

    for i in range(case["nseq"]):
        lo, hi = int(cu[i]), int(cu[i + 1])
        tokens[lo:hi] = -1
        for j in range(lo, hi):
            p, tok, u = target(j)
            r = p
            if j < hi - 1:
                at = np.nonzero(tok == x[j])[0]
                px = p[at[0]] if at.size else 0.0
                if a[j] * draft(j, x[j]) < px:
                    tokens[j] = x[j]
                    continue
                rest = np.maximum(p - draft(j, tok), 0.0)
                if rest.sum() > 0:
                    r = rest
            c = np.cumsum(r)
            ok = np.nonzero((c > u * c[-1]) & (r > 0))[0]
            tokens[j] = tok[ok[0] if ok.size else np.nonzero(r > 0)[0][-1]]
            count[i] = j - lo + 1
            break
    return torch.from_numpy(tokens), torch.from_numpy(count)


def _exact_verify(case, s):
    vals, idx = s["vals"].double().cpu().numpy(), s["idx"].cpu().numpy()
    prm = s["params"].double().cpu().numpy()

    def target(j):
        v, k = vals[j], case["k"]
        top_k, top_p, temp = prm[j, :3]
        u = prm[j, 3] if case["cols"] == 4 else 0.5
        kk = int(top_k) if 1 <= top_k < k + 1 else k
        if not temp > 0 or kk == 1:
            e = np.array([1.0])
        else:
            e = np.exp((v[:kk] - v[0]) / temp)
            if top_p < 1:
                c = np.cumsum(e)
                e = e[:int(np.argmax(c >= top_p * c[-1])) + 1]
        return e / e.sum(), idx[j, :e.size], u

    return _exact_tokens(case, s, target, None)


def _exact_logits(case, s):
    temp, u = s["temperature"].double().cpu().numpy(), s["draw"].double().cpu().numpy()
    every = np.arange(case["V"])

    def target(j):
        z = s["logits"][j].double().cpu().numpy()
        if not temp[j] > 0:
            p = np.zeros(case["V"])
            p[int(np.argmax(z))] = 1.0
        else:
            p = np.exp((z - z.max()) / temp[j])
            p /= p.sum()
        return p, every, u[j]

    return _exact_tokens(case, s, target, None)


def _exact_moe(case, s):
    T, k, sh = case["T"], case["topk"], case["shared"]
    x = s["x"].double()
    norm = torch.sqrt((x ** 2).sum(-1) / case["H"] + 1e-5)
    t = x * s["gamma"].double() / norm[:, None]
    logit = (s["router_w"].double()[None] * t[:, None]).sum(-1)
    bias = s["router_b"].double()
    hidden = torch.empty((T, case["H"]), dtype=torch.float64, device=DEV)
    ids = torch.empty((T, k + sh), dtype=torch.int32)
    wts = torch.ones((T, k + sh), dtype=torch.float64)
    grid = torch.tensor(FP4, dtype=torch.float64, device=DEV)
    alpha, beta, limit = _act_args(case)

    def matrix(name, e):
        w = s["w" + name][e]
        if case["w"] == "bf16":
            return w.double()
        m = torch.empty((w.shape[0], 2 * w.shape[1]), dtype=torch.float64, device=DEV)
        m[:, 0::2], m[:, 1::2] = grid[(w % 16).long()], grid[(w // 16).long()]
        return m * torch.repeat_interleave(torch.pow(2.0, s["s" + name][e].double() - 127), 32, dim=1)

    for i in range(T):
        score = (1 / (1 + torch.exp(-logit[i])) if case["score"] == "sigmoid" else logit[i]).cpu().numpy()
        key = score + bias.cpu().numpy()
        chosen = np.lexsort((np.arange(case["E"]), -key))[:k]
        ids[i, :k] = torch.from_numpy(chosen.astype(np.int32))
        ids[i, k:] = torch.arange(case["E"], case["E"] + sh, dtype=torch.int32)
        w = score[chosen] * 2.5 / score[chosen].sum() if case["score"] == "sigmoid" else np.exp(key[chosen] - key.max())
        wts[i, :k] = torch.from_numpy(w if case["score"] == "sigmoid" else w / w.sum())
    acc = x.clone()
    for e in range(case["E"] + sh):
        where = (ids == e).nonzero().tolist()
        if not where:
            continue
        w1, w2 = matrix("1", e), matrix("2", e)
        for i, slot in where:
            h = w1 @ t[i] + s["b1"][e].double()
            if case["act"] == "relu2":
                a = torch.where(h > 0, h, 0.0) ** 2
            else:
                half = case["I"]
                gate, up = (h[::2], h[1::2]) if case["act"] == "clamped" else (h[:half], h[half:])
                if limit:
                    gate, up = torch.minimum(gate, torch.full_like(gate, limit)), up.clamp(-limit, limit)
                a = gate / (1 + torch.exp(-alpha * gate)) * (up + beta)
            acc[i] += float(wts[i, slot]) * (w2 @ a + s["b2"][e].double())
    hidden.copy_(acc)
    return hidden, ids.to(DEV), wts.to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "verify_logits": _exact_logits, "moe": _exact_moe}[case["op"]](case, s)

"""Training operators on vocabulary logits, measured: their cases, inputs, plain forms and exact values.

  token_logprobs   log-probabilities of given tokens, the rows' log-sum-exps and entropies; and their gradient
  policy_loss      the clipped policy loss with its KL and entropy terms, and its gradient
  preference_loss  the paired preference loss over whole sequences, and its gradient
  distill_topk     distillation from a teacher's top logits (what the tail writes), and its gradient

A row r has logits z_r [V], p_r = softmax(z_r / T), l_r(v) = log p_r(v), H_r = -sum_v p_r(v) l_r(v).  A row whose token
is outside [0, V) (distill_topk: whose list has no id inside) is ignored: results 0, gradient 0, logits of any value.

  token_logprobs   l_r(t_r), lse_r = log sum_v exp(z_rv / T), H_r; gradient of sum_r a_r l_r(t_r) + b_r H_r:
                   dz_rv = (a_r (1[v = t_r] - p_r(v)) - b_r p_r(v) (l_r(v) + H_r)) / T
  policy_loss      with R = exp(l_r(t_r) - old_r), k = exp(ref_r - l_r(t_r)) - (ref_r - l_r(t_r)) - 1:
                   loss_r = w_r (max(-A_r R, -A_r clip(R, 1 - c_lo, 1 + c_hi)) + kl k - ent H_r)
  preference_loss  with L_s = sum (or mean) of l_r(t_r) over the sequence's counted rows, sequences 2i (chosen) and
                   2i + 1 (rejected): h = beta ((L_2i - ref_2i) - (L_2i+1 - ref_2i+1)) - margin,
                   loss_i = w_i ((1 - eps) log(1 + exp(-h)) + eps log(1 + exp(h)))
  distill_topk     q = softmax over the list's t_i / T and, where it is given, the rest (the log of what the teacher's
                   other tokens sum to): loss_r = w_r (sum_i q_i (log q_i - l_r(id_i)) + q_rest (log q_rest -
                   log sum_{v not listed} p_r(v)))
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the tokens of one decode step of four sequences, scored on the tail's fp32 logits
        dict(name="logprobs_step", op="logprobs", dir="forward", rows=4, V=201088, l="f32", T=0.8, ent=True, skip=0.0),
        # a batch of finished completions, scored in 16 bits
        dict(name="logprobs_batch", op="logprobs", dir="forward", rows=1536, V=201088, l="bf16", T=1.0, ent=False,
             skip=0.1),
        # the gradient of a loss of the user's own, an odd vocabulary whose rows start inside 16-byte vectors
        dict(name="logprobs_grad_odd", op="logprobs", dir="backward", rows=777, V=50021, l="bf16", T=1.0, ent=True,
             skip=0.05),
        # one short completion under a policy step, on fp32 logits: the latency of a call
        dict(name="policy_short", op="policy", rows=12, V=201088, l="f32", T=1.0, ref=True, ent=0.0, skip=0.0),
        # a micro-batch of a small model, with an entropy bonus and masked prompt rows
        dict(name="policy_odd", op="policy", rows=333, V=50021, l="f16", T=0.7, ref=True, ent=0.01, skip=0.2),
        # a long training batch in 16 bits
        dict(name="policy_large", op="policy", rows=2048, V=201088, l="bf16", T=1.0, ref=True, ent=0.0, skip=0.1),
        # one pair of short answers
        dict(name="preference_pair", op="preference", pairs=1, lmin=9, lmax=17, prompt=3, pad=0, V=32000, l="f16",
             T=1.0, mean=False, eps=0.0),
        # a batch of pairs of ragged answers, rows left over behind them
        dict(name="preference_batch", op="preference", pairs=8, lmin=40, lmax=120, prompt=8, pad=37, V=201088, l="bf16",
             T=1.0, mean=False, eps=0.1),
        # a draft model's rows of one step against the tail's top-k
        dict(name="distill_step", op="distill", rows=8, V=201088, l="f32", k=256, t="f32", rest=False, T=1.0, skip=0.0),
        # stored lists of an odd length in 16 bits, with the rest's weight
        dict(name="distill_odd", op="distill", rows=500, V=50021, l="bf16", k=77, t="bf16", rest=True, T=1.5, skip=0.1),
        # a training batch of a draft model
        dict(name="distill_large", op="distill", rows=1024, V=201088, l="f32", k=256, t="f32", rest=True, T=1.0,
             skip=0.05),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "preference", "distill"])
    l = rng.choice(["f32", "f16", "bf16"])
    V = _log_int(rng, 300, 201088)
    most = max(1, min(2048, int(1.2e9 / (2 * V * SIZE[l]))))
    c = dict(op=op, V=V, l=l, T=rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.0), 2)]))
    if op == "preference":
        lmin = _log_int(rng, 1, 60)
        pairs = _log_int(rng, 1, 24)
        span = rng.randint(0, 40)
        if 2 * pairs * (lmin + span) > most:
            pairs, span = 1, 0
            lmin = max(1, min(lmin, most // 2))
        return dict(c, pairs=pairs, lmin=lmin, lmax=lmin + span, prompt=rng.choice([0, 0, 2]),
                    pad=rng.choice([0, 0, rng.randint(1, 30)]), mean=rng.choice([False, True]),
                    eps=rng.choice([0.0, 0.1]))
    c.update(rows=_log_int(rng, 1, most), skip=rng.choice([0.0, 0.1, 0.3]))
    if op == "logprobs":
        return dict(c, dir=rng.choice(["forward", "backward"]), ent=rng.choice([False, True]))
    if op == "policy":
        return dict(c, ref=rng.choice([False, True]), ent=rng.choice([0.0, 0.0, 0.01]))
    return dict(c, k=_log_int(rng, 1, min(V // 2, 1024)), t=rng.choice(["f32", "f32", "f16", "bf16"]),
                rest=rng.choice([False, True]))


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _logits(case, rows, g):
    """Logits as a model gives them: a broad body and a few columns that the context makes likely; in one row of
    eight a third of the vocabulary is masked."""
    V = case["V"]
    z = 2.2 * torch.randn((rows, V), generator=g, device=DEV)
    peaks = torch.randint(0, V, (rows, 24), generator=g, device=DEV)
    z.scatter_add_(1, peaks, 4.0 + 4.0 * torch.rand((rows, 24), generator=g, device=DEV))
    start = torch.randint(0, V, (rows, 1), generator=g, device=DEV)
    col = torch.arange(V, device=DEV)
    off = ((col + start) % V < V // 3) & (torch.arange(rows, device=DEV) % 8 == 5)[:, None]
    return z.masked_fill_(off, -math.inf).to(DTYPES[case["l"]])


def _tokens(z, T, skip, g):
    """A token a row, drawn from softmax(z / T), some of them -1: prompt positions and padding."""
    race = z.float() / T - torch.log(torch.empty(z.shape, device=DEV).exponential_(generator=g).clamp_(min=1e-30))
    t = torch.argmax(race, dim=-1).to(torch.int32)
    return torch.where(torch.rand(t.shape, generator=g, device=DEV) < skip, -1, t)


def _scores(z, tokens, T):
    """(l(t), lse) in 64 bits, the rows a few at a time."""
    out = []
    for i in range(0, z.shape[0], 256):
        y = z[i:i + 256].double() / T
        n = torch.logsumexp(y, -1)
        out.append(torch.stack((y.gather(1, tokens[i:i + 256, None].long().clamp(min=0))[:, 0] - n, n)))
    return torch.cat(out, 1)


def _randn(n, g):
    return torch.randn(n, generator=g, device=DEV)


def _weights(case, n):
    """The mean over n losses; times a loss scale where gradients are held in fp16."""
    return torch.full((n,), (1024.0 if case["l"] == "f16" else 1.0) / n, device=DEV)


def _prepare_logprobs(case, seed):
    g, rows = _gen(seed), case["rows"]
    z = _logits(case, rows, g)
    t = _tokens(z, case["T"], case["skip"], g)
    s = dict(case=case, z=z, t=t)
    if case["dir"] == "forward":
        s.update(logprob=torch.empty(rows, device=DEV), lse=torch.empty(rows, device=DEV),
                 entropy=torch.empty(rows, device=DEV))
        return s
    a = _randn(rows, g) * _weights(case, rows)
    s.update(lse=_scores(z, t, case["T"])[1].float(), a=a, grad=torch.empty_like(z))
    if case["ent"]:
        s["b"] = 0.05 * torch.rand(rows, generator=g, device=DEV) * _weights(case, rows)
        s["entropy"] = torch.cat([_entropy64(z[i:i + 256], case["T"]) for i in range(0, rows, 256)]).float()
    return s


def _entropy64(z, T):
    y = z.double() / T
    p = torch.softmax(y, -1)
    return torch.logsumexp(y, -1) - torch.where(p > 0, p * y, 0.0).sum(-1)


CLIP = (0.2, 0.28)
KL = 0.05


def _prepare_policy(case, seed):
    g, rows = _gen(seed), case["rows"]
    z = _logits(case, rows, g)
    t = _tokens(z, case["T"], case["skip"], g)
    l = _scores(z, t, case["T"])[0]
    # the policy moved by a few steps since the rollout; the gradient jumps at the clip's two borders, so no row's
    # ratio lies where 32 bits could not tell its side
    d = 0.2 * _randn(rows, g).double()
    for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
        d = torch.where((d - border).abs() < 1e-3, d + 4e-3, d)
    return dict(case=case, z=z, t=t, old=(l - d).float(), adv=_randn(rows, g),
                ref=(l + 0.3 * _randn(rows, g)).float() if case["ref"] else None,
                w=_weights(case, rows), loss=torch.empty(rows, device=DEV),
                logprob=torch.empty(rows, device=DEV), grad=torch.empty_like(z))


def _prepare_preference(case, seed):
    g = _gen(seed)
    n, span = 2 * case["pairs"], case["lmax"] - case["lmin"] + 1
    length = case["lmin"] + torch.arange(n) * 7 % span
    length = length[torch.randperm(n, generator=torch.Generator().manual_seed(seed))]
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), torch.cumsum(length, 0))).to(DEV)
    rows = int(cu[-1]) + case["pad"]
    z = _logits(case, rows, g)
    t = _tokens(z, case["T"], 0.0, g)
    row = torch.arange(rows, device=DEV)
    seq = (torch.searchsorted(cu, row, right=True) - 1).clamp_(max=n - 1)
    t = torch.where(row - cu[seq] < case["prompt"], -1, t)  # the prompts' last rows come along uncounted
    l = torch.where((t >= 0) & (row < cu[-1]), _scores(z, t, case["T"])[0], 0.0)
    total = torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, seq, l)
    if case["mean"]:
        live = ((t >= 0) & (row < cu[-1])).double()
        total /= torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, seq, live).clamp_(min=1.0)
    ref = total + (0.5 if case["mean"] else 6.0) * _randn(n, g)
    return dict(case=case, z=z, t=t, cu=cu.to(torch.int32), ref=ref.float(),
                w=_weights(case, case["pairs"]), grad=torch.empty_like(z),
                loss=torch.empty(case["pairs"], device=DEV), logprob=torch.empty(n, device=DEV))


def _beta(case):
    return 2.0 if case["mean"] else 0.1


MARGIN = 0.25


def _prepare_distill(case, seed):
    g, rows, V, k, T = _gen(seed), case["rows"], case["V"], case["k"], case["T"]
    z = _logits(case, rows, g)
    teacher = z.float().clamp(min=-30.0)  # the teacher and its draft agree roughly; what is masked, it does not list
    teacher += 0.8 * torch.randn(z.shape, generator=g, device=DEV)
    top = torch.topk(teacher, k, dim=-1)
    vals, idx = top.values.to(DTYPES[case["t"]]), top.indices.to(torch.int32)
    rest = None
    # lists shorter than k end in -1
    cut = torch.where(torch.rand((rows, 1), generator=g, device=DEV) < 0.2, (k + 1) // 2, k)
    kept = torch.arange(k, device=DEV) < cut
    idx = torch.where(kept, idx, -1)
    if case["rest"]:
        teacher.scatter_(1, top.indices, torch.where(kept, -math.inf, top.values))
        rest = torch.logsumexp(teacher / T, -1)
    del teacher, top
    # the student's mask covers none of the listed tokens
    at = idx.clamp(min=0).long()
    got = z.gather(1, at)
    z.scatter_(1, at, torch.where(torch.isinf(got), -8.0, got.float()).to(z.dtype))
    idx = torch.where((torch.rand(rows, generator=g, device=DEV) < case["skip"])[:, None], -1, idx)
    return dict(case=case, z=z, vals=vals, idx=idx, rest=rest, w=_weights(case, rows),
                loss=torch.empty(rows, device=DEV), grad=torch.empty_like(z))


def prepare(case, seed):
    return {"logprobs": _prepare_logprobs, "policy": _prepare_policy, "preference": _prepare_preference,
            "distill": _prepare_distill}[case["op"]](case, seed)


# --------------------------------------------------------------------------- plain forms

def _softmax(y):
    """(y less its row maximum, exponentials, others, log of their sum) in 32 bits.  The maximum's own exponential, 1, is
    kept apart from the sum of the others: a likely token's log-probability -log(1 + others) and 1 - p =
    others / (1 + others) are then as exact as an unlikely one's."""
    top, at = y.max(-1, keepdim=True)
    y = y - top
    e = torch.exp(y)
    others = e.scatter(1, at, 0.0).sum(-1, keepdim=True)
    return y, e, others, torch.log1p(others)


def _rest_of(e, others):
    """1 - p of entries with exponentials e."""
    return torch.where(e == 1.0, others, 1.0 + others - e) / (1.0 + others)


def _soft(s):
    """What _softmax says of a state's logits, the tokens' columns and which rows are live."""
    y, e, others, ln = _softmax(s["z"].float() / s["case"]["T"])
    live = (s["t"] >= 0) & (s["t"] < y.shape[1])
    t = torch.where(live, s["t"], 0).long()[:, None]
    return y, e, others, ln, t, live


def _entropy(y, e, others, ln):
    return (ln - torch.where(e > 0, e * y, 0.0).sum(-1, keepdim=True) / (1.0 + others))[:, 0]


def _spread(s, p, rest, c, t, live, more=None):
    """(c (1[v = t] - p) + more) / T on the live rows, in the logits' type; rest: 1 - p at the tokens."""
    g = (-c[:, None] * p).scatter_(1, t, c[:, None] * rest)
    if more is not None:
        g = g + more
    return torch.where(live[:, None], g / s["case"]["T"], 0.0).to(s["z"].dtype)


def _plain_logprobs(s):
    case = s["case"]
    if case["dir"] == "forward":
        y, e, others, ln, t, live = _soft(s)
        top = s["z"].float().amax(-1) / case["T"]
        out = [torch.where(live, (y.gather(1, t) - ln)[:, 0], 0.0), torch.where(live, top + ln[:, 0], 0.0)]
        if case["ent"]:
            out.append(torch.where(live, _entropy(y, e, others, ln), 0.0))
        return out
    # 64 bits: differences of logits and sums of about 20, exponentiated
    live = (s["t"] >= 0) & (s["t"] < case["V"])
    t = torch.where(live, s["t"], 0).long()[:, None]
    l = s["z"].double() / case["T"] - s["lse"].double()[:, None]
    rest = -torch.expm1(l.gather(1, t)).float()
    l = l.float()
    p = torch.exp(l)
    more = None
    if case["ent"]:
        more = -s["b"][:, None] * torch.where(p > 0, p * (l + s["entropy"][:, None]), 0.0)
    return _spread(s, p, rest, s["a"], t, live, more)


def _plain_policy(s):
    case, w, A = s["case"], s["w"], s["adv"]
    y, e, others, ln, t, live = _soft(s)
    l = (y.gather(1, t) - ln)[:, 0]
    R = torch.exp(l - s["old"])
    a, b = -A * R, -A * torch.clamp(R, 1 - CLIP[0], 1 + CLIP[1])
    loss = torch.maximum(a, b)
    c = torch.where(a >= b, a, 0.0)
    if s["ref"] is not None:
        d = s["ref"] - l
        loss = loss + KL * (torch.expm1(d) - d)
        c = c - KL * torch.expm1(d)
    p = e / (1.0 + others)
    more = None
    if case["ent"]:
        H = _entropy(y, e, others, ln)
        loss = loss - case["ent"] * H
        more = (case["ent"] * w)[:, None] * torch.where(e > 0, p * (y - ln + H[:, None]), 0.0)
    g = _spread(s, p, _rest_of(e.gather(1, t), others), w * c, t, live, more)
    return torch.where(live, w * loss, 0.0), torch.where(live, l, 0.0), g


def _plain_preference(s):
    case, w = s["case"], s["w"]
    n = 2 * case["pairs"]
    cu = s["cu"].long()
    y, e, others, ln, t, live = _soft(s)
    row = torch.arange(y.shape[0], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    live = live & (seq >= 0) & (seq < n)
    seq = seq.clamp(0, n - 1)
    # 64 bits: the sums of a sequence's hundreds of log-probabilities, and the difference of two of them
    l = torch.where(live, (y.gather(1, t) - ln)[:, 0], 0.0).double()
    L = torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, seq, l)
    one = torch.ones(n, dtype=torch.float64, device=DEV)
    if case["mean"]:
        one = one / torch.zeros_like(one).index_add_(0, seq, live.double()).clamp_(min=1.0)
    L = L * one
    r = L - s["ref"].double()
    h = _beta(case) * (r[0::2] - r[1::2]) - MARGIN
    up = torch.clamp(-h, min=0.0) + torch.log1p(torch.exp(-h.abs()))  # log(1 + exp(-h))
    loss = w * ((1 - case["eps"]) * up + case["eps"] * (up + h))
    d = w * _beta(case) * (case["eps"] - torch.sigmoid(-h))
    c = (torch.stack((d, -d), 1).reshape(-1) * one)[seq]
    g = _spread(s, e / (1.0 + others), _rest_of(e.gather(1, t), others), c.float(), t, live)
    return loss.float(), L.float(), g


def _plain_distill(s):
    case, T, V, k = s["case"], s["case"]["T"], s["case"]["V"], s["case"]["k"]
    y, e, others, ln = _softmax(s["z"].float() / T)
    there = (s["idx"] >= 0) & (s["idx"] < V)
    live = there.any(-1)
    at = torch.where(there, s["idx"], 0).long()
    u = torch.where(there, s["vals"].float() / T, -math.inf)
    if s["rest"] is not None:
        u = torch.cat((u, s["rest"][:, None]), 1)
    u, f, f_others, lf = _softmax(u)
    q = f / (1.0 + f_others)
    lq = u - lf
    l = y.gather(1, at) - ln
    loss = torch.where(q[:, :k] > 0, q[:, :k] * (lq[:, :k] - l), 0.0).sum(-1)
    g = e / (1.0 + others)
    p = g.gather(1, at)
    # where both lie near 1, by what each lacks
    here = torch.where((p > 0.5) & (q[:, :k] > 0.5),
                       _rest_of(f[:, :k], f_others) - _rest_of(e.gather(1, at), others), p - q[:, :k])
    if s["rest"] is not None:
        listed_ = torch.zeros(y.shape, dtype=torch.int32, device=DEV).scatter_add_(1, at, there.int()) > 0
        out, inside = torch.where(listed_, 0.0, e), torch.where(listed_, e, 0.0)
        out_s, in_s = out.sum(-1), inside.sum(-1)
        more, less = q[:, k], out_s / (out_s + in_s)
        l_out = torch.where(less > 0.5, -torch.log1p(in_s / out_s), torch.log(less))
        l_more = torch.where(more > 0.5, -torch.log1p((f[:, :k].sum(-1) / f[:, k])), lq[:, k])
        loss = loss + torch.where(more > 0, more * (l_more - l_out), 0.0)
        off = torch.where((more > 0.5) & (less > 0.5), q[:, :k].sum(-1) - in_s / (out_s + in_s), less - more)
        g = torch.where(out_s > 0, off / out_s, 0.0)[:, None] * out
    # a list's padding points at column 0: the entry there, if any, is written by itself
    pad = torch.where(there, at, V)
    g = torch.cat((g, g[:, :1]), 1).scatter_(1, pad, here)[:, :V]
    g = s["w"][:, None] * g / T
    return torch.where(live, s["w"] * loss, 0.0), torch.where(live[:, None], g, 0.0).to(s["z"].dtype)


# --------------------------------------------------------------------------- the framework's calls

def _own(s):
    import decode_sampling_tail_gb300 as dst
    case = s["case"]
    if case["op"] == "logprobs":
        if case["dir"] == "forward":
            dst.token_logprobs(s["z"], s["t"], case["T"], out_logprob=s["logprob"], out_lse=s["lse"],
                               out_entropy=s["entropy"] if case["ent"] else None)
            return [s["logprob"], s["lse"]] + ([s["entropy"]] if case["ent"] else [])
        return dst.token_logprobs_grad(s["z"], s["t"], s["lse"], s["a"], case["T"], d_entropy=s.get("b"),
                                       entropy=s.get("entropy"), out_grad=s["grad"])
    if case["op"] == "policy":
        dst.policy_loss(s["z"], s["t"], s["old"], s["adv"], ref_logprob=s["ref"], temperature=case["T"],
                        clip_low=CLIP[0], clip_high=CLIP[1], kl_coef=KL if case["ref"] else 0.0,
                        entropy_coef=case["ent"], weight=s["w"], out_loss=s["loss"], out_logprob=s["logprob"],
                        out_grad=s["grad"])
        return s["loss"], s["logprob"], s["grad"]
    if case["op"] == "preference":
        dst.preference_loss(s["z"], s["t"], s["cu"], ref_logprob=s["ref"], beta=_beta(case), margin=MARGIN,
                            label_smoothing=case["eps"], average=case["mean"], temperature=case["T"], weight=s["w"],
                            out_loss=s["loss"], out_seq_logprob=s["logprob"], out_grad=s["grad"])
        return s["loss"], s["logprob"], s["grad"]
    dst.distill_topk(s["z"], s["vals"], s["idx"], teacher_rest=s["rest"], temperature=case["T"], weight=s["w"],
                     out_loss=s["loss"], out_grad=s["grad"])
    return s["loss"], s["grad"]


def run(state):
    if own:
        return _own(state)
    return {"logprobs": _plain_logprobs, "policy": _plain_policy, "preference": _plain_preference,
            "distill": _plain_distill}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass: the counted rows' logits read once, the gradient of every row written once,
    the small arrays."""
    size = SIZE[case["l"]]
    if case["op"] == "preference":
        span = case["lmax"] - case["lmin"] + 1
        n = 2 * case["pairs"]
        length = [case["lmin"] + i * 7 % span for i in range(n)]
        rows = sum(length) + case["pad"]
        live = sum(max(0, x - case["prompt"]) for x in length)
        small = 4 * rows + 8 * n + 12 * case["pairs"]
    else:
        rows = case["rows"]
        live = rows * (1 - case["skip"])
        small = rows * {"logprobs": 20, "policy": 28, "distill": 12}[case["op"]]
        if case["op"] == "distill":
            small += rows * case["k"] * (4 + SIZE[case["t"]])
    grad = 0 if case.get("dir") == "forward" else rows
    return {"bytes": float((live + grad) * case["V"] * size + small),
            "flops": live * case["V"] * (6.0 if case.get("dir") else 10.0)}


# --------------------------------------------------------------------------- exact values

def _rows64(s, i):
    """Row i: probabilities and log-probabilities in 64 bits."""
    y = s["z"][i].double() / s["case"]["T"]
    l = torch.log_softmax(y, 0)
    return torch.exp(l), l, y


def _exact_logprobs(case, s):
    V, t = case["V"], s["t"].tolist()
    rows = len(t)
    if case["dir"] == "forward":
        out = torch.zeros((3, rows), dtype=torch.float64, device=DEV)
        for i in range(rows):
            if 0 <= t[i] < V:
                p, l, y = _rows64(s, i)
                out[0, i], out[1, i], out[2, i] = l[t[i]], torch.logsumexp(y, 0), -torch.special.xlogy(p, p).sum()
        return [out[0], out[1]] + ([out[2]] if case["ent"] else [])
    grad = torch.zeros((rows, V), dtype=torch.float64, device=DEV)
    for i in range(rows):
        if 0 <= t[i] < V:
            l = s["z"][i].double() / case["T"] - float(s["lse"][i])
            p = torch.exp(l)
            g = -float(s["a"][i]) * p
            g[t[i]] += float(s["a"][i])
            if case["ent"]:
                g -= float(s["b"][i]) * (torch.special.xlogy(p, p) + p * float(s["entropy"][i]))
            grad[i] = g / case["T"]
    return grad


def _exact_policy(case, s):
    V, t = case["V"], s["t"].tolist()
    small = {n: s[n].double().tolist() for n in ("old", "adv", "w")}
    ref = s["ref"].double().tolist() if s["ref"] is not None else None
    loss, logprob = [0.0] * len(t), [0.0] * len(t)
    grad = torch.zeros((len(t), V), dtype=torch.float64, device=DEV)
    for i, tok in enumerate(t):
        if not 0 <= tok < V:
            continue
        p, l, _ = _rows64(s, i)
        lp = float(l[tok])
        ratio, A = math.exp(lp - small["old"][i]), small["adv"][i]
        inside = min(max(ratio, 1 - CLIP[0]), 1 + CLIP[1])
        value = -min(A * ratio, A * inside)
        slope = -A * ratio if A * ratio <= A * inside else 0.0
        if ref:
            k = math.exp(ref[i] - lp)
            value += KL * (k - 1 - (ref[i] - lp))
            slope += KL * (1 - k)
        g = -slope * p
        g[tok] += slope
        if case["ent"]:
            minus_h = torch.special.xlogy(p, p).sum()
            value += case["ent"] * float(minus_h)
            g += case["ent"] * (torch.special.xlogy(p, p) - p * minus_h)
        loss[i], logprob[i] = small["w"][i] * value, lp
        grad[i] = g * (small["w"][i] / case["T"])
    of = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
    return of(loss), of(logprob), grad


def _exact_preference(case, s):
    cu, t, V = s["cu"].tolist(), s["t"].tolist(), case["V"]
    ref, w = s["ref"].double().tolist(), s["w"].double().tolist()
    rows = len(t)
    total, number, at = [], [], []
    for q in range(2 * case["pairs"]):
        mine = [i for i in range(cu[q], cu[q + 1]) if 0 <= t[i] < V]
        v = math.fsum(float(_rows64(s, i)[1][t[i]]) for i in mine)
        total.append(v / max(1, len(mine)) if case["mean"] else v)
        number.append(max(1, len(mine)) if case["mean"] else 1)
        at.append(mine)
    loss, grad = [], torch.zeros((rows, V), dtype=torch.float64, device=DEV)
    for i in range(case["pairs"]):
        a, b = 2 * i, 2 * i + 1
        h = _beta(case) * ((total[a] - ref[a]) - (total[b] - ref[b])) - MARGIN
        soft = lambda x: math.log1p(math.exp(x)) if x < 30 else x + math.log1p(math.exp(-x))  # noqa: E731
        loss.append(w[i] * ((1 - case["eps"]) * soft(-h) + case["eps"] * soft(h)))
        sig = 1 / (1 + math.exp(-h))
        dh = w[i] * _beta(case) * (case["eps"] * sig - (1 - case["eps"]) * (1 - sig))
        for q, sign in ((a, 1.0), (b, -1.0)):
            for r in at[q]:
                g = -_rows64(s, r)[0]
                g[t[r]] += 1.0
                grad[r] = g * (sign * dh / number[q] / case["T"])
    of = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
    return of(loss), of(total), grad


def _exact_distill(case, s):
    V, T, k = case["V"], case["T"], case["k"]
    rows = case["rows"]
    loss, grad = torch.zeros(rows, dtype=torch.float64, device=DEV), torch.zeros((rows, V), dtype=torch.float64, device=DEV)
    w = s["w"].double().tolist()
    number = ((s["idx"] >= 0) & (s["idx"] < V)).sum(-1).tolist()
    for i in range(rows):
        n = number[i]  # the list's valid ids come first
        if n == 0:
            continue
        ids = s["idx"][i, :n].long()
        u = s["vals"][i, :n].double() / T
        if s["rest"] is not None:
            u = torch.cat((u, s["rest"][i:i + 1].double()))
        lq = torch.log_softmax(u, 0)
        q = torch.exp(lq)
        p, l, y = _rows64(s, i)
        value = (q[:n] * (lq[:n] - l[ids])).sum()
        g = p.clone()
        if s["rest"] is not None:
            y[ids] = -math.inf
            if n < V:
                outside = torch.logsumexp(y, 0) - torch.logsumexp(s["z"][i].double() / T, 0)
                value = value + q[n] * (lq[n] - outside)
                g -= q[n] * torch.softmax(y, 0)
            elif float(q[n]) > 0:
                value = value + math.inf
        g.index_add_(0, ids, -q[:n])
        loss[i], grad[i] = w[i] * value, g * (w[i] / T)
    return loss, grad


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "policy": _exact_policy, "preference": _exact_preference,
            "distill": _exact_distill}[case["op"]](case, s)

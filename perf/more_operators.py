"""The choices made from a row's softmax, as measured work: cases, their inputs, the plain form
of each operator in torch, and the library's calls.

Operators (rows of logits in f32, bf16 or f16; the random numbers are inputs):

- ``sample_rows``    a token drawn from each row's softmax by a given uniform number
- ``verify_drafts``  drafted tokens accepted or replaced so that what is emitted follows the target
- ``route_rows``     each row's experts and their gates
- ``route_grad``     the gradient of the gates with respect to the router's logits
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 1 << 26  # logits of a block of rows, where inputs are made and checked block by block

SAMPLE = {"temperature": 1.0, "mixed": False, "banned": 0, "logp": False, "sigma": 3.0}
VERIFY = {"temperature": 1.0, "mixed": False, "draft": True, "noise": 1.0, "tail": 0, "logp": False, "sigma": 3.0}
ROUTE = {"score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 2, "renormalise": True,
         "scale": 1.0, "masked": 0.0, "banned": 0, "counts": False, "sigma": 1.5}


def listed():
    return [
        # one request's next token: launches and latencies count
        dict(SAMPLE, name="sample_1x32000", op="sample_rows", type="bf16", rows=1, vocab=32000, stride=32000,
             temperature=0.8),
        # a decode batch of a large vocabulary, some tokens banned by -inf
        dict(SAMPLE, name="sample_256x151936", op="sample_rows", type="bf16", rows=256, vocab=151936, stride=152064,
             temperature=0.7, banned=1000),
        # rollouts: requests with temperatures of their own, some greedy, log-probabilities kept for training; odd rows
        dict(SAMPLE, name="sample_f32_1024x50257", op="sample_rows", type="f32", rows=1024, vocab=50257, stride=50257,
             mixed=True, logp=True),
        # a few requests, up to four drafts each, of a small vocabulary
        dict(VERIFY, name="verify_f16_4x4_32000", op="verify_drafts", type="f16", requests=4, drafts=4, vocab=32000,
             stride=32000, temperature=0.8),
        # drafts looked up in the prompt: nothing was drawn, so there are no draft logits; an odd vocabulary in f32
        dict(VERIFY, name="verify_f32_lookup_32x6_50257", op="verify_drafts", type="f32", requests=32, drafts=6,
             vocab=50257, stride=50257, draft=False, mixed=True),
        # a serving batch: ragged drafts, capacity left over at the end
        dict(VERIFY, name="verify_64x4_151936", op="verify_drafts", type="bf16", requests=64, drafts=4, vocab=151936,
             stride=152064, temperature=0.7, tail=13),
        # many rollouts with long drafts; the largest
        dict(VERIFY, name="verify_256x7_128256", op="verify_drafts", type="bf16", requests=256, drafts=7,
             vocab=128256, stride=128256, logp=True, noise=0.7),
        # a decode batch's routing: sigmoid scores, balance by bias, experts in groups
        dict(ROUTE, name="route_f32_32x256", op="route_rows", type="f32", rows=32, experts=256, stride=256, k=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
        # the same for a training batch, with the counts that move the bias
        dict(ROUTE, name="route_16384x256", op="route_rows", type="bf16", rows=16384, experts=256, stride=256, k=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5, masked=0.1, counts=True),
        # softmax scores over few experts, odd rows: gates are the probabilities themselves
        dict(ROUTE, name="route_f32_30011x60", op="route_rows", type="f32", rows=30011, experts=60, stride=60, k=4,
             renormalise=False, counts=True),
        # the training batch's gradient
        dict(ROUTE, name="route_grad_16384x256", op="route_grad", type="bf16", rows=16384, experts=256, stride=256,
             k=8, score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5, masked=0.1),
        # every expert's logit has a gradient where the gates are not renormalised
        dict(ROUTE, name="route_grad_f32_30011x60", op="route_grad", type="f32", rows=30011, experts=60, stride=60,
             k=4, renormalise=False),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample_rows", "verify_drafts", "verify_drafts", "route_rows", "route_grad"])
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op.startswith("route"):
        experts = rng.choice([8, 16, 60, 64, 96, 128, 160, 200, 256, 384])
        rows = _between(rng, 1, min(40000, 5_000_000 // experts))
        groups, top_groups = rng.choice([(1, 1), (1, 1), (4, 2), (8, 4), (8, 3)])
        if experts % groups or experts // groups < 4:
            groups, top_groups = 1, 1
        return dict(ROUTE, op=op, type=kind, rows=rows, experts=experts,
                    stride=experts if rng.random() < 0.7 else experts + rng.randint(1, 40),
                    k=rng.randint(1, min(16, top_groups * (experts // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]), renormalise=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.2]),
                    banned=rng.choice([0, 0, experts // 8]), counts=op == "route_rows" and rng.random() < 0.5)
    vocab = _between(rng, 1000, 151936)
    most = 230_000_000 // vocab  # rows of logits and draft logits: below the largest listed case's
    same = dict(op=op, type=kind, vocab=vocab, stride=vocab if rng.random() < 0.6 else -(-vocab // 128) * 128,
                temperature=rng.choice([1.0, 0.7, 1.2]), mixed=rng.random() < 0.3, logp=rng.random() < 0.4)
    if op == "sample_rows":
        return dict(SAMPLE, **same, rows=_between(rng, 1, min(2048, most)), banned=rng.choice([0, vocab // 50]))
    drafts = rng.randint(1, 8)
    return dict(VERIFY, **same, drafts=drafts, requests=_between(rng, 1, max(2, min(512, most // (2 * drafts + 2)))),
                draft=rng.random() < 0.75, noise=rng.choice([0.5, 1.0]), tail=rng.choice([0, 0, 7]))


# -- inputs ---------------------------------------------------------------------

def _lengths(case):
    """Rows of each request of a verification: its drafts and one more; ragged, the longest first."""
    r = random.Random(7919 * case["requests"] + case["drafts"])
    return [case["drafts"] + 1] + [r.randint(1, case["drafts"]) + 1 for _ in range(case["requests"] - 1)]


def _rows(case):
    return sum(_lengths(case)) + case["tail"] if case["op"] == "verify_drafts" else case["rows"]


def _blocks(rows, cols):
    step = max(1, CHUNK // cols)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _uniform(n, gen):
    return torch.rand(n, generator=gen, device="cuda").clamp_(max=1 - 2.0 ** -24)


def _clear_of_borders(w, u):
    """Numbers near u that fall well inside a column's share of the weights w: what lies within the
    rounding of a border says nothing of either side, and neither does a column hardly wider than
    a step of the numbers themselves (the widest column takes its place)."""
    cum = w.cumsum(1)
    total = cum[:, -1:]
    at = (cum <= u.double()[:, None] * total).sum(1, keepdim=True).clamp_(max=w.shape[1] - 1)
    at = torch.where(w.gather(1, at) < 8e-6 * total, w.argmax(1, keepdim=True), at)
    hi, share = cum.gather(1, at) / total, w.gather(1, at) / total
    inside = ((u.double()[:, None] - (hi - share)) / share).clamp(0.25, 0.75)
    return (hi - share + inside * share)[:, 0].float().clamp_(0.0, 1 - 2.0 ** -24)


def _logits(rows, vocab, stride, kind, sigma, gen):
    x = torch.empty(rows, stride, dtype=TYPES[kind], device="cuda")
    for a, b in _blocks(rows, stride):
        x[a:b] = torch.randn(b - a, stride, generator=gen, device="cuda") * sigma
    return x[:, :vocab]


def _temperatures(case, rows, gen):
    """None, or a temperature for every row, about an eighth of them 0."""
    if not case["mixed"]:
        return None
    t = 0.5 + _uniform(rows, gen)
    return torch.where(_uniform(rows, gen) < 0.125, 0.0, t)


def _softmax64(x, t):
    return torch.softmax(x.double() / t.double()[:, None], 1)


def _prepare_sample(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    x = _logits(rows, vocab, case["stride"], case["type"], case["sigma"], gen)
    if case["banned"]:
        x[:, torch.randperm(vocab, generator=gen, device="cuda")[:case["banned"]]] = -math.inf
    t = _temperatures(case, rows, gen)
    u = _uniform(rows, gen)
    tt = torch.full((rows,), case["temperature"], device="cuda") if t is None else torch.where(t == 0, 1.0, t)
    for a, b in _blocks(rows, vocab):
        u[a:b] = _clear_of_borders(_softmax64(x[a:b], tt[a:b]), u[a:b])
    return {"case": case, "logits": x, "temperature": case["temperature"] if t is None else t, "uniforms": u}


def _prepare_verify(case, gen):
    lengths, vocab = _lengths(case), case["vocab"]
    rows = _rows(case)
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    x = _logits(rows, vocab, case["stride"], case["type"], case["sigma"], gen)
    y = torch.empty(rows, case["stride"], dtype=TYPES[case["type"]], device="cuda")[:, :vocab] if case["draft"] else None
    t = _temperatures(case, len(lengths), gen)
    if t is not None:  # a request's rows share its temperature
        t = torch.cat([t.repeat_interleave(torch.tensor(lengths, device="cuda")), t.new_ones(case["tail"])])
    tt = torch.full((rows,), case["temperature"], device="cuda") if t is None else torch.where(t == 0, 1.0, t)
    last = torch.zeros(rows, dtype=torch.bool, device="cuda")
    last[torch.tensor(ends[1:], device="cuda") - 1] = True
    last[ends[-1]:] = True
    drafts = torch.empty(rows, dtype=torch.int64, device="cuda")
    u = _uniform(2 * rows, gen).view(rows, 2)
    for a, b in _blocks(rows, vocab):
        p = _softmax64(x[a:b], tt[a:b])
        if y is not None:  # another model's view of the same rows, and a token drawn from it
            near = x[a:b].float() + case["noise"] * torch.randn(b - a, vocab, generator=gen, device="cuda")
            y[a:b] = near.to(y.dtype)
            q = _softmax64(y[a:b], tt[a:b])
            noise = torch.empty(b - a, vocab, device="cuda").exponential_(generator=gen).clamp_min_(1e-30)
            d = (q.log() - noise.log_().double()).argmax(1, keepdim=True)
            ratio = (p.gather(1, d) / q.gather(1, d))[:, 0]
        else:  # the token that followed the same words before: often the likeliest, else any of the likely ones
            likely = p.topk(16, dim=1)[1]
            which = torch.randint(0, 16, (b - a, 1), generator=gen, device="cuda")
            which = torch.where(_uniform(b - a, gen)[:, None] < 0.6, 0, which)
            d = likely.gather(1, which)
            q = torch.zeros_like(p).scatter_(1, d, 1.0)
            ratio = p.gather(1, d)[:, 0]
        drafts[a:b] = torch.where(last[a:b], -1, d[:, 0])
        one = u[a:b, 0].double()
        one = torch.where((one / ratio - 1).abs() < 1e-3, 0.5 * ratio, one)  # as for the borders
        u[a:b, 0] = one.float()
        rest = torch.where(last[a:b, None], p, (p - q).clamp_(min=0))
        u[a:b, 1] = _clear_of_borders(rest, u[a:b, 1])
    if t is not None and case["draft"]:
        # a greedy request's drafts are the draft model's own greedy choices
        top = torch.cat([y[a:b].float().argmax(1) for a, b in _blocks(rows, vocab)])
        drafts = torch.where((t == 0) & ~last, top, drafts)
    return {"case": case, "logits": x, "draft_logits": y, "drafts": drafts, "uniforms": u,
            "temperature": case["temperature"] if t is None else t,
            "offsets": torch.tensor(ends, dtype=torch.int64, device="cuda")}


def _near_ties(case, x, bias):
    """Rows whose choice hangs on scores that are not equal and closer than a rounding."""
    z = x.double()
    c = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
    if bias is not None:
        c = c + bias.double()
    c = c.masked_fill(z == -math.inf, -math.inf)
    least = 1e-5 * c.abs().masked_fill(c == -math.inf, 0).amax(1, keepdim=True)
    bad = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    near = lambda v: ((-v.diff(dim=1) > 0) & (-v.diff(dim=1) < least)).any(1)  # noqa: E731
    G, g = case["groups"], case["top_groups"]
    if g < G:
        top = c.view(-1, G, c.shape[1] // G).sort(dim=2, descending=True)[0][:, :, :case["group_top"]]
        score = top.clamp(min=-1e9).masked_fill(top == -math.inf, 0).sum(2).masked_fill(top[:, :, 0] == -math.inf, -1e9)
        bad |= near(score.sort(dim=1, descending=True)[0][:, :g + 1])
        keep = torch.zeros_like(score, dtype=torch.bool)
        keep.scatter_(1, score.sort(dim=1, descending=True, stable=True)[1][:, :g], True)
        c = c.masked_fill(~keep.repeat_interleave(c.shape[1] // G, 1), -math.inf)
    return bad | near(c.sort(dim=1, descending=True)[0][:, :case["k"] + 1].clamp(min=-1e9))


def _prepare_route(case, gen):
    rows, E = case["rows"], case["experts"]
    bias = 0.05 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
    if bias is not None and case["score"] == "softmax":
        bias = bias / E
    banned = torch.randperm(E, generator=gen, device="cuda")[:case["banned"]]
    x = _logits(rows, E, case["stride"], case["type"], case["sigma"], gen)
    x[:, banned] = -math.inf
    for _ in range(30):
        bad = _near_ties(case, x, bias).nonzero()[:, 0]
        if not len(bad):
            break
        fresh = (torch.randn(len(bad), E, generator=gen, device="cuda") * case["sigma"]).to(x.dtype)
        fresh[:, banned] = -math.inf
        x[bad] = fresh
    st = {"case": case, "logits": x, "bias": bias, "weights": None}
    off = int(round(case["masked"] * rows))
    if off:  # padding rows
        st["weights"] = torch.ones(rows, device="cuda")
        st["weights"][torch.randperm(rows, generator=gen, device="cuda")[:off]] = 0.0
    if case["op"] == "route_grad":
        st["chosen"] = _plain_route(st)["chosen"]
        st["gates_grad"] = torch.randn(rows, case["k"], generator=gen, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed * 7919 + 17)
    if case["op"] == "sample_rows":
        return _prepare_sample(case, gen)
    if case["op"] == "verify_drafts":
        return _prepare_verify(case, gen)
    return _prepare_route(case, gen)


# -- the operators --------------------------------------------------------------

def _exps(x, t):
    """d = (x - m) / T and e = exp(d) in f32; the sum of e in f64."""
    z = x.float() / (t[:, None] if isinstance(t, torch.Tensor) else t)
    d = z - z.amax(1, keepdim=True)
    e = d.exp()
    return d, e, e.double().sum(1)


def _pick(w, u):
    """The first column at which the running sum of w passes u of the whole: sums in f64."""
    cum = w.double().cumsum(1)
    return (cum <= u.double()[:, None] * cum[:, -1:]).sum(1).clamp_(max=w.shape[1] - 1)


def _first_max(x):
    """The first column that holds the row's largest value."""
    at = torch.arange(x.shape[1], device=x.device)
    return torch.where(x == x.amax(1, keepdim=True), at, x.shape[1]).amin(1)


def _greedy(t):
    """The rows of temperature 0, or None; and the temperatures with 1 in their place."""
    if not isinstance(t, torch.Tensor):
        return None, t
    return t == 0, torch.where(t == 0, 1.0, t)


def _plain_sample(st):
    greedy, t = _greedy(st["temperature"])
    d, e, s = _exps(st["logits"], t)
    tokens = _pick(e, st["uniforms"])
    if greedy is not None:
        tokens = torch.where(greedy, _first_max(d), tokens)
    out = {"tokens": tokens}
    if st["case"]["logp"]:
        logp = d.gather(1, tokens[:, None])[:, 0] - s.log().float()
        out["logp"] = logp if greedy is None else torch.where(greedy, 0.0, logp)
    return out


def _plain_verify(st):
    drafts, u, ends = st["drafts"], st["uniforms"], st["offsets"]
    greedy, t = _greedy(st["temperature"])
    rows, S = drafts.shape[0], ends.shape[0] - 1
    d, e, s = _exps(st["logits"], t)
    p = e / s.float()[:, None]
    has, at = drafts >= 0, drafts.clamp(min=0)[:, None]
    if st["draft_logits"] is None:
        q = torch.zeros_like(p).scatter_(1, at, 1.0)
    else:
        _, eq, sq = _exps(st["draft_logits"], t)
        q = eq / sq.float()[:, None]
    accept = has & (u[:, 0] * q.gather(1, at)[:, 0] < p.gather(1, at)[:, 0])
    rest = torch.where(has[:, None], (p - q).clamp(min=0), p)
    rest = torch.where((rest.sum(1) > 0)[:, None], rest, p)
    picked = _pick(rest, u[:, 1])
    if greedy is not None:
        top = _first_max(d)
        accept = torch.where(greedy, has & (drafts == top), accept)
        picked = torch.where(greedy, top, picked)
    token = torch.where(accept, drafts, picked)
    # a request's rows up to the first that is not accepted
    index = torch.arange(rows, device=drafts.device)
    owner = torch.searchsorted(ends, index, right=True) - 1
    inside = (owner >= 0) & (owner < S)
    stops = torch.cat([ends.new_zeros(1), (~accept).long().cumsum(0)])
    reached = inside & (stops[index] == stops[ends[owner.clamp(0, S - 1)]])
    taken = torch.cat([ends.new_zeros(1), (reached & accept).long().cumsum(0)])
    out = {"accepted": taken[ends[1:]] - taken[ends[:-1]], "tokens": torch.where(reached, token, -1)}
    if st["case"]["logp"]:
        logp = d.gather(1, token[:, None])[:, 0] - s.log().float()
        if greedy is not None:
            logp = torch.where(greedy, 0.0, logp)
        out["logp"] = torch.where(reached, logp, 0.0)
    return out


def _scores(case, x):
    z = x.float()
    if case["score"] == "sigmoid":
        return 1 / (1 + (-z).exp())
    e = (z - z.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _plain_route(st):
    c, x, w = st["case"], st["logits"], st["weights"]
    rows, E = x.shape
    scores = _scores(c, x)
    by = scores if st["bias"] is None else scores + st["bias"]
    by = torch.where(x == -math.inf, -math.inf, by)
    if c["top_groups"] < c["groups"]:
        per = E // c["groups"]
        best = by.view(rows, c["groups"], per).sort(dim=2, descending=True)[0][:, :, :min(per, c["group_top"])]
        group = torch.where(best == -math.inf, 0.0, best).sum(2)
        group = torch.where(best[:, :, 0] == -math.inf, -math.inf, group)
        kept = group.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros(rows, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        by = torch.where(keep.repeat_interleave(per, 1), by, -math.inf)
    value, chosen = by.sort(dim=1, descending=True, stable=True)
    value, chosen = value[:, :c["k"]], chosen[:, :c["k"]]
    on = value > -math.inf
    if w is not None:
        on &= (w != 0)[:, None]
    gates = torch.where(on, scores.gather(1, chosen), 0.0)
    if c["renormalise"]:
        total = gates.sum(1, keepdim=True)
        gates = torch.where(total > 0, gates / total, 0.0)
    out = {"chosen": torch.where(on, chosen, -1), "gates": gates * c["scale"]}
    if c["counts"]:
        out["counts"] = torch.zeros(E, dtype=torch.int64, device=x.device).scatter_add_(0, chosen.flatten(),
                                                                                      on.flatten().long())
    return out


def _plain_route_grad(st):
    c, x, chosen = st["case"], st["logits"], st["chosen"]
    scores = _scores(c, x)
    on = chosen >= 0
    at = chosen.clamp(min=0)
    g = torch.where(on, st["gates_grad"] * c["scale"], 0.0)
    s = torch.where(on, scores.gather(1, at), 0.0)
    if c["renormalise"]:
        total = s.sum(1, keepdim=True)
        share = torch.where(total > 0, s / total, 0.0)
        g = torch.where(total > 0, (g - (g * share).sum(1, keepdim=True)) / total, 0.0)
        g = torch.where(on, g, 0.0)
    by = torch.zeros_like(scores).scatter_add_(1, at, g)  # with respect to the scores
    if c["score"] == "sigmoid":
        grad = by * scores * (1 - scores)
    else:
        grad = scores * (by - (g * s).sum(1, keepdim=True))
    if st["weights"] is not None:
        grad = torch.where((st["weights"] != 0)[:, None], grad, 0.0)
    return {"grad": grad.to(x.dtype)}


def _own(st):
    import row_wise_softmax_ce_gb300 as ce
    c, op = st["case"], st["case"]["op"]
    if op == "sample_rows":
        got = ce.sample_rows(st["logits"], st["uniforms"], temperature=st["temperature"], logp=c["logp"])
        return {"tokens": got[0], "logp": got[1]} if c["logp"] else {"tokens": got}
    if op == "verify_drafts":
        accepted, tokens, logp = ce.verify_drafts(st["logits"], st["drafts"], st["offsets"], st["uniforms"],
                                                  draft_logits=st["draft_logits"], temperature=st["temperature"],
                                                  logp=c["logp"])
        out = {"accepted": accepted, "tokens": tokens}
        return {**out, "logp": logp} if c["logp"] else out
    how = dict(score=c["score"], renormalise=c["renormalise"], scale=c["scale"], weights=st["weights"])
    if op == "route_grad":
        return {"grad": ce.route_grad(st["logits"], st["chosen"], st["gates_grad"], **how)}
    chosen, gates, counts = ce.route_rows(st["logits"], c["k"], bias=st["bias"], groups=c["groups"],
                                          top_groups=c["top_groups"], group_top=c["group_top"], counts=c["counts"],
                                          **how)
    out = {"chosen": chosen, "gates": gates}
    return {**out, "counts": counts} if c["counts"] else out


def run(state):
    if own:
        return _own(state)
    return {"sample_rows": _plain_sample, "verify_drafts": _plain_verify, "route_rows": _plain_route,
            "route_grad": _plain_route_grad}[state["case"]["op"]](state)


def work(case):
    """Every row of logits that may count read once, the outputs written once, a few numbers a row."""
    op, size, rows = case["op"], SIZE[case["type"]], _rows(case)
    if op.startswith("route"):
        E, k = case["experts"], case["k"]
        live = rows - int(round(case["masked"] * rows))
        numbers = rows * (12 * k + (4 if case["masked"] else 0))
        each = 6 if op == "route_rows" else 8  # score, bias and a comparison; score and its derivative
        return {"bytes": live * E * size + (rows * E * size if op == "route_grad" else 0) + numbers + 12 * E,
                "flops": live * (E * each + 4 * k)}
    logits = rows * case["vocab"]
    numbers = rows * (16 + (4 if case["logp"] else 0))
    if op == "verify_drafts":
        if case["tail"]:
            logits -= case["tail"] * case["vocab"]
        if case["draft"]:
            logits += (rows - case["tail"] - case["requests"]) * case["vocab"]
        numbers += rows * 16 + 16 * case["requests"]
    return {"bytes": logits * size + numbers, "flops": 4 * logits}


# -- the definition in 64 bits ----------------------------------------------------

def _exact_draw(weights, u):
    """Column of u under the distribution that `weights` (f64, one row) are in proportion to."""
    cdf = torch.cumsum(weights / weights.sum(), 0)
    return min(int(torch.searchsorted(cdf, u.double() * cdf[-1], right=True)), weights.shape[0] - 1)


def _exact_sample(case, st):
    t = st["temperature"]
    tokens, logp = [], []
    for i in range(case["rows"]):
        x, ti = st["logits"][i].double(), float(t[i]) if case["mixed"] else t
        lp = torch.log_softmax(x / (ti if ti > 0 else 1.0), 0)
        k = int((x == x.max()).nonzero()[0]) if ti == 0 else _exact_draw(lp.exp(), st["uniforms"][i])
        tokens.append(k)
        logp.append(lp[k] if ti > 0 else lp.new_zeros(()))
    out = {"tokens": torch.tensor(tokens, device="cuda")}
    if case["logp"]:
        out["logp"] = torch.stack(logp)
    return out


def _exact_verify(case, st):
    ends, drafts = st["offsets"].tolist(), st["drafts"].tolist()
    temperature = st["temperature"].tolist() if case["mixed"] else [case["temperature"]] * len(drafts)
    tokens = [-1] * len(drafts)
    logp = torch.zeros(len(drafts), dtype=torch.float64, device="cuda")
    accepted = []
    for a, b in zip(ends, ends[1:]):
        n = 0
        for r in range(a, b):
            x, T, d = st["logits"][r].double(), temperature[r], drafts[r]
            lp = torch.log_softmax(x / (T or 1.0), 0)
            if T == 0:
                tokens[r] = int((x == x.max()).nonzero()[0])
                if tokens[r] != d:
                    break
                n += 1
                continue
            p = lp.exp()
            if d >= 0:
                if st["draft_logits"] is None:
                    q = torch.zeros_like(p)
                    q[d] = 1.0
                else:
                    q = torch.softmax(st["draft_logits"][r].double() / T, 0)
                if bool(st["uniforms"][r, 0].double() < p[d] / q[d]):
                    tokens[r], logp[r] = d, lp[d]
                    n += 1
                    continue
                p = torch.relu(p - q)
            tokens[r] = _exact_draw(p, st["uniforms"][r, 1])
            logp[r] = lp[tokens[r]]
            break
        accepted.append(n)
    out = {"accepted": torch.tensor(accepted, device="cuda"), "tokens": torch.tensor(tokens, device="cuda")}
    if case["logp"]:
        out["logp"] = logp
    return out


def _exact_choice(case, st):
    """Scores in f64, and the chosen experts one after another: the best that is left, the lowest of equals."""
    x = st["logits"].double()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    by = s if st["bias"] is None else s + st["bias"].double()
    by = torch.where(torch.isinf(x), -math.inf, by)
    E, G = case["experts"], case["groups"]

    def best_of(v, n):
        v, got = v.clone(), []
        column = torch.arange(v.shape[1], device="cuda")
        for _ in range(n):
            top = v.max(1, keepdim=True)[0]
            at = torch.where(v == top, column, v.shape[1]).min(1, keepdim=True)[0]
            got.append(torch.where(top == -math.inf, -1, at))
            v.scatter_(1, at, -math.inf)
        return torch.cat(got, 1)

    if case["top_groups"] < G:
        parts = by.unflatten(1, (G, E // G))
        first, at = parts.max(2)
        score = first
        if case["group_top"] == 2 and E // G > 1:
            second = parts.scatter(2, at[:, :, None], -math.inf).max(2)[0]
            score = first + torch.where(second == -math.inf, 0.0, second)
        kept = best_of(score, case["top_groups"])
        of = torch.arange(E, device="cuda") // (E // G)
        by = torch.where((of[None, :, None] == kept[:, None, :]).any(2), by, -math.inf)
    chosen = best_of(by, case["k"])
    if st["weights"] is not None:
        chosen[st["weights"] == 0] = -1
    return s, chosen


def _exact_gates(case, s, chosen):
    picked = s.gather(1, chosen.clamp(min=0)) * (chosen >= 0)
    if case["renormalise"]:
        picked = picked / picked.sum(1, keepdim=True).clamp(min=1e-300)
    return picked * case["scale"]


def _exact_route(case, st):
    s, chosen = _exact_choice(case, st)
    out = {"chosen": chosen, "gates": _exact_gates(case, s, chosen)}
    if case["counts"]:
        out["counts"] = torch.bincount(chosen[chosen >= 0], minlength=case["experts"])
    return out


def _exact_route_grad(case, st):
    x = st["logits"].double()
    x = torch.where(torch.isinf(x), -1e4, x).requires_grad_()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    total = (_exact_gates(case, s, st["chosen"]) * st["gates_grad"].double()).sum()
    grad, = torch.autograd.grad(total, x)
    if st["weights"] is not None:
        grad = grad * (st["weights"] != 0)[:, None]
    return {"grad": grad}


def exact(case, seed):
    st = prepare(case, seed)
    return {"sample_rows": _exact_sample, "verify_drafts": _exact_verify, "route_rows": _exact_route,
            "route_grad": _exact_route_grad}[case["op"]](case, st)

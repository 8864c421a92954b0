"""The objectives over sampled answers and over pairs of answers, as measured work: cases,
their inputs, the plain form of each operator in torch, and the library's calls.

Operators (logits ``[rows, vocab]`` in f32, bf16 or f16, one label a row; a row of weight 0 --
a prompt or padding token -- takes no part, and its label is -100):

- ``logp_rows``        each label's log-probability at a temperature, and the row's entropy
- ``policy_loss``      the clipped policy loss with a KL term and an entropy bonus
- ``policy_step``      the same with its gradient
- ``preference_loss``  the loss of pairs of sequences (sigmoid, hinge, squared)
- ``preference_step``  the same with its gradient
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 1 << 27  # logits of a block of rows, where inputs are made and checked block by block

LOGP = {"temperature": 1.0, "entropy": False, "masked": 0.0, "banned": 0, "sigma": 2.0}
POLICY = {"temperature": 1.0, "entropy": False, "masked": 0.0, "kl": 0.0, "bonus": 0.0, "low": 0.2, "high": 0.2,
          "sigma": 2.0}
PREFERENCE = {"temperature": 1.0, "kind": "sigmoid", "beta": 0.1, "smoothing": 0.0, "margin": 0.0, "average": False,
              "reference": True, "prompt": 0.25, "tail": 0, "loss_scale": 1.0, "sigma": 2.0}


def listed():
    return [
        # 16 requests of a decode batch: the chosen tokens' log-probabilities, some tokens banned by -inf
        dict(LOGP, name="logp_decode_16x151936", op="logp_rows", type="bf16", rows=16, vocab=151936, stride=152064,
             temperature=0.7, banned=1000),
        # scoring a batch of rollouts under the current and the frozen model, entropies for the log; the largest forward
        dict(LOGP, name="logp_rollout_8192x128256", op="logp_rows", type="bf16", rows=8192, vocab=128256,
             stride=128256, entropy=True, masked=0.125),
        # an odd vocabulary in f32, answers beside prompts
        dict(LOGP, name="logp_f32_4096x50257", op="logp_rows", type="f32", rows=4096, vocab=50257, stride=50257,
             masked=0.25, sigma=3.0),
        # the policy's loss alone, as an evaluation step takes it
        dict(POLICY, name="policy_loss_1024x151936", op="policy_loss", type="bf16", rows=1024, vocab=151936,
             stride=152064, kl=0.04),
        # a small model's loss in f16
        dict(POLICY, name="policy_loss_f16_2048x32000", op="policy_loss", type="f16", rows=2048, vocab=32000,
             stride=32000, entropy=True, masked=0.1),
        # the smallest training step: launches count
        dict(POLICY, name="policy_step_f32_64x1000", op="policy_step", type="f32", rows=64, vocab=1000, stride=1000,
             kl=0.04, masked=0.125),
        # a batch of answers with a quarter of padding
        dict(POLICY, name="policy_step_4096x32000", op="policy_step", type="bf16", rows=4096, vocab=32000,
             stride=32000, kl=0.02, masked=0.25, high=0.28),
        # odd rows in 16 bits: every row starts at another phase of 16 bytes
        dict(POLICY, name="policy_step_8192x50257", op="policy_step", type="bf16", rows=8192, vocab=50257,
             stride=50257, kl=0.04, temperature=0.9),
        # f32 logits of a large vocabulary, with an entropy bonus; the largest
        dict(POLICY, name="policy_step_f32_4096x128256", op="policy_step", type="f32", rows=4096, vocab=128256,
             stride=128256, entropy=True, bonus=0.01),
        # four short pairs of a small model
        dict(PREFERENCE, name="preference_step_f32_4x1000", op="preference_step", type="f32", pairs=4, rows=160,
             vocab=1000, stride=1000, prompt=0.0),
        # eight pairs of a large vocabulary, a quarter of each a shared prompt, capacity left over at the end
        dict(PREFERENCE, name="preference_step_8x128256", op="preference_step", type="bf16", pairs=8, rows=3000,
             vocab=128256, stride=128256, tail=72, smoothing=0.05),
        # the loss of held-out pairs, averaged over each answer's tokens, without a reference model
        dict(PREFERENCE, name="preference_loss_24x50257", op="preference_loss", type="bf16", pairs=24, rows=6001,
             vocab=50257, stride=50257, beta=2.0, margin=0.5, average=True, reference=False),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp_rows", "policy_loss", "policy_step", "policy_step", "preference_loss", "preference_step"])
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    vocab = _between(rng, 1000, 151936)
    most = 250_000_000 // vocab  # a quarter of the largest listed case's logits
    stride = vocab if rng.random() < 0.6 else -(-vocab // 128) * 128
    temperature = rng.choice([1.0, 1.0, 0.7, 1.3])
    same = dict(op=op, type=kind, vocab=vocab, stride=stride, temperature=temperature)
    if op == "logp_rows":
        return dict(LOGP, **{**same, "rows": _between(rng, 8, min(8192, most)), "entropy": rng.random() < 0.5,
                             "masked": rng.choice([0.0, 0.2]), "banned": rng.choice([0, vocab // 50])})
    if op.startswith("policy"):
        bonus = rng.choice([0.0, 0.01])
        return dict(POLICY, **{**same, "rows": _between(rng, 64, min(8192, most)), "kl": rng.choice([0.0, 0.04]),
                               "bonus": bonus, "entropy": bonus > 0 or rng.random() < 0.3,
                               "masked": rng.choice([0.0, 0.1, 0.4]), "high": rng.choice([0.2, 0.28])})
    pairs = _between(rng, 2, 32)
    rows = max(8 * pairs, _between(rng, 100, min(8192, most)))
    average = rng.random() < 0.3
    return dict(PREFERENCE, **{**same, "pairs": pairs, "rows": rows, "kind": rng.choice(["sigmoid", "sigmoid", "squared"]),
                               "beta": 2.0 if average else 0.1, "average": average, "reference": not average,
                               "smoothing": rng.choice([0.0, 0.1]), "prompt": rng.choice([0.0, 0.4]),
                               "tail": rng.choice([0, 0, rows // 20]),
                               "loss_scale": 1024.0 if kind == "f16" else 1.0})


# -- inputs ---------------------------------------------------------------------

def _lengths(case):
    """The lengths of a preference case's 2 * pairs sequences: ragged, at least 2, their sum rows - tail."""
    n, total = 2 * case["pairs"], case["rows"] - case["tail"]
    r = random.Random(1000003 * case["pairs"] + case["rows"])
    share = [r.uniform(0.3, 1.7) for _ in range(n)]
    lengths = [2 + int((total - 2 * n) * s / sum(share)) for s in share]
    lengths[-1] += total - sum(lengths)
    return lengths


def _prompt(case, length):
    return int(case["prompt"] * length)


def _active(case):
    """Rows with a weight that is not 0."""
    if case["op"].startswith("preference"):
        return sum(n - _prompt(case, n) for n in _lengths(case))
    return case["rows"] - int(round(case["masked"] * case["rows"]))


def _blocks(rows, vocab):
    step = max(1, CHUNK // vocab)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _logits(case, gen):
    """Logits, the label of each row drawn from softmax(x / T), and its log-probability."""
    rows, vocab, stride = case["rows"], case["vocab"], case["stride"]
    x = torch.empty(rows, stride, dtype=TYPES[case["type"]], device="cuda")
    labels = torch.empty(rows, dtype=torch.int64, device="cuda")
    logp = torch.empty(rows, dtype=torch.float32, device="cuda")
    banned = torch.randperm(vocab, generator=gen, device="cuda")[:case["banned"]] if case.get("banned") else None
    for a, b in _blocks(rows, stride):
        x[a:b] = torch.randn(b - a, stride, generator=gen, device="cuda") * case["sigma"]
        if banned is not None:
            x[a:b, banned] = -math.inf
        z = x[a:b, :vocab].float() / case["temperature"]
        noise = torch.empty_like(z).exponential_(generator=gen).clamp_min_(1e-30)
        labels[a:b] = (z - noise.log_()).argmax(1)
        del noise
        m = z.amax(1)
        logp[a:b] = z.gather(1, labels[a:b, None])[:, 0] - m - (z - m[:, None]).exp_().sum(1).log()
    return x[:, :vocab], labels, logp


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed * 7919 + 13)
    rows = case["rows"]
    logits, labels, logp = _logits(case, gen)
    normal = lambda: torch.randn(rows, generator=gen, device="cuda")  # noqa: E731
    st = {"case": case, "logits": logits, "labels": labels, "weights": None}
    if case["op"].startswith("preference"):
        lengths = _lengths(case)
        ends = [0]
        weights = torch.ones(rows, device="cuda")
        for n in lengths:
            weights[ends[-1]:ends[-1] + _prompt(case, n)] = 0.0
            ends.append(ends[-1] + n)
        weights[ends[-1]:] = 0.0
        st["offsets"] = torch.tensor(ends, dtype=torch.int64, device="cuda")
        st["ref"] = None
        if case["reference"]:  # the frozen model's log-probabilities of the sequences
            total = torch.stack([(weights * logp)[a:b].sum() for a, b in zip(ends, ends[1:])])
            if case["average"]:
                total = total / torch.stack([weights[a:b].sum() for a, b in zip(ends, ends[1:])])
            st["ref"] = (total + 4 * torch.randn(total.shape, generator=gen, device="cuda")).float()
        st["scale"] = case["loss_scale"] / case["pairs"]
        if case["prompt"] or case["tail"]:
            st["weights"] = weights
    else:
        off = int(round(case["masked"] * rows))
        if off:
            st["weights"] = torch.ones(rows, device="cuda")
            st["weights"][torch.randperm(rows, generator=gen, device="cuda")[:off]] = 0.0
        if case["op"].startswith("policy"):
            st["scale"] = 1.0 / (rows - off)
            old = logp + 0.1 * normal()  # the policy that sampled, some updates ago
            for edge in (1 - case["low"], 1 + case["high"]):
                # a ratio at a clip border to within the rounding of either side would say nothing
                old = torch.where(((logp - old).exp() - edge).abs() < 1e-3, old + 0.01, old)
            st["old"] = old
            st["advantages"] = 0.4 + normal()
            st["ref"] = logp + 0.2 * normal() if case["kl"] else None
    if st["weights"] is not None:
        st["labels"] = torch.where(st["weights"] != 0, labels, -100)
    return st


# -- the operators --------------------------------------------------------------

def _rows_plain(x, labels, weights, temperature):
    """d = (x - m) / T, e = exp(d), its sum, and each label's column and log-probability."""
    z = x.float() / temperature
    d = z - z.amax(1, keepdim=True)
    e = d.exp()
    s = e.sum(1, keepdim=True)
    at = labels if weights is None else torch.where(weights != 0, labels, 0)
    logp = d.gather(1, at[:, None])[:, 0] - s[:, 0].log()
    return d, e, s, at, logp


def _entropy_plain(d, e, s):
    return s[:, 0].log() - torch.where(e > 0, e * d, 0.0).sum(1) / s[:, 0]


def _keep(value, weights):
    return value if weights is None else torch.where(weights != 0, value, 0.0)


def _grad_plain(e, s, at, g, weights, scale, temperature, dtype, extra=None):
    """scale w / T (g ([j = label] - p) + extra), rounded once."""
    grad = e / s * -g[:, None]
    grad.scatter_add_(1, at[:, None], g[:, None])
    if extra is not None:
        grad += extra
    grad *= scale / temperature
    if weights is not None:
        grad = torch.where(weights[:, None] != 0, grad * weights[:, None], 0.0)
    return grad.to(dtype)


def _plain_logp(st):
    c, w = st["case"], st["weights"]
    d, e, s, _, logp = _rows_plain(st["logits"], st["labels"], w, c["temperature"])
    out = {"logp": _keep(logp, w)}
    if c["entropy"]:
        out["entropy"] = _keep(_entropy_plain(d, e, s), w)
    return out


def _plain_policy(st, step):
    c, w, A = st["case"], st["weights"], st["advantages"]
    d, e, s, at, logp = _rows_plain(st["logits"], st["labels"], w, c["temperature"])
    r = (logp - st["old"]).exp()
    plain, clipped = -A * r, -A * r.clamp(1 - c["low"], 1 + c["high"])
    rows = torch.maximum(plain, clipped)
    g = torch.where(plain >= clipped, plain, 0.0)
    if c["kl"]:
        far = st["ref"] - logp
        rows = rows + c["kl"] * (torch.expm1(far) - far)
        g = g - c["kl"] * torch.expm1(far)
    H = _entropy_plain(d, e, s) if c["entropy"] else None
    if c["bonus"]:
        rows = rows - c["bonus"] * H
    rows = _keep(rows, w)
    total = (rows if w is None else rows * w).double().sum() * st["scale"]
    out = {"loss": total.float(), "loss_rows": rows, "logp": _keep(logp, w)}
    if c["entropy"]:
        out["entropy"] = _keep(H, w)
    if step:
        extra = None
        if c["bonus"]:
            p = e / s
            extra = c["bonus"] * p * torch.where(p > 0, d - s.log() + H[:, None], 0.0)
        out["grad"] = _grad_plain(e, s, at, g, w, st["scale"], c["temperature"], st["logits"].dtype, extra)
    return out


def _plain_preference(st, step):
    c, w, P = st["case"], st["weights"], st["case"]["pairs"]
    _, e, s, at, logp = _rows_plain(st["logits"], st["labels"], w, c["temperature"])
    logp = _keep(logp, w)
    one = torch.ones_like(logp) if w is None else w
    upto = lambda v: torch.cat([v.new_zeros(1, dtype=torch.float64), v.double().cumsum(0)])[st["offsets"]]  # noqa: E731
    total, count = upto(one * logp).diff(), upto(one).diff()
    per = torch.ones_like(count)
    if c["average"]:
        per = torch.where(count != 0, 1 / count, 0.0)
    seq = total * per
    h = seq[:P] - seq[P:]
    if st["ref"] is not None:
        ref = st["ref"].double()
        h = h - (ref[:P] - ref[P:])
    beta, eps = c["beta"], c["smoothing"]
    if c["kind"] == "squared":
        off = h - c["margin"] - 0.5 / beta
        loss, dh = off * off, 2 * off
    else:
        z = beta * h - c["margin"]
        up, down = 1 / (1 + (-z).exp()), 1 / (1 + z.exp())  # sigma(z), sigma(-z)
        loss, dh = -(1 - eps) * up.log() - eps * down.log(), beta * (eps * up - (1 - eps) * down)
    out = {"loss": (loss.sum() * st["scale"]).float(), "loss_pairs": loss.float(), "seq_logp": seq.float(),
           "logp": logp}
    if step:
        seq_of = torch.searchsorted(st["offsets"], torch.arange(logp.shape[0], device=logp.device), right=True) - 1
        inside = (seq_of >= 0) & (seq_of < 2 * P)
        factor = torch.cat([dh, -dh]) * per
        g = torch.where(inside, factor[seq_of.clamp(0, 2 * P - 1)], 0.0).float()
        out["grad"] = _grad_plain(e, s, at, g, w, st["scale"], c["temperature"], st["logits"].dtype)
    return out


def _own(st):
    import row_wise_softmax_ce_gb300 as ce
    c, op = st["case"], st["case"]["op"]
    if op == "logp_rows":
        got = ce.logp_rows(st["logits"], st["labels"], weights=st["weights"], temperature=c["temperature"],
                           entropy=c["entropy"])
        return {"logp": got[0], "entropy": got[1]} if c["entropy"] else {"logp": got}
    if op.startswith("policy"):
        more = dict(ref_logp=st["ref"], weights=st["weights"], clip_low=c["low"], clip_high=c["high"], kl_coef=c["kl"],
                    entropy_coef=c["bonus"], temperature=c["temperature"], entropy=c["entropy"])
        args = (st["logits"], st["labels"], st["old"], st["advantages"], st["scale"])
        names = ("loss", "loss_rows", "logp", "entropy")
        got = ce.policy_loss(*args, **more) if op == "policy_loss" else ce.policy_step(*args, **more)
    else:
        more = dict(ref_logp=st["ref"], weights=st["weights"], kind=c["kind"], beta=c["beta"],
                    label_smoothing=c["smoothing"] if c["kind"] == "sigmoid" else 0.0, margin=c["margin"],
                    average=c["average"],
                    temperature=c["temperature"])
        args = (st["logits"], st["labels"], st["offsets"], st["scale"])
        names = ("loss", "loss_pairs", "seq_logp", "logp")
        got = ce.preference_loss(*args, **more) if op == "preference_loss" else ce.preference_step(*args, **more)
    if op.endswith("step"):
        names = ("grad",) + names
    return {k: v for k, v in zip(names, got) if v is not None}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "logp_rows":
        return _plain_logp(state)
    if op.startswith("policy"):
        return _plain_policy(state, op == "policy_step")
    return _plain_preference(state, op == "preference_step")


def work(case):
    """The logits of the rows that count read once, the whole gradient written once, a few numbers a row."""
    op, rows, vocab, size = case["op"], case["rows"], case["vocab"], SIZE[case["type"]]
    active = _active(case)
    step = op.endswith("step")
    numbers = {"logp": 4, "policy": 6, "preference": 3}[op.split("_")[0]]
    each = 4 + (2 if case.get("entropy") else 0) + (5 if step else 0)  # subtract, scale, exp, add; normalise and scale
    return {"bytes": active * vocab * size + (rows * vocab * size if step else 0) + rows * 4 * numbers,
            "flops": active * vocab * each}


# -- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op, rows, vocab, T = case["op"], case["rows"], case["vocab"], case["temperature"]
    live = torch.ones(rows, dtype=torch.bool, device="cuda") if st["weights"] is None else st["weights"] != 0
    w = live.double() if st["weights"] is None else st["weights"].double()
    lse = torch.zeros(rows, dtype=torch.float64, device="cuda")
    logp, entropy = torch.zeros_like(lse), torch.zeros_like(lse)
    for a, b in _blocks(rows, vocab):
        z = st["logits"][a:b].double() / T
        lse[a:b] = torch.logsumexp(z, 1)
        logp[a:b] = z[torch.arange(b - a, device="cuda"), st["labels"][a:b].clamp(min=0)] - lse[a:b]
        if case.get("entropy"):
            lp = z - lse[a:b, None]
            entropy[a:b] = -(lp.exp() * lp.clamp(min=-1e300)).sum(1)
    logp, entropy = logp * live, entropy * live
    g = torch.zeros_like(logp)
    if op == "logp_rows":
        return {"logp": logp, "entropy": entropy} if case["entropy"] else {"logp": logp}
    if op.startswith("policy"):
        A, r = st["advantages"].double(), (logp - st["old"].double()).exp()
        rows_loss = torch.where(A >= 0, -A * r.clamp(max=1 + case["high"]), -A * r.clamp(min=1 - case["low"]))
        g = torch.where(torch.where(A >= 0, r <= 1 + case["high"], r >= 1 - case["low"]), -A * r, 0.0)
        if case["kl"]:
            k = (st["ref"].double() - logp).exp()
            rows_loss, g = rows_loss + case["kl"] * (k - k.log() - 1), g + case["kl"] * (1 - k)
        rows_loss = (rows_loss - case["bonus"] * entropy) * live
        out = {"loss": (rows_loss * w).sum() * st["scale"], "loss_rows": rows_loss, "logp": logp}
        if case["entropy"]:
            out["entropy"] = entropy
    else:
        P, ends = case["pairs"], st["offsets"].tolist()
        seq, per = [], []
        for a, b in zip(ends, ends[1:]):
            total, count = (w[a:b] * logp[a:b]).sum(), w[a:b].sum()
            per.append(1 / count if case["average"] else torch.ones_like(count))
            seq.append(total * per[-1])
        seq = torch.stack(seq)
        h = seq[:P] - seq[P:]
        if st["ref"] is not None:
            h = h - st["ref"][:P].double() + st["ref"][P:].double()
        h = h.requires_grad_()
        z = case["beta"] * h - case["margin"]
        if case["kind"] == "squared":
            pairs = (h - case["margin"] - 1 / (2 * case["beta"])) ** 2
        else:
            eps = case["smoothing"]
            pairs = (1 - eps) * torch.log1p((-z).exp()) + eps * torch.log1p(z.exp())
        dh, = torch.autograd.grad(pairs.sum(), h)
        for p in range(P):
            g[ends[p]:ends[p + 1]] = dh[p] * per[p]
            g[ends[P + p]:ends[P + p + 1]] = -dh[p] * per[P + p]
        pairs = pairs.detach()
        out = {"loss": pairs.sum() * st["scale"], "loss_pairs": pairs, "seq_logp": seq.detach(), "logp": logp}
    if op.endswith("step"):
        grad = torch.empty(rows, vocab, dtype=torch.float64, device="cuda")
        factor = st["scale"] * w * live / T
        for a, b in _blocks(rows, vocab):
            lp = st["logits"][a:b].double() / T - lse[a:b, None]
            p = lp.exp()
            t = -p * g[a:b, None]
            t[torch.arange(b - a, device="cuda"), st["labels"][a:b].clamp(min=0)] += g[a:b]
            if case.get("bonus"):
                t += case["bonus"] * p * (lp + entropy[a:b, None])
            grad[a:b] = t * factor[a:b, None]
        out["grad"] = grad
    return out

"""What the operators on whole rows of logits are measured on, beside the
sampler and the verifier.

A serving loop scores tokens: the log probabilities of those it was given or
has drawn, the entropy of each distribution and its likeliest alternatives
("score").  The target's alternatives, kept with their log probabilities, are
what a draft model learns from: the divergence from a teacher of whom only the
top is known ("distill"), with its gradient ("distill_grad"), and the gradient
of log probabilities and entropies themselves ("score_grad").

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, with `own` set, through the package's public calls; `exact` is the
definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
LARGEST = 4093 * 152064 * 2          # bytes of logits that a scoring call reads
LARGEST_STEP = 4096 * 128256 * 2     # of a training call, which writes as many
CHUNK = 1 << 27                      # elements made at a time


# ---------------------------------------------------------------- cases


def listed():
    base = {"temp": False, "mask": False, "pad": False, "skip": 0.0}
    score = dict(base, op="score", ids=1, top=0, entropy=False)
    grad = dict(base, op="score_grad", ids=1, entropy=False)
    loss = dict(base, op="distill", k=20, tail=True)
    step = dict(base, op="distill_grad", k=20, tail=True)
    return [
        # one user's token with five alternatives, where only latency counts
        dict(score, name="score_b1", rows=1, vocab=128256, dtype="bf16", top=5, entropy=True),
        # the positions of a verify step of 32 requests with four drafts, each row at its request's temperature
        dict(score, name="score_verify_b32", rows=160, vocab=32000, dtype="f32", top=8, temp=True),
        # a full decoding batch with twenty alternatives, an eighth of its rows under a constraint mask
        dict(score, name="score_batch", rows=256, vocab=128256, dtype="bf16", top=20, entropy=True, mask=True),
        # the tokens of a prompt of odd length over a large vocabulary
        dict(score, name="score_prompt", rows=4093, vocab=152064, dtype="bf16", top=1, entropy=True),
        # a teacher's pass over training text: the 64 likeliest tokens of every position, at temperature
        dict(score, name="score_teacher", rows=2048, vocab=128256, dtype="bf16", ids=0, top=64, temp=True),
        # a short answer's gradient, over a vocabulary that no vector divides, cut from a padded projection
        dict(grad, name="score_grad_small", rows=37, vocab=50021, dtype="f32", pad=True),
        # policy gradient with an entropy term over a training batch, prompts left out
        dict(grad, name="score_grad_batch", rows=4096, vocab=128256, dtype="bf16", entropy=True, skip=0.25),
        # one verify step's worth of positions checked against the teacher's record
        dict(loss, name="distill_verify_b32", rows=160, vocab=32000, dtype="bf16"),
        # validation loss in binary32 over a large vocabulary
        dict(loss, name="distill_eval", rows=2039, vocab=152064, dtype="f32", k=64),
        # the smallest training call: a few positions, renormalised teacher
        dict(step, name="distill_grad_small", rows=61, vocab=8191, dtype="f32", k=16, tail=False),
        # a training batch over a large vocabulary
        dict(step, name="distill_grad_batch", rows=4096, vocab=128256, dtype="bf16", k=64),
        # padded sequences over a small vocabulary: a quarter of the rows is no token
        dict(step, name="distill_grad_padded", rows=8192, vocab=32000, dtype="bf16", skip=0.25, temp=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["score", "score", "score_grad", "distill", "distill_grad"])
    vocab = _log(rng, 8000, 152064)
    if rng.random() < 0.6:           # most vocabularies are padded to whole tiles, some are not
        vocab = max(8000, vocab // 64 * 64)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = (LARGEST if op in ("score", "distill") else LARGEST_STEP) // (vocab * BYTES[dtype])
    case = {"op": op, "rows": _log(rng, 1, min(8192, most)), "vocab": vocab, "dtype": dtype, "temp": rng.random() < 0.4,
            "mask": rng.random() < 0.2, "pad": rng.random() < 0.3, "skip": rng.choice([0.0, 0.0, 0.25])}
    if op == "score":
        case.update(ids=rng.choice([0, 1, 1, 1, 4]), top=rng.choice([0, 1, 5, 8, 20, 20, 64]), entropy=rng.random() < 0.6)
        if not case["ids"] and not case["top"]:
            case["entropy"] = True
    elif op == "score_grad":
        case.update(ids=rng.choice([1, 1, 4]), entropy=rng.random() < 0.5)
    else:
        case.update(k=rng.choice([8, 16, 20, 32, 64, 100]), tail=rng.random() < 0.7)
    return case


def live_rows(case):
    """Rows that hold a token; the others are padding, spread evenly."""
    every = int(round(1.0 / case["skip"])) if case["skip"] else 0
    return [not every or r % every != every - 1 for r in range(case["rows"])]


def work(case):
    rows, v, op = case["rows"], case["vocab"], case["op"]
    live = sum(live_rows(case))
    if op == "score":
        read = rows if case["entropy"] or case["top"] else live
        n = read * v
        return {"bytes": n * BYTES[case["dtype"]] + rows * (8 * case["ids"] + 8 * case["top"] + 4 * case["entropy"]),
                "flops": (7 if case["entropy"] else 4) * n}
    n = live * v
    if op == "score_grad":
        return {"bytes": (n + rows * v) * BYTES[case["dtype"]] + rows * (8 * case["ids"] + 4 * case["entropy"]),
                "flops": (14 if case["entropy"] else 8) * n}
    write = rows * v * BYTES[case["dtype"]] if op == "distill_grad" else 0
    return {"bytes": n * BYTES[case["dtype"]] + write + rows * (8 * case["k"] + 4), "flops": (8 if write else 4) * n}


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, v, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    stride = -(-v // 64) * 64 + 64 if case["pad"] else v
    store = torch.zeros((rows, stride), dtype=dt, device=DEV)
    logits = store[:, :v]
    k = case.get("k", 0)
    s = {"case": dict(case), "logits": logits, "temp": None}
    if case["temp"]:
        s["temp"] = torch.rand(rows, generator=g, device=DEV) + 0.5
    teach_ids = torch.empty((rows, k), dtype=torch.int32, device=DEV)
    teach = torch.empty((rows, k), dtype=torch.float32, device=DEV)
    likely = torch.empty((rows, 24), dtype=torch.int64, device=DEV)
    step = max(1, CHUNK // v)
    for lo in range(0, rows, step):  # a bulk of unlikely tokens and a few dozen that the context allows
        hi = min(rows, lo + step)
        z = torch.randn((hi - lo, v), generator=g, device=DEV).mul_(2.0)
        at = torch.randint(0, v // 24, (hi - lo, 24), generator=g, device=DEV) + torch.arange(24, device=DEV) * (v // 24)
        at = (at + torch.randint(0, v, (hi - lo, 1), generator=g, device=DEV)) % v    # 24 ids, all different
        up = 16.0 - 0.5 * torch.arange(24, device=DEV) + torch.randn((hi - lo, 24), generator=g, device=DEV)
        z.scatter_(1, at, up)
        likely[lo:hi] = at
        if case["mask"]:             # every eighth row may only say an eighth of the vocabulary
            bad = torch.rand((hi - lo, v), generator=g, device=DEV) > 0.125
            bad[(torch.arange(lo, hi, device=DEV) % 8 != 7)] = False
            bad.scatter_(1, at, False)
            z.masked_fill_(bad, -math.inf)
        logits[lo:hi] = z.to(dt)
        if k:                        # the teacher agrees but for noise; its record is at the same temperature
            z.add_(torch.randn((hi - lo, v), generator=g, device=DEV))
            if s["temp"] is not None:
                z.div_(s["temp"][lo:hi, None])
            top = z.topk(k, -1)
            teach_ids[lo:hi] = top.indices.int()
            teach[lo:hi] = top.values - z.logsumexp(-1, keepdim=True)
    live = torch.tensor(live_rows(case), device=DEV)
    new = lambda *shape, t=torch.float32: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
    if case["op"] in ("score", "score_grad"):
        n = case["ids"]
        ids = likely.gather(1, torch.randint(0, 24, (rows, max(n, 1)), generator=g, device=DEV))[:, :n].int()
        s["ids"] = torch.where(live[:, None], ids, -1).contiguous() if n else None
    if case["op"] == "score":
        top = case["top"]
        s["out"] = (new(rows, n) if n else None, new(rows) if case["entropy"] else None,
                    new(rows, top, t=torch.int32) if top else None, new(rows, top) if top else None)
    elif case["op"] == "score_grad":
        s["up"] = torch.randn((rows, n), generator=g, device=DEV)
        s["up_entropy"] = torch.where(live, 0.01 * torch.rand(rows, generator=g, device=DEV), 0.0) if case["entropy"] else None
    else:
        s["teach_ids"] = torch.where(live[:, None], teach_ids, -1).contiguous()
        s["teach"], s["loss"] = teach, new(rows)
        s["weight"] = live.float() / live.sum()
    if case["op"] in ("score_grad", "distill_grad"):
        s["grad"] = torch.empty_strided(logits.shape, logits.stride(), dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _scaled(s):
    z = s["logits"].float()
    return z if s["temp"] is None else z / s["temp"][:, None]


def _lse(y):
    top = y.amax(-1, keepdim=True)
    return top + torch.log(torch.exp(y - top).sum(-1, keepdim=True))


def _plain_score(s):
    c, y = s["case"], _scaled(s)
    lse, res = _lse(y), {}
    if c["ids"]:
        lp = y.gather(1, s["ids"].long().clamp(min=0)) - lse
        res["logprobs"] = torch.where(s["ids"] >= 0, lp, 0.0)
    if c["entropy"]:
        p = torch.exp(y - lse)
        res["entropy"] = (lse[:, 0] - torch.where(p > 0, p * y, 0.0).sum(-1))
    if c["top"]:                     # logits in order, the lower id first among equal ones: one whole number for both
        bits = s["logits"].float().add(0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) - torch.arange(c["vocab"], device=DEV)
        best = key.topk(c["top"], -1).values
        at = (-best) & 0xFFFFFFFF
        res["top_ids"], res["top_logprobs"] = at.int(), y.gather(1, at) - lse
    return res


def _plain_score_grad(s):
    y = _scaled(s)
    lp = y - _lse(y)
    p = torch.exp(lp)
    up = torch.where(s["ids"] >= 0, s["up"], 0.0)
    factor = up.sum(-1, keepdim=True)
    if s["up_entropy"] is not None:
        seen = torch.where(p > 0, lp, 0.0)
        entropy = -(p * seen).sum(-1, keepdim=True)
        factor = factor + s["up_entropy"][:, None] * (seen + entropy)
    grad = -p * factor
    grad.scatter_add_(1, s["ids"].long().clamp(min=0), up)
    if s["temp"] is not None:
        grad = grad / s["temp"][:, None]
    return {"grad": grad.to(s["logits"].dtype)}


def _plain_distill(s):
    c, y = s["case"], _scaled(s)
    rows, v = y.shape
    live = s["teach_ids"] >= 0
    at = s["teach_ids"].long().clamp(min=0)
    lse, l = _lse(y), s["teach"]
    if not c["tail"]:
        l = l - _lse(l)
    exact_t = torch.where(live, torch.exp(l.double()), 0.0)
    t, given = exact_t.float(), exact_t.sum(-1, keepdim=True).float()
    loss = torch.where(t > 0, t * (l - (y.gather(1, at) - lse)), 0.0).sum(-1)
    if c["tail"]:
        seen = torch.zeros((rows, v + 1), dtype=torch.bool, device=DEV)
        seen.scatter_(1, torch.where(live, at, v), True)
        y_rest = y.masked_fill(seen[:, :v], -math.inf)
        lse_rest = _lse(y_rest)
        rest = (1.0 - exact_t.sum(-1, keepdim=True)).clamp(min=0.0).float()    # a small difference of large numbers
        rest = torch.where(live.any(-1, keepdim=True), rest, 0.0)
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - (lse_rest - lse)), 0.0)[:, 0]
    res = {"loss": loss}
    if c["op"] == "distill_grad":
        if c["tail"]:
            grad = torch.exp(y - lse) * (given + rest) - rest * torch.exp(y_rest - lse_rest)
        else:
            grad = torch.exp(y - lse) * given
        grad.scatter_add_(1, at, -t)
        grad *= s["weight"][:, None]
        if s["temp"] is not None:
            grad /= s["temp"][:, None]
        res["grad"] = grad.to(s["logits"].dtype)
    return res


PLAIN = {"score": _plain_score, "score_grad": _plain_score_grad, "distill": _plain_distill, "distill_grad": _plain_distill}


def run(s):
    c = s["case"]
    if not own:
        return PLAIN[c["op"]](s)
    from spec_verify_gb300 import scores

    temp = 1.0 if s["temp"] is None else s["temp"]
    if c["op"] == "score":
        got = scores.token_logprobs(s["logits"], s["ids"], top=c["top"], entropy=c["entropy"], temperature=temp, out=s["out"])
        return {name: t for name, t in got._asdict().items() if t is not None}
    if c["op"] == "score_grad":
        return {"grad": scores.token_logprobs_grad(s["logits"], s["ids"], s["up"], s["up_entropy"], temperature=temp,
                                                   out=s["grad"])}
    if c["op"] == "distill":
        return {"loss": scores.distill_loss(s["logits"], s["teach_ids"], s["teach"], tail=c["tail"], temperature=temp,
                                            out=s["loss"])}
    loss, grad = scores.distill_grad(s["logits"], s["teach_ids"], s["teach"], weight=s["weight"], tail=c["tail"],
                                     temperature=temp, out_loss=s["loss"], out=s["grad"])
    return {"loss": loss, "grad": grad}


# ---------------------------------------------------------------- 64 bits


def _exact_part(c, s, lo, hi):
    """The definitions, for rows lo to hi."""
    y = s["logits"][lo:hi].double()
    tau = 1.0 if s["temp"] is None else s["temp"][lo:hi].double()[:, None]
    y = y / tau
    logp = torch.log_softmax(y, -1)
    p, res = logp.exp(), {}
    plogp = (p * logp.clamp(min=-1e4))
    if c["op"] == "score":
        if c["ids"]:
            ids = s["ids"][lo:hi].long()
            res["logprobs"] = torch.where(ids < 0, 0.0, logp.gather(1, ids.clamp(min=0)))
        if c["entropy"]:
            res["entropy"] = -plogp.sum(-1)
        if c["top"]:
            res["top_ids"], res["top_logprobs"] = None, logp.topk(c["top"], -1).values
        return res
    if c["op"] == "score_grad":
        ids = s["ids"][lo:hi].long()
        up = s["up"][lo:hi].double() * (ids >= 0)
        grad = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), up) - up.sum(-1, keepdim=True) * p
        if c["entropy"]:
            entropy = -plogp.sum(-1, keepdim=True)
            grad -= s["up_entropy"][lo:hi].double()[:, None] * (plogp + p * entropy)
        return {"grad": grad / tau}
    ids, l = s["teach_ids"][lo:hi].long(), s["teach"][lo:hi].double()
    live, at = ids >= 0, ids.clamp(min=0)
    if not c["tail"]:
        l = torch.log_softmax(l, -1)
    t = l.exp() * live
    loss = (t * (l - logp.gather(1, at))).sum(-1)
    target = torch.zeros_like(p).scatter_add_(1, at, t)      # the teacher's distribution, its tail shared out as the student's
    if c["tail"]:
        rest = torch.where(live.any(-1), 1.0 - t.sum(-1), 0.0).clamp(min=0.0)
        outside = torch.ones_like(p).scatter_(1, at, 0.0)
        mine = (p * outside).sum(-1)
        loss = loss + torch.xlogy(rest, rest / mine)
        target += (rest / mine)[:, None] * p * outside
    res["loss"] = torch.where(live.any(-1), loss, 0.0)
    if c["op"] == "distill_grad":
        total = target.sum(-1, keepdim=True)
        res["grad"] = (p * total - target) * s["weight"][lo:hi].double()[:, None] / tau
    return res


def exact(case, seed):
    s, rows = prepare(case, seed), case["rows"]
    step = max(1, CHUNK // case["vocab"])
    parts = [_exact_part(case, s, lo, min(rows, lo + step)) for lo in range(0, rows, step)]
    return {name: None if parts[0][name] is None else torch.cat([part[name] for part in parts]) for name in parts[0]}

"""What the operators of one speculative decoding step are measured on.

A step of a target model that checks k drafted tokens per request, as a
serving loop runs it: block tables and slot maps for the tokens of the step
("plan"), the norms of its queries and keys with the position rotation
("rope"), the keys and values written into an 8-bit paged cache ("append"),
attention over that cache ("attend") and the check of the drafts against the
target's probabilities from given random numbers ("verify").

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, with `own` set, through the package's public calls; `exact` is the
definition in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX, I8_MAX = 448.0, 127.0
MIN_EXP = -100                       # smallest scale exponent of a cache block
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
WORKSPACE = 64 << 20                 # bytes a serving loop keeps for attention


# ---------------------------------------------------------------- cases


def listed():
    return [
        # 32 requests that each add a token and 4 drafts: the step's bookkeeping, where only latency counts
        {"name": "plan_verify_b32", "op": "plan", "batch": 32, "add": 5, "ragged": False, "len": 4096, "block": 16},
        # a burst of prompts admitted at once: half a million slots
        {"name": "plan_prompts", "op": "plan", "batch": 509, "add": 2048, "ragged": True, "len": 512, "block": 64},
        # queries and keys of one verify step, cut from the fused projection's rows
        {"name": "rope_verify_b32", "op": "rope", "tokens": 160, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "dtype": "bf16"},
        # a prompt chunk
        {"name": "rope_prompt", "op": "rope", "tokens": 16381, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "dtype": "bf16"},
        # the same step's keys and values: five tokens into each request's last blocks
        {"name": "append_verify_b32", "op": "append", "batch": 32, "add": 5, "len": 4096, "kv_heads": 8, "dim": 128,
         "block": 16, "codes": "e4m3", "dtype": "bf16"},
        # ragged prompt chunks, most of them starting inside a block
        {"name": "append_prompts_i8", "op": "append", "batch": 37, "add": 443, "len": 300, "kv_heads": 8, "dim": 128,
         "block": 64, "codes": "i8", "dtype": "bf16"},
        # one user, one token, a short context
        {"name": "attend_b1", "op": "attend", "batch": 1, "add": 1, "len": 1029, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "codes": "e4m3", "dtype": "bf16", "window": 0, "lse": False},
        # the verify step of 32 requests with contexts of many lengths
        {"name": "attend_verify_b32", "op": "attend", "batch": 32, "add": 5, "len": 4096, "heads": 32, "kv_heads": 8,
         "dim": 128, "block": 16, "codes": "e4m3", "dtype": "bf16", "window": 0, "lse": False},
        # few requests with long documents, one token each
        {"name": "attend_long_i8", "op": "attend", "batch": 4, "add": 1, "len": 131072, "heads": 64, "kv_heads": 8,
         "dim": 128, "block": 64, "codes": "i8", "dtype": "bf16", "window": 0, "lse": True},
        # long contexts verified, eight query heads to a key head
        {"name": "attend_verify_long", "op": "attend", "batch": 8, "add": 5, "len": 65536, "heads": 64, "kv_heads": 8,
         "dim": 128, "block": 32, "codes": "e4m3", "dtype": "bf16", "window": 0, "lse": False},
        # the verifier's own workload shape
        {"name": "verify_b32", "op": "verify", "batch": 32, "k": 4, "vocab": 32000, "dtype": "f32"},
        # a full batch of a large vocabulary
        {"name": "verify_b256", "op": "verify", "batch": 256, "k": 4, "vocab": 128256, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attend", "attend", "verify"])
    if op == "plan":
        batch = _log(rng, 1, 2048)
        return {"op": op, "batch": batch, "add": _log(rng, 1, min(8192, (1 << 19) // batch)), "ragged": rng.random() < 0.7,
                "len": _log(rng, 1, 8192), "block": rng.choice([16, 32, 64, 128])}
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        inter = rng.random() < 0.4
        rotary = dim if rng.random() < 0.6 else dim // 2
        return {"op": op, "tokens": _log(rng, 1, min(16381, 16381 * 40 * 64 // ((heads + kv) * dim))), "heads": heads,
                "kv_heads": kv, "dim": dim, "rotary": rotary, "interleaved": inter, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    codes = rng.choice(["e4m3", "i8"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    block = rng.choice([16, 32, 64, 128])
    if op == "append":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 256)
        most = 16381 * 8 * 64 // (batch * kv * dim)
        return {"op": op, "batch": batch, "add": _log(rng, 1, max(1, min(4096, most))), "len": _log(rng, 1, 2048),
                "kv_heads": kv, "dim": dim, "block": block, "codes": codes, "dtype": dtype}
    if op == "attend":
        dim = rng.choice([64, 96, 128, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8, 8])
        batch = _log(rng, 1, 128)
        add = rng.choice([1, 1, 2, 4, 5, 8, 17])
        most = (8 * 65536 * 8 * 128 * 40 // max(40, add * group)) // (batch * kv * dim) // 2
        return {"op": op, "batch": batch, "add": add, "len": _log(rng, min(add, most), min(131072, most)), "heads": kv * group,
                "kv_heads": kv, "dim": dim, "block": block, "codes": codes, "dtype": dtype,
                "window": rng.choice([0, 0, 0, 1000]), "lse": rng.random() < 0.5}
    vocab = rng.choice([500, 8191, 32000, 50021, 128256, 152064])
    dtype = rng.choice(["f32", "bf16"])
    k = rng.choice([1, 2, 3, 4, 5, 8])
    most = 256 * 128256 * 5 // (vocab * (k + 1))
    return {"op": op, "batch": _log(rng, 1, min(256, most)), "k": k, "vocab": vocab, "dtype": dtype}


def lengths(case):
    """Tokens held before the step and tokens added, for each request: part of
    the case, the same for every seed."""
    b, add, top = case["batch"], case["add"], case["len"]
    r = random.Random(7919 * b + 104729 * add + top)
    if case["op"] == "attend":       # lengths after the step, the longest is `len`
        after = [max(add, int(top * r.uniform(0.25, 1.0))) for _ in range(b)]
        after[r.randrange(b)] = max(add, top)
        adds = [add if r.random() < 0.75 else r.randint(1, add) for _ in range(b)]
        return [a - n for a, n in zip(after, adds)], adds
    held = [r.randint(0, top) for _ in range(b)]
    adds = [r.randint(0, 2 * add) if case.get("ragged") else add for _ in range(b)]
    if sum(adds) == 0:
        adds[0] = add
    return held, adds


def work(case):
    op = case["op"]
    if op == "plan":
        held, adds = lengths(case)
        total, b = sum(adds), case["batch"]
        fresh = sum(-(-(h + a) // case["block"]) - -(-h // case["block"]) for h, a in zip(held, adds))
        return {"bytes": 16 * total + 8 * fresh + 24 * b, "flops": 0}
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * n * size + case["tokens"] * (4 * case["rotary"] + 4) + 8 * case["dim"], "flops": 7 * n}
    if op == "append":
        held, adds = lengths(case)
        size = 2 if case["dtype"] == "bf16" else 4
        t = sum(adds)
        touched = sum(-(-(h + a) // case["block"]) - h // case["block"] for h, a in zip(held, adds) if a)
        n = 2 * t * case["kv_heads"] * case["dim"]
        return {"bytes": n * (size + 1) + 8 * t + 12 * touched * case["kv_heads"], "flops": 3 * n}
    if op == "attend":
        held, adds = lengths(case)
        size = 2 if case["dtype"] == "bf16" else 4
        seen, pairs = 0, 0
        for h, a in zip(held, adds):
            w = case["window"]
            seen += min(h + a, w + a - 1) if w else h + a
            pairs += sum(min(p + 1, w) if w else p + 1 for p in range(h, h + a))
        blocks = -(-seen // case["block"])
        n = sum(adds) * case["heads"] * case["dim"]
        return {"bytes": 2 * seen * case["kv_heads"] * case["dim"] + blocks * (8 * case["kv_heads"] + 4) + 2 * n * size
                + (4 * sum(adds) * case["heads"] if case["lse"] else 0),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    # one row each of the target, the draft (not read where every draft is kept) and the noise
    size = 2 if case["dtype"] == "bf16" else 4
    b, v = case["batch"], case["vocab"]
    kept = len(_all_kept(b))
    return {"bytes": b * v * (size + 4) + (b - kept) * v * size + b * case["k"] * (4 + 4 + 2 * size), "flops": 3 * b * v}


# ---------------------------------------------------------------- inputs


def _all_kept(batch):
    return range(3, batch, 4)        # requests whose uniforms keep every draft


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pages(held, block, columns, blocks, g):
    """A block table whose requests hold ceil(held / block) blocks drawn at
    random from `blocks`, the number held, and the blocks left over."""
    n = torch.tensor([-(-h // block) for h in held], dtype=torch.int64)
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(held), columns), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(columns, device=DEV)[None] < n.to(DEV)[:, None]] = order[: int(n.sum())]
    return table, n.to(torch.int32).to(DEV), order[int(n.sum()):].clone()


def _codes(shape, name, g):
    x = torch.randn(shape, generator=g, device=DEV)
    if name == "e4m3":
        return (x * 64.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return (x * 32.0).round_().clamp_(-I8_MAX, I8_MAX).to(torch.int8)


def _cache(case, blocks, g):
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    unit = 2.0 ** -6 if case["codes"] == "e4m3" else 2.0 ** -5
    scale = lambda: unit * 2.0 ** torch.randint(-1, 2, shape[:2], generator=g, device=DEV).float()  # noqa: E731
    return _codes(shape, case["codes"], g), _codes(shape, case["codes"], g), scale(), scale()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op == "plan":
        held, adds = lengths(case)
        need = [-(-(h + a) // case["block"]) for h, a in zip(held, adds)]
        columns, blocks = max(need) + 3, sum(need) + 17
        table, n, free = _pages(held, case["block"], columns, blocks, g)
        cap = (sum(adds) + 63) // 64 * 64                 # the captured step's token capacity
        b = case["batch"]
        new = lambda *shape, t=torch.int32: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
        s.update(lens=_ints(held), add=_ints(adds), held=n, free=free, head=_ints([3]), table=table, blocks=blocks, cap=cap,
                 out=(new(b), new(b), new(1), new(b + 1), new(cap), new(cap), new(cap, t=torch.int64)))
        return s
    if op == "rope":
        dt, t, h, kv, d = DTYPES[case["dtype"]], case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        fused = torch.randn((t, h + 2 * kv, d), generator=g, device=DEV).mul_(2.0).to(dt)
        rows = 32768
        pos = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None]
        freq = 10000.0 ** (-2.0 * torch.arange(case["rotary"] // 2, dtype=torch.float64, device=DEV) / case["rotary"])
        s.update(q=fused[:, :h], k=fused[:, h:h + kv], table=torch.cat([(pos * freq).cos(), (pos * freq).sin()], 1).float(),
                 pos=torch.randint(0, rows, (t,), generator=g, device=DEV, dtype=torch.int32),
                 qw=1.0 + 0.1 * torch.randn(d, generator=g, device=DEV), kw=1.0 + 0.1 * torch.randn(d, generator=g, device=DEV),
                 oq=torch.empty((t, h, d), dtype=dt, device=DEV), ok=torch.empty((t, kv, d), dtype=dt, device=DEV))
        return s
    if op in ("append", "attend"):
        held, adds = lengths(case)
        bs, dt = case["block"], DTYPES[case["dtype"]]
        after = [h + a for h, a in zip(held, adds)]
        need = [-(-x // bs) for x in after]
        columns, blocks = max(need) + 1, sum(need) + 5
        table, _, _ = _pages(after, bs, columns, blocks, g)
        cache = _cache(case, blocks, g)
        start = [0]
        for a in adds:
            start.append(start[-1] + a)
        t = start[-1]
        req = torch.repeat_interleave(torch.arange(len(adds), device=DEV), torch.tensor(adds, device=DEV))
        first = torch.tensor(start[:-1], device=DEV)[req]
        pos = torch.tensor(held, device=DEV)[req] + torch.arange(t, device=DEV) - first
        s.update(cache=cache, start=_ints(start), lens=_ints(after), table=table, req=req, most=max(adds), columns=max(need),
                 local=torch.arange(t, device=DEV) - first)
        if op == "append":
            fused = torch.randn((t, 2 * case["kv_heads"], case["dim"]), generator=g, device=DEV).mul_(2.0)
            fused *= 2.0 ** torch.randint(-2, 3, (t, 1, 1), generator=g, device=DEV).float()
            fused = fused.to(dt)
            s.update(k=fused[:, :case["kv_heads"]], v=fused[:, case["kv_heads"]:],
                     slots=table[req, pos // bs].long() * bs + pos % bs)
        else:
            s.update(q=torch.randn((t, case["heads"], case["dim"]), generator=g, device=DEV).mul_(1.5).to(dt),
                     out=torch.empty((t, case["heads"], case["dim"]), dtype=dt, device=DEV),
                     lse=torch.empty((t, case["heads"]), dtype=torch.float32, device=DEV) if case["lse"] else None,
                     workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV))
        return s
    b, k, v, dt = case["batch"], case["k"], case["vocab"], DTYPES[case["dtype"]]
    q = torch.empty((b, k, v), dtype=dt, device=DEV)
    p = torch.empty((b, k + 1, v), dtype=dt, device=DEV)
    for i in range(k + 1):           # the draft's logits and the target's, one position at a time
        z = torch.randn((b, v), generator=g, device=DEV).mul_(2.0)
        if i < k:
            q[:, i] = torch.softmax(z, -1).to(dt)
        p[:, i] = torch.softmax(z.add_(torch.randn((b, v), generator=g, device=DEV)), -1).to(dt)
    ids = torch.empty((b, k), dtype=torch.int32, device=DEV)
    for i in range(k):               # drafts drawn from the draft's distribution
        race = q[:, i].float() / torch.empty((b, v), device=DEV).exponential_(generator=g)
        ids[:, i] = race.argmax(-1).to(torch.int32)
    u = torch.rand((b, k), generator=g, device=DEV)
    u[list(_all_kept(b))] = 0.0
    noise = torch.empty((b, v), device=DEV).exponential_(generator=g).clamp_(min=1e-30)
    s.update(p=p, q=q, ids=ids, u=u, noise=noise, accepted=torch.empty(b, dtype=torch.int32, device=DEV),
             tokens=torch.empty((b, k + 1), dtype=torch.int32, device=DEV))
    return s


# ---------------------------------------------------------------- plain forms


def _plain_plan(s):
    c, bs, cap = s["case"], s["case"]["block"], s["cap"]
    lens, add, table = s["lens"].long(), s["add"].long(), s["table"]
    after = lens + add
    need = torch.maximum(s["held"].long(), (after + bs - 1) // bs)
    fresh = need - s["held"]
    start = torch.zeros(c["batch"] + 1, dtype=torch.int64, device=DEV)
    start[1:] = add.cumsum(0)
    taken = fresh.cumsum(0) - fresh + s["head"]
    col = torch.arange(table.shape[1], device=DEV)[None]
    new = (col >= s["held"][:, None]) & (col < need[:, None])
    at = (taken[:, None] + col - s["held"][:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][at], table))
    tok = torch.arange(cap, device=DEV)
    live = tok < start[-1]
    req = torch.searchsorted(start, tok, right=True).sub(1).clamp(max=c["batch"] - 1)
    pos = lens[req] + tok - start[req]
    slot = table[req, (pos // bs).clamp(0, table.shape[1] - 1)].long() * bs + pos % bs
    none = torch.full_like(tok, -1)
    return {"lens": after.int(), "held": need.int(), "head": (s["head"] + fresh.sum()).int(), "start": start.int(),
            "position": torch.where(live, pos, none).int(), "request": torch.where(live, req, none).int(),
            "slot": torch.where(live, slot, none), "table": table}


def _plain_norm_rope(x, w, cos, sin, case):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
    r = case["rotary"]
    if case["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., : r // 2], y[..., r // 2: r]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, y[..., r:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    half = c["rotary"] // 2
    t = s["table"][s["pos"].long()][:, None]
    cos, sin = t[..., :half], t[..., half:]
    return {"q": _plain_norm_rope(s["q"], s["qw"], cos, sin, c), "k": _plain_norm_rope(s["k"], s["kw"], cos, sin, c)}


def _take(codes, at):
    """codes[at] through bytes: not every version indexes 8-bit floats."""
    return codes.view(torch.uint8)[at].view(codes.dtype)


def _plain_append_one(codes, scale, x, blk, off, run, name):
    """x [T, heads, dim] into codes at (blk, off); run: the tokens that open a
    block's run.  A block's scale is the power of two that its largest value
    needs, or the one it has if tokens written before need more."""
    top = E4M3_MAX if name == "e4m3" else I8_MAX
    y = x.float()
    need = torch.zeros_like(scale).index_reduce_(0, blk, y.abs().amax(-1), "amax")
    m, e = torch.frexp(need[blk[run]])           # need = m 2^e, 0.5 <= m < 1; top = limit 2^bits
    limit, bits = math.frexp(top)
    e = torch.where(m > limit, e + 1, e).sub(bits).clamp(min=MIN_EXP)
    e = torch.where(m == 0.0, torch.full_like(e, MIN_EXP), e)
    new = torch.ldexp(torch.ones_like(m), e)
    old, b, first = scale[blk[run]], blk[run], off[run]
    keep = (first > 0)[:, None]
    new = torch.where(keep, torch.maximum(new, old), new)
    before = torch.arange(codes.shape[2], device=DEV)[None] < first[:, None]
    raw = codes.view(torch.uint8)
    was = _take(codes, b).float()
    again = was * (old / new)[:, :, None, None]
    again = again.round() if name == "i8" else again
    raw[b] = torch.where(before[:, None, :, None], again, was).to(codes.dtype).view(torch.uint8)
    scale[b] = new
    z = (y / scale[blk][..., None]).clamp(-top, top)
    raw[blk, :, off] = (z.round() if name == "i8" else z).to(codes.dtype).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    k, v, ks, vs = s["cache"]
    blk, off = s["slots"] // c["block"], s["slots"] % c["block"]
    run = torch.ones_like(blk, dtype=torch.bool)
    run[1:] = blk[1:] != blk[:-1]
    _plain_append_one(k, ks, s["k"], blk, off, run, c["codes"])
    _plain_append_one(v, vs, s["v"], blk, off, run, c["codes"])
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _plain_attend(s):
    c = s["case"]
    b, h, kv, d, bs, n = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["block"], s["most"]
    pages = s["table"][:, : s["columns"]].long().clamp(min=0)
    full = lambda x, sc: (_take(x, pages).float() * sc[pages][..., None, None]).transpose(1, 2).reshape(b, kv, -1, d)  # noqa: E731
    k, v = full(s["cache"][0], s["cache"][2]), full(s["cache"][1], s["cache"][3])
    start, lens = s["start"].long(), s["lens"].long()
    adds = start[1:] - start[:-1]
    i = torch.arange(n, device=DEV)
    q = s["q"][(start[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.reshape(b, n, kv, h // kv, d).permute(0, 2, 1, 3, 4).reshape(b, kv, -1, d)
    logit = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).reshape(b, kv, n, h // kv, -1)
    at = (lens - adds)[:, None] + i[None]
    key = torch.arange(logit.shape[-1], device=DEV)
    seen = (key <= at[..., None]) & (key < lens[:, None, None])
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    seen = seen[:, None, :, None]
    logit.masked_fill_(~seen, -math.inf)
    top = logit.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(logit - top)
    total = e.sum(-1, keepdim=True)
    out = (e.reshape(b, kv, -1, e.shape[-1]) @ v).reshape(b, kv, n, h // kv, d) / total.clamp(min=1e-30)
    back = lambda x: x.permute(0, 2, 1, 3, 4).reshape(b, n, h, -1)[s["req"], s["local"]]  # noqa: E731
    res = {"out": back(out).to(s["q"].dtype)}
    if c["lse"]:
        res["lse"] = back(top + torch.log(total))[..., 0]
    return res


def _plain_verify(s):
    p, q, ids, u, noise = s["p"], s["q"], s["ids"].long(), s["u"], s["noise"]
    b, k = ids.shape
    px = p[:, :k].gather(2, ids[..., None])[..., 0].float()
    qx = q.gather(2, ids[..., None])[..., 0].float()
    stop = torch.cat([~(u * qx < px), torch.ones((b, 1), dtype=torch.bool, device=DEV)], 1).int().argmax(1)
    row = torch.arange(b, device=DEV)
    target = p[row, stop].float()
    draft = torch.where((stop < k)[:, None], q[row, stop.clamp(max=k - 1)].float(), torch.zeros((), device=DEV))
    rest = (target - draft).clamp(min=0.0)
    rest = torch.where((rest.amax(1) > 0)[:, None], rest, target)
    token = torch.where(rest > 0, rest / noise, torch.zeros((), device=DEV)).argmax(1)
    col = torch.arange(k + 1, device=DEV)[None]
    padded = torch.cat([ids, torch.zeros((b, 1), dtype=torch.int64, device=DEV)], 1)
    out = torch.where(col < stop[:, None], padded, torch.where(col == stop[:, None], token[:, None], -1))
    return {"accepted": stop.int(), "ids": out.int()}


PLAIN = {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}


def run(s):
    if not own:
        return PLAIN[s["case"]["op"]](s)
    from spec_verify_gb300 import binding, cache

    c = s["case"]
    if c["op"] == "plan":
        lens, held, head, start, pos, req, slot = cache.block_plan(
            s["lens"], s["add"], s["held"], s["free"], s["head"], s["table"], c["block"], s["blocks"], s["cap"], out=s["out"])
        return {"lens": lens, "held": held, "head": head, "start": start, "position": pos, "request": req, "slot": slot,
                "table": s["table"]}
    if c["op"] == "rope":
        q, k = cache.qk_norm_rope(s["q"], s["k"], s["pos"], s["table"], s["qw"], s["kw"], eps=1e-6,
                                  interleaved=c["interleaved"], out_q=s["oq"], out_k=s["ok"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        cache.cache_append(s["cache"], s["k"], s["v"], s["slots"])
        k, v, ks, vs = s["cache"]
        return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}
    if c["op"] == "attend":
        out = cache.cache_attention(s["cache"], s["q"], s["start"], s["lens"], s["table"], window=c["window"], out=s["out"],
                                    lse=s["lse"], workspace=s["workspace"])
        return {"out": out, "lse": s["lse"]} if c["lse"] else {"out": out}
    accepted, ids = binding.spec_verify_probs(s["p"], s["q"], s["ids"], s["u"], s["noise"], out_accepted=s["accepted"],
                                              out_ids=s["tokens"])
    return {"accepted": accepted, "ids": ids}


# ---------------------------------------------------------------- 64 bits


def _exact_code(z, name):
    """The 8-bit value nearest to z (ties to even), as a 64-bit number."""
    if name == "i8":
        return z.round().clamp(-I8_MAX, I8_MAX)
    z = z.clamp(-E4M3_MAX, E4M3_MAX)
    grid = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3.0)
    return ((z / grid).round() * grid).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s):
    c, bs = s["case"], s["case"]["block"]
    top = E4M3_MAX if c["codes"] == "e4m3" else I8_MAX
    res = {}
    runs, slots = [], s["slots"].tolist()
    for t, slot in enumerate(slots):
        if t == 0 or slot // bs != slots[t - 1] // bs:
            runs.append([t, t + 1, slot // bs, slot % bs])
        else:
            runs[-1][1] = t + 1
    for name, x, codes, scale in (("k", s["k"], s["cache"][0], s["cache"][2]), ("v", s["v"], s["cache"][1], s["cache"][3])):
        codes, scale, x = codes.double(), scale.double(), x.double()
        for lo, hi, blk, off in runs:
            part = x[lo:hi]                                                  # [n, heads, dim]
            need = part.abs().amax((0, 2)) / top
            new = torch.exp2(torch.ceil(torch.log2(need.clamp(min=2.0 ** MIN_EXP))))
            if off:
                new = torch.maximum(new, scale[blk])
                codes[blk, :, :off] = _exact_code(codes[blk, :, :off] * (scale[blk] / new)[:, None, None], c["codes"])
            scale[blk] = new
            codes[blk, :, off:off + hi - lo] = _exact_code(part.transpose(0, 1) / new[:, None, None], c["codes"])
        res[name], res[name + "_scale"] = (codes if c["codes"] == "e4m3" else None), scale
    return res


def _exact_rope(s):
    c, r = s["case"], s["case"]["rotary"]
    table = s["table"].double()[s["pos"].long()][:, None]
    turn = torch.complex(table[..., : r // 2], table[..., r // 2:])
    res = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        y = w.double() * x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["dim"] + 1e-6)
        if c["interleaved"]:
            z = torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], r // 2, 2).contiguous()) * turn
            y[..., :r] = torch.view_as_real(z).reshape(*y.shape[:-1], r)
        else:
            z = torch.complex(y[..., : r // 2].contiguous(), y[..., r // 2: r].contiguous()) * turn
            y[..., : r // 2], y[..., r // 2: r] = z.real, z.imag
        res[name] = y
    return res


def _exact_attend(s):
    c, bs = s["case"], s["case"]["block"]
    kv, group, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    for b, length in enumerate(lens):
        pages = s["table"][b, : -(-length // bs)].long()
        k, v = ((_take(x, pages).double() * sc[pages].double()[..., None, None]).transpose(0, 1).reshape(kv, -1, d)[:, :length]
                for x, sc in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
        n = start[b + 1] - start[b]
        for i in range(n):
            last = length - n + i
            lo = max(0, last - c["window"] + 1) if c["window"] else 0
            q = s["q"][start[b] + i].double().reshape(kv, group, d)
            z = torch.einsum("hgd,htd->hgt", q, k[:, lo:last + 1]) / math.sqrt(d)
            total = torch.logsumexp(z, -1)
            out[start[b] + i] = torch.einsum("hgt,htd->hgd", torch.exp(z - total[..., None]), v[:, lo:last + 1]).reshape(-1, d)
            lse[start[b] + i] = total.reshape(-1)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def exact(case, seed):
    op = case["op"]
    if op in ("plan", "verify"):     # whole numbers alone
        return None
    if op == "append" and case["batch"] * case["add"] > 100000:
        return None                  # one block after another: too long
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[op](s)

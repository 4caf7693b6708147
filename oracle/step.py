"""Plain fp64 forms of the cached speculative step: block plan, norm and
rotation, append to the 8-bit paged cache, attention over it, and the check
of drafts against probabilities.  One request, token or row after another;
shares no code with the CUDA library.
"""

import math

import numpy as np

MIN_EXP = -100
TOP = {"e4m3": 448.0, "i8": 127.0}


def _e4m3_table():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent field 0 is subnormal, 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if c & 0x7F == 0x7F:
            x = math.nan
        out[c] = -x if c & 0x80 else x
    return out


E4M3 = _e4m3_table()
_POSITIVE = E4M3[:0x7F]                      # ascending, 0 .. 448


def decode(codes, kind):
    """fp64 values of an array of bytes."""
    codes = np.asarray(codes)
    return E4M3[codes.view(np.uint8)] if kind == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(x, kind):
    """Bytes of the codes nearest to x (ties to even; beyond the largest code:
    that code; NaN: the NaN code, or 0 for i8)."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    if kind == "i8":
        return np.where(nan, 0, np.clip(np.rint(np.where(nan, 0, x)), -127, 127)).astype(np.int8).view(np.uint8)
    mag = np.minimum(np.abs(np.where(nan, 0, x)), 448.0)
    hi = np.searchsorted(_POSITIVE, mag)                     # first code with value >= mag
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - mag, mag - _POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(x) & ~nan, code | 0x80, code)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def needed_scale(amax, kind):
    """The smallest power of two s >= 2^-100 with amax <= TOP * s."""
    e = MIN_EXP
    if amax > 0:
        e = max(e, math.frexp(amax / TOP[kind])[1] - 2)
        while TOP[kind] * 2.0 ** e < amax:
            e += 1
    return 2.0 ** e


def block_plan(lens, add, held, free_blocks, free_head, table, block_size, num_blocks, max_tokens):
    """Returns a dict of the outputs, the extended table and `status`."""
    batch, stride = len(lens), table.shape[1]
    table = table.copy()
    out = {"lens": [], "held": [], "start": [], "position": [], "request": [], "slot": []}
    status = 0
    head_ok = 0 <= free_head <= len(free_blocks)
    avail = len(free_blocks) - free_head if head_ok else 0
    if not head_ok:
        status |= 16
    tokens = blocks = 0
    full = False
    for b in range(batch):
        length, n, have = int(lens[b]), int(add[b]), int(held[b])
        need = -(-(length + n) // block_size)
        valid = length >= 0 and n >= 0 and length + n < 2 ** 31 and -(-length // block_size) <= have <= stride and need <= stride
        out["start"].append(tokens)
        if not valid:
            status |= 16
        fresh = max(0, need - have)
        if not valid or n == 0:
            out["lens"].append(length)
            out["held"].append(have)
            continue
        if full or tokens + n > max_tokens or blocks + fresh > avail:
            full = True
            status |= 32
            out["lens"].append(length)
            out["held"].append(have)
            continue
        for i in range(fresh):
            table[b, have + i] = free_blocks[free_head + blocks + i]
        blocks += fresh
        tokens += n
        out["lens"].append(length + n)
        out["held"].append(have + fresh)
        for p in range(length, length + n):
            block = int(table[b, p // block_size])
            ok = 0 <= block < num_blocks
            if not ok:
                status |= 64
            out["position"].append(p)
            out["request"].append(b)
            out["slot"].append(block * block_size + p % block_size if ok else -1)
    out["start"].append(tokens)
    for key in ("position", "request", "slot"):
        out[key] += [-1] * (max_tokens - len(out[key]))
    res = {key: np.array(v, dtype=np.int64) for key, v in out.items()}
    res.update(free_head=free_head + blocks, table=table, status=status)
    return res


def norm_rope(x, weight, positions, table, eps, interleaved):
    """x [T, H, D]; table [rows, R] or None.  Returns (y, bound) where bound is
    |a| + |b| of each element's pair (|y| where nothing rotates), the scale of
    its rounding errors.  Padding tokens (position < 0) are left as x."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    bound = np.abs(y)
    rotary = 0 if table is None else table.shape[1]
    out, half = y.copy(), rotary // 2
    for t, pos in enumerate(positions):
        if pos < 0:
            out[t] = x[t]
            continue
        if rotary and pos >= table.shape[0]:
            out[t] = np.nan
            continue
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, half + j)
            c, s = float(table[pos, j]), float(table[pos, half + j])
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            both = np.abs(y[t, :, a]) + np.abs(y[t, :, b])
            bound[t, :, a] = bound[t, :, b] = both
    return out, bound


def append(codes, scale, x, slots, block_size, kind):
    """codes [N, H, bs, D] bytes, scale [N, H] float32, x [T, H, D]: the cache
    after the append, and the status."""
    codes, scale, x = codes.copy(), scale.astype(np.float64), np.asarray(x, dtype=np.float64)
    status, t = 0, 0
    while t < len(slots):
        slot = int(slots[t])
        if slot < 0 or slot >= codes.shape[0] * block_size:
            status |= 16 if slot >= 0 else 0
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slot + n and (slot + n) % block_size:
            n += 1
        block, off = slot // block_size, slot % block_size
        for h in range(codes.shape[1]):
            part = x[t:t + n, h]
            finite = np.isfinite(part)
            if not finite.all():
                status |= 2
            s = needed_scale(float(np.abs(part[finite]).max(initial=0.0)), kind)
            if off:
                old = scale[block, h]
                s = max(s, old)
                if s != old:
                    codes[block, h, :off] = encode(decode(codes[block, h, :off], kind) * (old / s), kind)
            scale[block, h] = s
            codes[block, h, off:off + n] = encode(part / s, kind)
        t += n
    return codes, scale.astype(np.float32), status


def attention(k, v, k_scale, v_scale, kind, q, start, lens, table, scale, window):
    """k, v: bytes [N, H, bs, D].  Returns (out, lse, weight, reach): weight is
    sum_j p_j |v_j|, the scale of an element's rounding errors, and reach the
    largest sum_d |q_d k_jd| * |scale| over the visible keys of a row."""
    q = np.asarray(q, dtype=np.float64)
    t, hq, d = q.shape
    n_blocks, kv, bs, _ = k.shape
    group = hq // kv
    out, weight = np.zeros_like(q), np.zeros_like(q)
    lse, reach = np.full((t, hq), -np.inf), np.zeros((t, hq))
    for b in range(len(lens)):
        n = int(start[b + 1] - start[b])
        for i in range(n):
            p = int(lens[b]) - n + i
            lo = max(0, p - window + 1) if window else 0
            js = [j for j in range(lo, p + 1) if 0 <= table[b, j // bs] < n_blocks]
            if not js:
                continue
            js = np.array(js)
            blk = table[b, js // bs]
            kk = decode(k[blk, :, js % bs], kind) * k_scale[blk][:, :, None].astype(np.float64)    # [n, kv, d]
            vv = decode(v[blk, :, js % bs], kind) * v_scale[blk][:, :, None].astype(np.float64)
            for h in range(hq):
                row = start[b] + i
                z = kk[:, h // group] @ q[row, h] * scale
                top = z.max()
                e = np.exp(z - top)
                total = e.sum()
                out[row, h] = (e / total) @ vv[:, h // group]
                weight[row, h] = (e / total) @ np.abs(vv[:, h // group])
                lse[row, h] = top + math.log(total)
                reach[row, h] = (np.abs(kk[:, h // group]) @ np.abs(q[row, h])).max() * abs(scale)
    return out, lse, weight, reach


def verify_probs(p, q, ids, lens, uniforms, noise):
    """Rows of (accepted, ids, status).  Products, differences and quotients
    are rounded to binary32, as the rule says."""
    f = np.float32
    batch, k1, vocab = p.shape
    out = []
    for b in range(batch):
        k = k1 - 1 if lens is None else int(lens[b])
        if not 0 <= k <= k1 - 1 or any(not 0 <= x < vocab for x in ids[b, :k]):
            out.append((-1, [-1] * k1, 8))
            continue
        stop = k
        for i in range(k):
            x = ids[b, i]
            qx = f(1) if q is None else f(q[b, i, x])
            if not f(uniforms[b, i]) * qx < f(p[b, i, x]):
                stop = i
                break
        w = p[b, stop].astype(f)
        if stop < k:
            minus = np.zeros(vocab, dtype=f)
            if q is None:
                minus[ids[b, stop]] = 1
            else:
                minus = q[b, stop].astype(f)
            rest = w - minus
            if (rest > 0).any():
                w = rest
        best, token = f(0), -1
        for x in np.flatnonzero(w > 0):
            score = w[x] / f(noise[b, x])
            if score > best:
                best, token = score, int(x)
        if token < 0:
            out.append((-1, [-1] * k1, 2))
        else:
            out.append((stop, [int(x) for x in ids[b, :stop]] + [token] + [-1] * (k1 - 1 - stop), 0))
    return out

"""Plain fp64 forms of the calls on rows of logits: log probabilities of tokens
with entropy and likeliest tokens, distillation from a teacher's likeliest
tokens, and their gradients.  Row by row, from the definitions.

`None` in place of a row's result is an error row.
"""

import numpy as np

MIN_T, MAX_T = 2.0 ** -30, 2.0 ** 30
BAD_PARAMS, NONFINITE, BAD_TOKEN = 1, 2, 128


def _row(z, temperature):
    """(ln p, flag) of one row: NaN counts as -inf; flag 0 when it is a row."""
    if not MIN_T <= temperature <= MAX_T:
        return None, BAD_PARAMS
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, dtype=np.float64))
    if not np.isfinite(z.max()):
        return None, NONFINITE
    y = (z - z.max()) / np.float64(temperature)
    return y - np.log(np.exp(y).sum()), 0


def _temperatures(temperature, rows):
    return np.broadcast_to(np.asarray(temperature, dtype=np.float64), (rows,))


def entropy_of(logp):
    live = logp > -np.inf
    return -(np.exp(logp[live]) * logp[live]).sum()


def token_logprobs(z, ids, top, temperature=1.0):
    """Per row: (logprobs [count], entropy, top ids [top], top log probabilities
    [top]); also the flags of the whole call.  ids: [rows, count] or None."""
    out, flags = [], 0
    for r, (row, t) in enumerate(zip(z, _temperatures(temperature, len(z)))):
        mine = [] if ids is None else [int(i) for i in ids[r]]
        if any(i >= len(row) for i in mine):
            flags |= BAD_TOKEN
        logp, bad = _row(row, t)
        flags |= bad
        if logp is None:
            out.append((np.array([0.0 if i < 0 else np.nan for i in mine]), np.nan, np.full(top, -1), np.full(top, np.nan)))
            continue
        given = np.array([0.0 if i < 0 else np.nan if i >= len(row) else logp[i] for i in mine])
        clean = np.where(np.isnan(row), -np.inf, np.asarray(row, dtype=np.float64))
        order = np.argsort(-clean, kind="stable")[:top]
        order = order[clean[order] > -np.inf]
        best, value = np.full(top, -1), np.full(top, -np.inf)
        best[:len(order)], value[:len(order)] = order, logp[order]
        out.append((given, entropy_of(logp), best, value))
    return out, flags


def token_logprobs_grad(z, ids, up, up_entropy, temperature=1.0):
    """The gradient [rows, vocab], a bound of its terms' magnitudes (what an
    error relative to each term is relative to), and the flags."""
    rows, v = np.shape(z)
    grad, reach, flags = np.zeros((rows, v)), np.zeros((rows, v)), 0
    for r, (row, t) in enumerate(zip(z, _temperatures(temperature, rows))):
        mine = [] if ids is None else [(int(i), np.float64(g)) for i, g in zip(ids[r], up[r]) if i >= 0]
        h = 0.0 if up_entropy is None else np.float64(up_entropy[r])
        if not mine and h == 0.0:
            continue
        if any(i >= v for i, _ in mine):
            flags |= BAD_TOKEN
            grad[r] = np.nan
        logp, bad = _row(row, t)
        flags |= bad if not np.isnan(grad[r, 0]) or bad == BAD_PARAMS else 0
        if bad or np.isnan(grad[r, 0]):
            grad[r] = np.nan
            continue
        p, big = np.exp(logp), np.where(logp > -np.inf, logp, 0.0)
        entropy = entropy_of(logp)
        grad[r] = -p * (sum(g for _, g in mine) + h * (big + entropy)) / t
        reach[r] = p * (sum(abs(g) for _, g in mine) + abs(h) * (np.abs(big) + entropy)) / t
        for i, g in mine:
            grad[r, i] += g / t
            reach[r, i] += abs(g) / t
    return grad, reach, flags


def teacher_row(ids, values, tail, vocab):
    """([(id, t, ln t)], r, flag) of one teacher's row; no places: ([], 0, 0)."""
    places = [(int(i), np.float64(v)) for i, v in zip(ids, values) if i >= 0]
    if not places:
        return [], 0.0, 0
    flag = BAD_TOKEN if any(i >= vocab for i, _ in places) else 0
    l = np.array([v for _, v in places])
    if np.isnan(l).any() or (l == np.inf).any():
        return places, 0.0, flag | BAD_PARAMS
    if tail:
        rest = max(0.0, 1.0 - np.exp(l).sum())
        if np.exp(l).sum() > 1.0 + 2.0 ** -6:
            flag |= BAD_PARAMS
    else:
        rest = 0.0
        if l.max() == -np.inf:
            return places, 0.0, flag | BAD_PARAMS
        l = l - l.max() - np.log(np.exp(l - l.max()).sum())
    return [(i, np.exp(v), v) for (i, _), v in zip(places, l)], rest, flag


def distill(z, ids, values, tail, weights=None, temperature=1.0):
    """(loss [rows], gradient [rows, vocab], loss bound, gradient bound, flags):
    the bounds are the sums of the terms' magnitudes."""
    rows, v = np.shape(z)
    loss, grad = np.zeros(rows), np.zeros((rows, v))
    loss_reach, reach, flags = np.zeros(rows), np.zeros((rows, v)), 0
    for r, (row, t) in enumerate(zip(z, _temperatures(temperature, rows))):
        places, rest, flag = teacher_row(ids[r], values[r], tail, v)
        if not places:
            continue
        logp = None
        if MIN_T <= t <= MAX_T:
            if not flag:
                logp, flag = _row(row, t)
        else:
            flag |= BAD_PARAMS
        flags |= flag
        if flag:
            loss[r], grad[r] = np.nan, np.nan
            continue
        w = 1.0 if weights is None else np.float64(weights[r])
        outside = np.ones(v, dtype=bool)
        outside[[i for i, _, _ in places]] = False
        beyond = logp[outside]
        beyond = beyond[beyond > -np.inf]
        if len(beyond) == 0:
            rest = 0.0
        total = 0.0
        for i, share, log_share in places:
            total += share
            if share > 0.0:
                loss[r] += share * (log_share - logp[i])
                loss_reach[r] += share * (abs(log_share) + abs(logp[i]))
        p = np.exp(logp)
        grad[r] = reach[r] = p * (total + rest)
        if rest > 0.0:
            log_rest = beyond.max() + np.log(np.exp(beyond - beyond.max()).sum())
            loss[r] += rest * (np.log(rest) - log_rest)
            loss_reach[r] += rest * (abs(np.log(rest)) + abs(log_rest)) + 2.0 ** -16 * (1 + abs(np.log(rest)) + abs(log_rest))
            part = np.where(outside, np.exp(np.where(outside, logp, -np.inf) - beyond.max()), 0.0)
            part *= rest / part.sum()                       # log_rest may have lost the logarithm of the sum, at masks of -1e38 say
            grad[r] = grad[r] - part
            reach[r] = reach[r] + part
        for i, share, _ in places:
            grad[r, i] -= share
            reach[r, i] += share
        grad[r] *= w / t
        reach[r] *= abs(w) / t
        loss_reach[r] += total + rest
    return loss, grad, loss_reach, reach, flags

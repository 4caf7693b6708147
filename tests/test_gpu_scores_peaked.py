"""Gradients of rows of logits whose likeliest tokens lie far above the rest, up
to where 2^127 is the difference in weight, against the plain forms in 64 bits.

Tolerances are those of test_gpu_scores.py.  With entropies the gradient also has
p h / T times (ln p + H), whose two parts are distances D from a reference that
may nearly cancel: the mean of D is within 2^-16 of itself (the sums it comes
from), and D itself has the rounding of z c and m c, 128 * 2^-24 at most.  D is the
leaders' height above the row's bulk where sums are relative to that: 84 at most,
since 2^121 times 121 is no finite sum; 2^16 of weight else.  A weight below 2^-126 is flushed, and with it
what the gradient multiplies it by: up to 2^-126 (|G| + |h| (|ln p| + H)) / T, of
which |ln p| is 128 ln 2 here (2^-120 alone allows for 64); what is flushed of yet
smaller weights is less, p |ln p| falling with p."""

import numpy as np
import pytest

from oracle import scores as oracle
from spec_verify_gb300 import scores
from tests.test_gpu_scores import DTYPES, _lib, check_distill, check_grad, host, status, torch, up  # noqa: F401

pytestmark = pytest.mark.gpu


def check_scores_grad(view, z, ids, g, h, dtype, temperature, height):
    t = np.float32(temperature)
    far = height if height < 84 else 16 * np.log(2)
    for entropies in (None, h):
        want, reach, flags = oracle.token_logprobs_grad(z, ids, g, entropies, t)
        if entropies is not None:
            share = np.stack([np.exp(oracle._row(row, t)[0]) for row in z])
            reach = reach + share * np.abs(h)[:, None] / t * (far / 2 + 0.25)       # check_grad takes 2^-15 of it
            flushed = np.minimum(np.stack([np.abs(oracle._row(row, t)[0]) for row in z]), 89) + np.log(z.shape[1])
            reach = reach + 2.0 ** (15 - 126) / t * (np.abs(g).sum(1) + np.abs(h) * flushed.T).T
        st = status()
        got = scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), None if entropies is None else up(entropies),
                                         temperature=float(t), status=st)
        assert int(st) == flags == 0
        check_grad(got, want, reach, dtype, t)


def later_units(cluster, vocab, threads, dtype):
    """Places that lie behind every thread's first unit of four vectors."""
    length, at = -(-vocab // cluster), np.arange(vocab)
    return at[at % length >= threads * 4 * (4 if dtype == "f32" else 8)]


def leading_rows(rng, vocab, later, height, temperature, dtype):
    z = np.zeros((8, vocab))
    for r, leaders in enumerate((1, 2, 3, 40, 1000, 2, len(later), 3)):
        at = rng.permutation(later)[:leaders]
        z[r, at] = height
        if r == 5:
            z[r] += rng.normal(0, 0.1, vocab)
        if r == 7:
            z[r, at] += [0.0, -1.0, -3.0]
    return host(up(z * temperature, DTYPES[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cluster,vocab", [(1, 16384), (1, 32768), (1, 32003), (4, 131072)])
@pytest.mark.parametrize("temperature", [1.0, 0.1, 3.0])
@pytest.mark.parametrize("height", [14.0, 40.0, 60.0, 83.5, 86.0, 88.5])
def test_leaders_far_above_the_first_units(height, temperature, cluster, vocab, dtype, monkeypatch):
    monkeypatch.setenv("SMP_FORCE_CLUSTER", str(cluster))
    rng = np.random.default_rng(int(height * 10) + vocab)
    later = later_units(cluster, vocab, 256, dtype)
    z = leading_rows(rng, vocab, later, height, temperature, dtype)
    view = up(z, DTYPES[dtype])
    ids = np.stack([z.argmax(1), rng.integers(0, vocab, 8), rng.permutation(later)[:8]], 1)
    g, h = rng.normal(0, 1, (8, 3)).astype(np.float32), rng.normal(0, 1, 8).astype(np.float32)
    check_scores_grad(view, z, ids, g, h, dtype, temperature, height)
    values = np.log(rng.dirichlet(np.ones(4), 8)[:, :3]).astype(np.float32)
    weight = (2.0 ** -12 * rng.normal(0, 1, 8)).astype(np.float32)
    for places in (ids, rng.integers(0, 4096, (8, 3))):                   # on the leaders, and off them
        check_distill(view, z, places, values, dtype, temperature=temperature, weight=weight)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("height", [60.0, 86.0, 88.5])
def test_leaders_in_many_rows(height, dtype):
    """Rows enough for small thread blocks, whose results are those of the first eight."""
    rng = np.random.default_rng(int(height))
    vocab = 8192 if dtype == "f32" else 16384
    z = leading_rows(rng, vocab, later_units(1, vocab, 128, dtype), height, 1.0, dtype)
    view = up(np.tile(z, (60, 1)), DTYPES[dtype])
    ids = np.stack([z.argmax(1), rng.integers(0, vocab, 8)], 1)
    g, values = rng.normal(0, 1, (8, 2)).astype(np.float32), np.log(rng.dirichlet(np.ones(3), 8)[:, :2]).astype(np.float32)
    every = lambda a: up(np.tile(a, (60, 1)))  # noqa: E731
    got = scores.token_logprobs_grad(view, every(ids).int(), every(g))
    want, reach, _ = oracle.token_logprobs_grad(z, ids, g, None)
    check_grad(got[:8], want, reach, dtype)
    loss, dz = scores.distill_grad(view, every(ids).int(), every(values), tail=True)
    _, want, _, reach, _ = oracle.distill(z, ids, values, 1)
    check_grad(dz[:8], want, reach, dtype)
    for t in (got, loss, dz):
        assert all(torch.equal(t[8 * i:8 * i + 8], t[:8]) for i in range(60))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distillation_with_the_rest_between_bulk_and_ids(dtype, monkeypatch):
    """The ids lie more than 126 binary orders above the first units, the rest's top a
    little below the ids."""
    monkeypatch.setenv("SMP_FORCE_CLUSTER", "1")
    rng = np.random.default_rng(6)
    later = later_units(1, 32768, 256, dtype)
    z, ids = np.zeros((6, 32768)), np.empty((6, 2), dtype=int)
    for r in range(6):
        at = rng.permutation(later)[:12]
        ids[r] = at[:2]
        z[r, at[:2]], z[r, at[2:]] = 92.0 + 4 * r, 80.0 + 4 * min(r, 2) - rng.uniform(0, 3, 10)
    z = host(up(z, DTYPES[dtype]))
    values = np.log(rng.dirichlet(np.ones(3), 6)[:, :2]).astype(np.float32)
    check_distill(up(z, DTYPES[dtype]), z, ids, values, dtype)

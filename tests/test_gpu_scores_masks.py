"""Gradients of rows that are masked with large finite numbers: with entropies, in
slices of whole units (tolerances of test_gpu_scores_peaked.py), and distillation
from teachers who leave masked tokens alone (tolerances of test_gpu_scores.py)."""

import numpy as np
import pytest

from tests.test_gpu_scores import DTYPES, _lib, check_distill, host, torch, up  # noqa: F401
from tests.test_gpu_scores_peaked import check_scores_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [8192, 16384])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 2.0, 4.0])
@pytest.mark.parametrize("bonus", [10.0, -10.0, 1.0, 0.01])
def test_finite_masks(bonus, temperature, vocab, dtype, monkeypatch):
    monkeypatch.setenv("SMP_FORCE_CLUSTER", "1")
    rng = np.random.default_rng(vocab)
    masks = (float(torch.finfo(DTYPES[dtype]).min), -1e38, -3e38, -1e30)
    z = rng.normal(-20, 1, (len(masks), vocab))
    for r, mask in enumerate(masks):                      # every thread keeps tokens that may be said
        z[r, ::2] = mask
    z[:, 1], z[:, 5] = 0.0, -1.5
    z = host(up(z, DTYPES[dtype]))
    ids = np.stack([np.full(len(z), 1), rng.integers(0, vocab, len(z))], 1)
    g, h = rng.normal(0, 1, (len(z), 2)).astype(np.float32), np.full(len(z), bonus, dtype=np.float32)
    check_scores_grad(up(z, DTYPES[dtype]), z, ids, g, h, dtype, temperature, 24 / temperature)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [5, 300, 16384])
@pytest.mark.parametrize("mask", [-1e4, -1e38, "lowest"])
def test_only_masked_tokens_outside_the_teachers_ids(mask, vocab, dtype):
    mask = float(torch.finfo(DTYPES[dtype]).min) if mask == "lowest" else mask
    rng = np.random.default_rng(vocab)
    ids = np.stack([rng.permutation(vocab)[:3] for _ in range(4)])
    z = np.full((4, vocab), mask)
    np.put_along_axis(z, ids, rng.normal(0, 2, (4, 3)), 1)
    z[1, ids[1, 0]] = mask
    z[2, rng.integers(0, vocab)] = 1.0
    z = host(up(z, DTYPES[dtype]))
    values = np.log(rng.dirichlet(np.ones(4), 4)[:, :3]).astype(np.float32)
    for temperature in (0.1, 1.0, 3.0):
        check_distill(up(z, DTYPES[dtype]), z, ids, values, dtype, temperature=temperature)

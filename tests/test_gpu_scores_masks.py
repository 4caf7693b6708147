"""Gradients with entropies of rows that are masked with large finite numbers, in
slices of whole units.  Tolerances are those of test_gpu_scores_peaked.py."""

import numpy as np
import pytest

from tests.test_gpu_scores import DTYPES, _lib, host, torch, up  # noqa: F401
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

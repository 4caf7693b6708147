"""The oracle's distillation where only tokens of large finite masks are left outside
the teacher's ids: equal tokens share the rest equally, and a gradient sums to 0."""

import numpy as np
import pytest

from oracle import scores


@pytest.mark.parametrize("mask", [-1e4, -1e16, -1e30, -1e38, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("temperature", [0.1, 1.0, 3.0])
def test_masked_tokens_share_the_rest(mask, temperature):
    z = np.array([[0.5, 1.0, mask, mask, mask], [0.5, mask, mask, mask, mask]])
    values = np.log([[0.5, 0.3], [0.5, 0.3]])
    _, grad, _, _, flags = scores.distill(z, [[0, 1], [0, 1]], values, 1, None, temperature)
    assert flags == 0
    assert np.abs(grad[:, 2:] + 0.2 / 3 / temperature).max() <= 2.0 ** -50 / temperature
    assert np.abs(grad.sum(1)).max() <= 2.0 ** -50 / temperature

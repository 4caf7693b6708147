"""Pins of the plain forms of log probabilities, distillation and their
gradients: hand values, identities and differences."""

import numpy as np
import pytest

from oracle import scores as o


def test_log_probabilities_by_hand():
    # odds 1 : 2 : 5, so p = 1/8, 1/4, 5/8
    z = np.log([[1.0, 2.0, 5.0]])
    (given, entropy, ids, value), = o.token_logprobs(z, [[2, -1, 0, 3]], 5)[0]
    assert np.allclose(given[[0, 2]], np.log([5 / 8, 1 / 8])) and given[1] == 0 and np.isnan(given[3])
    assert np.isclose(entropy, (1 / 8) * np.log(8) + (1 / 4) * np.log(4) + (5 / 8) * np.log(8 / 5))
    assert list(ids) == [2, 1, 0, -1, -1] and np.allclose(value[:3], np.log([5 / 8, 1 / 4, 1 / 8])) and value[3] == -np.inf
    assert o.token_logprobs(z, [[3]], 0)[1] == o.BAD_TOKEN


def test_temperature_masks_ties_and_empty_rows():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, np.nan]])
    (_, entropy, ids, value), = o.token_logprobs(z, None, 3, temperature=2.0)[0]
    assert list(ids) == [1, 2, 0]                                # the lower id first
    assert np.isclose(value[0] - value[2], 1.0)                  # ratio e^((3 - 1) / 2)
    assert np.isclose(entropy, o.token_logprobs(z[:, :3], None, 0, temperature=2.0)[0][0][1])
    uniform = o.token_logprobs(np.zeros((1, 64)), None, 0)[0][0]
    assert np.isclose(uniform[1], np.log(64))
    for bad, flag in ((np.full((1, 4), -np.inf), 2), (np.array([[0.0, np.inf]]), 2)):
        out, flags = o.token_logprobs(bad, [[0]], 2)
        assert flags == flag and np.isnan(out[0][0][0]) and list(out[0][2]) == [-1, -1]
    assert o.token_logprobs(np.zeros((1, 4)), [[0]], 0, temperature=0.0)[1] == o.BAD_PARAMS


def test_divergence_by_hand():
    z = np.log([[1.0, 2.0, 5.0]])
    # tail: the teacher gives 1/2 to token 2 and 1/2 to the rest; the student 5/8 and 3/8
    loss, grad, *_ = o.distill(z, [[2]], np.log([[0.5]]), 1)
    assert np.isclose(loss[0], 0.5 * np.log(0.5 / (5 / 8)) + 0.5 * np.log(0.5 / (3 / 8)))
    assert np.allclose(grad[0], [1 / 8 - 0.5 / 3, 2 / 8 - 1 / 3, 5 / 8 - 0.5])
    # no tail: one token, renormalised to 1: the cross entropy
    loss, grad, *_ = o.distill(z, [[2]], np.log([[0.5]]), 0)
    assert np.isclose(loss[0], -np.log(5 / 8)) and np.allclose(grad[0], [1 / 8, 2 / 8, -3 / 8])


def test_a_complete_teacher_gives_the_whole_divergence_and_its_own_rows_none():
    rng = np.random.default_rng(0)
    z, y = rng.normal(0, 2, (4, 9)), rng.normal(0, 2, (4, 9))
    logp, logt = (x - np.log(np.exp(x).sum(-1, keepdims=True)) for x in (z, y))
    ids = np.tile(rng.permutation(9), (4, 1))
    want = (np.exp(logt) * (logt - logp)).sum(-1)
    for tail in (0, 1):
        loss, grad, *_ = o.distill(z, ids, np.take_along_axis(logt, ids, 1), tail)
        assert np.allclose(loss, want) and np.allclose(grad, np.exp(logp) - np.exp(logt))
    own = np.argsort(-z, 1)[:, :4]
    loss, grad, *_ = o.distill(z, own, np.take_along_axis(logp, own, 1), 1)
    assert np.allclose(loss, 0) and np.allclose(grad, 0)          # the student is the teacher


@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.5])
def test_gradients_against_differences(temperature):
    rng = np.random.default_rng(1)
    v, eps = 11, 1e-5
    z = rng.normal(0, 2, (1, v))
    z[0, 4] = -np.inf
    ids, up, h = [[3, -1, 7, 3]], rng.normal(0, 1, (1, 4)), [0.6]
    t_ids = [[5, 2, -1, 5]]
    values = np.log([[0.2, 0.3, 0.1, 0.25]])

    def total(kind, x):
        if kind == "scores":
            (given, entropy, _, _), = o.token_logprobs(x, ids, 0, temperature)[0]
            return (given * up[0]).sum() + h[0] * entropy
        return 1.7 * o.distill(x, t_ids, values, kind == "tail", temperature=temperature)[0][0]

    for kind in ("scores", "tail", "top"):
        if kind == "scores":
            grad = o.token_logprobs_grad(z, ids, up, h, temperature)[0]
        else:
            grad = o.distill(z, t_ids, values, kind == "tail", [1.7], temperature)[1]
        for j in range(v):
            if j == 4:
                assert grad[0, j] == 0.0
                continue
            e = np.zeros((1, v))
            e[0, j] = eps
            assert abs((total(kind, z + e) - total(kind, z - e)) / (2 * eps) - grad[0, j]) < 1e-8, (kind, j)
        assert abs(grad.sum()) < 1e-12                           # a constant added to a row changes nothing


def test_rows_that_are_no_tokens():
    z = np.full((1, 5), np.nan)
    loss, grad, *_, flags = o.distill(z, [[-1, -1]], [[np.nan, 0.0]], 1)
    assert loss[0] == 0 and not grad.any() and flags == 0
    grad, _, flags = o.token_logprobs_grad(z, [[-1]], [[3.0]], [0.0])
    assert not grad.any() and flags == 0
    assert o.distill(np.zeros((1, 5)), [[0, 1]], [[-0.1, -0.1]], 1)[4] == o.BAD_PARAMS    # sums to 1.8
    assert o.distill(np.zeros((1, 5)), [[0, 1]], [[-np.inf, -np.inf]], 0)[4] == o.BAD_PARAMS
    # a student without mass outside the ids: the tail is left out
    loss, grad, *_ = o.distill(np.array([[0.0, 0.0, -np.inf]]), [[0, 1]], np.log([[0.25, 0.25]]), 1)
    assert np.isclose(loss[0], 0.5 * np.log(0.5)) and np.allclose(grad, 0)

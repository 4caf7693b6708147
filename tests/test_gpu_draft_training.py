"""The calls on rows of logits together, as examples/draft_training.py runs them:
the record, both gradients in the logits against their plain fp64 forms (bounds:
those of test_gpu_scores.py) and in the parameters against fp64 products of the
logits' gradients (n roundings of 2^-24 in a sum of n binary32 products)."""

import importlib.util
import os

import numpy as np
import pytest

from oracle import scores as oracle
from spec_verify_gb300 import binding, scores

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_training.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    spec = importlib.util.spec_from_file_location("draft_training", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(got, want, reach, step):
    assert (np.abs(host(got) - want) <= 2.0 ** -15 * reach + step * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -120).all()


def check_head(model, tokens, grad):
    """d head = hidden^T grad, of the model's own hidden rows."""
    hidden = host(model.embed[tokens] * model.embed.shape[1] ** -0.5)
    dz = host(grad)
    bound = (len(tokens) + 2) * 2.0 ** -24 * (np.abs(hidden).T @ np.abs(dz)) + 2.0 ** -120
    assert (np.abs(host(model.head.grad) - hidden.T @ dz) <= bound).all()


@pytest.mark.parametrize("dtype,step", [(torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)])
@pytest.mark.parametrize("rows,vocab,top", [(1, 50, 5), (37, 1003, 16), (300, 2000, 32)])
def test_training_steps(example, rows, vocab, top, dtype, step):
    g = torch.Generator("cuda").manual_seed(rows)
    target, model = example.Draft(vocab, 24, dtype, seed=1), example.Draft(vocab, 16, dtype, seed=2)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    with torch.no_grad():
        wanted = target(tokens)
        record = scores.token_logprobs(wanted, top=top)
        emitted = torch.multinomial(wanted.float().softmax(-1), 1, generator=g)[:, 0].int()
    if rows > 5:
        emitted[3] = -1
    optimizer = torch.optim.SGD(model.parameters(), lr=0.5)
    ids, values = record.top_ids.cpu().numpy(), record.top_logprobs.cpu().numpy()
    for _ in range(3):
        optimizer.zero_grad()
        loss, logits, grad = example.distill(model, tokens, record)
        want, dwant, lreach, reach, flags = oracle.distill(host(logits), ids, values, 1, np.full(rows, np.float32(1 / rows)))
        assert flags == 0 and (np.abs(host(loss) - want) <= 2.0 ** -16 * (1 + 2.0 ** -5 * lreach)).all()
        close(grad, dwant, reach, step)
        check_head(model, tokens, grad)
        optimizer.step()
        optimizer.zero_grad()
        value, logits, grad = example.follow(model, tokens, emitted)
        live = (emitted.cpu().numpy() >= 0).astype(np.float32)
        n = np.float32(max(live.sum(), 1))
        dwant, reach, flags = oracle.token_logprobs_grad(host(logits), emitted.cpu().numpy()[:, None], (-live / n)[:, None],
                                                         np.float32(-0.01) * live / n)
        assert flags == 0
        close(grad, dwant, reach, step * (1 + 2.0 ** -6) + 2.0 ** -22)      # the weights' own roundings: 2 steps of 2^-24
        check_head(model, tokens, grad)
        optimizer.step()
        assert np.isfinite(float(value))


def test_bad_tokens_are_reported(example):
    model = example.Draft(60, 8)
    tokens = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(RuntimeError, match="past the vocabulary"):
        example.follow(model, tokens, torch.tensor([1, 2, 60, -1], dtype=torch.int32, device="cuda"))

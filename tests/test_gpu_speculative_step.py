"""The calls of a cached speculative step together, as examples/speculative_step.py
runs them: every step's attention against its plain fp64 form over the cache as
it stands (bounds: those of the attention for bf16 queries, 2^-9 of the sum of
p |v| for the weights' two roundings, 2^-16 of the largest sum |q k| for the
scores, 2^-8 of the result), the bookkeeping of tokens and lengths, and the
same tokens from a second run."""

import importlib.util
import os

import numpy as np
import pytest

from oracle import step
from spec_verify_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_step.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    spec = importlib.util.spec_from_file_location("speculative_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def check_attention(model, plan):
    kv, q, plan, table, out = model.attended
    kind = "i8" if kv[0].dtype == torch.int8 else "e4m3"
    arrays = [host(t.view(torch.uint8)) for t in kv[:2]] + [host(t) for t in kv[2:]]
    want, _, weight, reach = step.attention(*arrays, kind, host(q), host(plan.start), host(plan.lens), host(table),
                                            q.shape[2] ** -0.5, 0)
    limit = 2.0 ** -9 * weight + 2.0 ** -16 * reach[:, :, None] * weight + 2.0 ** -8 * np.abs(want)
    assert (np.abs(host(out) - want) <= limit + 1e-30).all()


@pytest.mark.parametrize("batch,drafts,steps,codes", [
    (1, 1, 12, "float8_e4m3fn"),
    (3, 4, 8, "int8"),
    (6, 7, 5, "float8_e4m3fn"),
])
def test_generation(example, batch, drafts, steps, codes):
    run = lambda hook: example.generate(  # noqa: E731
        example.Target(vocab=300, blocks=40, codes=getattr(torch, codes)), batch, drafts, steps, prompt=40, after_step=hook)
    accepted, ids, lens = run(check_attention)
    acc, rows = accepted.cpu().numpy(), ids.cpu().numpy()
    assert acc.shape == (steps, batch) and rows.shape == (steps, batch, drafts + 1)
    assert (acc >= 0).all() and (acc <= drafts).all()
    live = np.arange(drafts + 1)[None, None] <= acc[:, :, None]
    assert (rows[live] >= 0).all() and (rows[live] < 300).all() and (rows[~live] == -1).all()
    prompts = np.array([(7 * b + 3) % 40 for b in range(batch)])           # less the last token of each
    assert np.array_equal(lens.cpu().numpy(), prompts + (acc + 1).sum(0))
    again = run(None)
    assert all(torch.equal(a, b) for a, b in zip((accepted, ids, lens), again))


def test_a_full_cache_is_reported(example):
    with pytest.raises(RuntimeError, match="too few blocks"):
        example.generate(example.Target(vocab=300, blocks=1), 2, 4, 1, prompt=5)      # two requests, one block

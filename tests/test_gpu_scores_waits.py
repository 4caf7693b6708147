"""Gradients whose copies have not landed when the wait for them runs out.  With a
limit of 0 the copy's barrier is looked at once, right after the copy was asked for
from HBM, which takes hundreds of nanoseconds: rows are late, and marked."""

import pytest

from spec_verify_gb300 import binding, scores
from tests.test_gpu_scores import _lib, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("call", ["grad", "distill"])
@pytest.mark.parametrize("rows,vocab", [(300, 50021), (1500, 128256)])      # pairs of CTAs or fours; small blocks
def test_late_rows_are_marked_and_the_others_right(rows, vocab, call, dtype, monkeypatch):
    g = torch.Generator("cuda").manual_seed(rows)
    logits = torch.randn(rows, vocab, generator=g, device="cuda").to(dtype)
    ids = torch.randint(0, vocab, (rows, 3), generator=g, device="cuda").int()
    up, h = torch.randn(rows, 3, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    values = torch.full((rows, 3), -1.5, device="cuda")

    def run(st):
        if call == "grad":
            return [scores.token_logprobs_grad(logits, ids, up, h, status=st)]
        loss, grad = scores.distill_grad(logits, ids, values, tail=True, status=st)
        return [grad, loss[:, None]]

    st = status()
    want = run(st)
    assert int(st) == 0
    monkeypatch.setenv("SMP_WAIT_LIMIT_NS", "0")
    got = run(st)
    late = torch.isnan(got[0]).any(1)
    assert bool(late.any()) and int(st) == binding.ROW_TIMEOUT
    assert all(torch.equal(a[~late], b[~late]) and bool(torch.isnan(a[late]).all()) for a, b in zip(got, want))
    monkeypatch.delenv("SMP_WAIT_LIMIT_NS")
    assert all(torch.equal(a, b) for a, b in zip(run(st), want)) and int(st) == 0

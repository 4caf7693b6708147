"""The cached step's calls with `stream=` given: on a stream of their own,
while the current one allocates, fills and frees memory, they give what they
give on the current stream."""

import numpy as np
import pytest

from spec_verify_gb300 import binding, cache
from tests.test_gpu_step import i32, status

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def a_step(state, stream):
    lens, add, held, free, head, table, x, rope, kv, probs = state
    table, kv = table.clone(), tuple(t.clone() for t in kv)
    st = [status() for _ in range(5)]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    plan = cache.block_plan(lens, add, held, free, head, table, 16, 900, 160, status=st[0], stream=stream)
    q, k = cache.qk_norm_rope(x[:, :32], x[:, 32:40], plan.position, rope, status=st[1], stream=stream)
    cache.cache_append(kv, k, x[:, 40:], plan.slot, status=st[2], stream=stream)
    out = cache.cache_attention(kv, q, plan.start, plan.lens, table, status=st[3], stream=stream)
    acc, ids = binding.spec_verify_probs(*probs, status=st[4], stream=stream)
    return [*plan, table, q, k, *kv, out, acc, ids, *st]


def test_calls_on_a_stream_of_their_own():
    rng = np.random.default_rng(1)
    g = torch.Generator("cuda").manual_seed(1)
    lens = rng.integers(1, 300, 32)
    held = -(-lens // 16)
    table, ids = np.full((32, 24), -1), rng.permutation(900)
    for b in range(32):
        table[b, :held[b]] = ids[held[:b].sum():held[:b + 1].sum()]
    kv = list(cache.new_cache(900, 8, 16, 128))
    for i in range(2):
        kv[i] = torch.randn(900, 8, 16, 128, generator=g, device="cuda").mul_(60).to(torch.float8_e4m3fn)
        kv[2 + i].fill_(1 / 64)
    p = torch.randn(32, 5, 3000, generator=g, device="cuda").softmax(-1)
    q = torch.randn(32, 4, 3000, generator=g, device="cuda").softmax(-1)
    probs = (p, q, torch.randint(0, 3000, (32, 4), generator=g, device="cuda", dtype=torch.int32),
             torch.rand(32, 4, generator=g, device="cuda"),
             torch.empty(32, 3000, device="cuda").exponential_(generator=g).clamp_(min=1e-30))
    x = torch.randn(160, 48, 128, generator=g, device="cuda").to(torch.bfloat16)
    state = (i32(lens), i32([5] * 32), i32(held), i32(ids[held.sum():]), i32([0]), i32(table), x, cache.rope_table(400, 128),
             tuple(kv), probs)
    want = a_step(state, None)
    torch.cuda.synchronize()
    assert all(int(s) == 0 for s in want[-5:])
    raw = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
    want = [raw(t).clone() for t in want]
    side = torch.cuda.Stream()
    for _ in range(10):
        got = a_step(state, side)
        for mb in (1, 2, 4, 8, 16, 32, 64):                      # what the calls had for themselves is not handed out here
            torch.full((mb << 18,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(raw(a), b) for a, b in zip(got, want))

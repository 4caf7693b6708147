"""Every kernel and size of the cached step's attention, batches that its CTAs
go through in several rounds, and offsets past 32 bits.  Bounds: those of
tests/test_gpu_step.py; the large layouts are compared with the same call on a
small one, bit for bit."""

import numpy as np
import pytest

from oracle import step
from spec_verify_gb300 import binding, cache
from tests.test_gpu_step import CODES, DT, attention_case, check_attention, check_plan, cuda, i32, status

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


@pytest.mark.parametrize("kind,dt", [("e4m3", "bf16"), ("i8", "bf16"), ("e4m3", "f32"), ("i8", "f32")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [0, 43, 70])
def test_row_tiles(tokens, d, kind, dt):
    # One request adds n tokens, 20 others one in all: rows of q past them set how many rows per key head the call
    # expects (about 4, 20 or 33: a kernel each), n how many the longest request has (8 to 56: every row tile, and
    # more than one of them).
    for n in (1, 2, 3, 4, 5, 7):
        rng = np.random.default_rng(n + d)
        adds, lens = [0] * 21, [3] * 21
        adds[2], lens[2], adds[20], lens[20] = n, 130 + n, 1, 19
        arrays, table, start, lens, q = attention_case(rng, adds, lens, 8, 1, d, 16, kind, dt)
        if tokens:
            q = torch.cat([q, torch.ones(tokens - q.shape[0], 8, d, dtype=q.dtype, device="cuda")])
        check_attention(arrays, kind, q, start, lens, table, dt)


@pytest.mark.parametrize("kind,dt", [("e4m3", "bf16"), ("i8", "f32")])
@pytest.mark.parametrize("batch", [64, 65, 129, 300])
@pytest.mark.parametrize("window", [0, 11])
def test_large_ragged_batches(batch, window, kind, dt):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 90, batch)
    adds = np.minimum(rng.integers(0, 4, batch), lens)           # empty requests among them
    adds[-1], lens[-1] = 2, 50
    arrays, table, start, lens, q = attention_case(rng, adds, lens, 4, 2, 64, 16, kind, dt)
    check_attention(arrays, kind, q, start, lens, table, dt, window=window)


def test_a_batch_whose_last_requests_alone_have_tokens():
    rng = np.random.default_rng(5)
    adds, lens = [0] * 200, [7] * 200
    adds[197], lens[197], adds[199], lens[199] = 3, 600, 1, 1
    arrays, table, start, lens, q = attention_case(rng, adds, lens, 8, 2, 128, 16, "e4m3", "bf16")
    check_attention(arrays, "e4m3", q, start, lens, table, "bf16")


# ---------------------------------------------------------------- past 32 bits


def far_and_near(kind, blocks, heads, bs, d, used):
    """An uninitialised cache of `blocks` blocks and one of the `used` ones
    alone, with the same contents there."""
    g = torch.Generator("cuda").manual_seed(1)
    raw = [torch.randint(0, 120, (len(used), heads, bs, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scale = [2.0 ** torch.randint(-7, -3, (len(used), heads), generator=g, device="cuda").float() for _ in range(2)]
    near = (*(x.clone().view(CODES[kind]) for x in raw), *(x.clone() for x in scale))
    at = torch.tensor(used, device="cuda")
    big = [torch.empty(blocks, heads, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y in zip(big, raw):
        x[at] = y
    far_scale = [torch.ones(blocks, heads, device="cuda") for _ in range(2)]
    for x, y in zip(far_scale, scale):
        x[at] = y
    return (*(x.view(CODES[kind]) for x in big), *far_scale), near, at


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_a_cache_of_more_than_four_gigabytes(kind):
    heads, bs, d = 8, 16, 256
    blocks = 2 ** 32 // (heads * bs * d) + 9                     # a block's first byte passes 2^32
    used = [blocks - 1, 3, blocks - 5, blocks // 2 + 1, blocks - 2, 0]
    far, near, at = far_and_near(kind, blocks, heads, bs, d, used)
    assert (blocks - 5) * heads * bs * d >= 2 ** 32
    g = torch.Generator("cuda").manual_seed(2)
    kv = torch.randn(37, 2 * heads, d, generator=g, device="cuda").to(torch.bfloat16)
    slots = []                                                   # in near's ids: 37 tokens from offset 9 of block 0 on
    for i in range(37):
        slots.append((9 + i) // bs * bs + (9 + i) % bs)
    slots = torch.tensor(slots, device="cuda")
    for c, s in ((near, slots), (far, at[slots // bs] * bs + slots % bs)):
        cache.cache_append(c, kv[:, :heads], kv[:, heads:], s)
    for x, y in zip(far, near):
        assert torch.equal(x.view(torch.uint8)[at].view(torch.uint8) if x.dim() == 4 else x[at],
                           y.view(torch.uint8) if y.dim() == 4 else y)
    q = torch.randn(5, 16, d, generator=g, device="cuda").to(torch.bfloat16)
    start, lens = i32([0, 3, 5]), i32([60, 31])
    table = torch.tensor([[0, 1, 2, 3], [4, 5, 0, 0]], dtype=torch.int32, device="cuda")
    outs = [cache.cache_attention(c, q, start, lens, t) for c, t in ((near, table), (far, at[table.long()].int()))]
    assert torch.equal(*outs) and outs[0].isfinite().all()
    assert torch.equal(near[0].view(torch.uint8), far[0].view(torch.uint8)[at])          # only read


def test_rows_past_32_bits():
    # tokens 2^30 elements apart: the third one begins at 2^31 elements
    apart, rng = 2 ** 30, np.random.default_rng(3)
    bufs = [torch.empty(2 * apart + 4096, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x = cuda(rng.normal(0, 1, (3, 12, 64)).astype(np.float32), DT["bf16"])
    wide = bufs[0].as_strided((3, 12, 64), (apart, 64, 1))
    wide.copy_(x)
    table, pos = cache.rope_table(20, 64), i32([3, 9, 19])
    out = bufs[1].as_strided((3, 8, 64), (apart, 64, 1))
    want, want_k = cache.qk_norm_rope(x[:, :8], x[:, 8:10], pos, table)
    _, got_k = cache.qk_norm_rope(wide[:, :8], wide[:, 8:10], pos, table, out_q=out)
    assert torch.equal(out, want) and torch.equal(got_k, want_k)
    odd = cache.rope_table(20, 60)                               # a size of the general form
    want, _ = cache.qk_norm_rope(x[:, :8], None, pos, odd)
    cache.qk_norm_rope(wide[:, :8], None, pos, odd, out_q=out)
    assert torch.equal(out, want)
    a, b = cache.new_cache(4, 2, 16, 64), cache.new_cache(4, 2, 16, 64)
    slots = torch.tensor([17, 18, 19], device="cuda")
    cache.cache_append(a, x[:, 8:10], x[:, 10:], slots)
    cache.cache_append(b, wide[:, 8:10], wide[:, 10:], slots)
    assert all(torch.equal(y.view(torch.uint8), z.view(torch.uint8)) for y, z in zip(a, b))
    where = (i32([0, 3]), i32([4]), i32([[1]]))
    want = cache.cache_attention(a, x[:, :8], *where)
    cache.cache_attention(a, wide[:, :8], *where, out=out)
    assert torch.equal(out, want)


def test_probabilities_past_32_bits():
    b, k, v = 1600, 8, 152064                                    # 2.2 * 10^9 target probabilities
    p = torch.zeros(b, k + 1, v, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(b, k, v, dtype=torch.bfloat16, device="cuda")
    noise = torch.ones(b, v, device="cuda")
    assert (b - 3) * (k + 1) * v > 2 ** 31 and (b - 3) * k * v * 2 > 2 ** 31
    g = torch.Generator("cuda").manual_seed(4)
    p[-3:] = torch.randn(3, k + 1, v, generator=g, device="cuda").softmax(-1).to(p.dtype)
    q[-3:] = torch.randn(3, k, v, generator=g, device="cuda").softmax(-1).to(q.dtype)
    noise[-3:] = torch.empty(3, v, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    ids = torch.randint(0, v, (b, k), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(b, k, generator=g, device="cuda") * 0.5
    acc, out = binding.spec_verify_probs(p, q, ids, u, noise)
    near = binding.spec_verify_probs(p[-3:].clone(), q[-3:].clone(), ids[-3:].clone(), u[-3:].clone(), noise[-3:].clone())
    assert torch.equal(acc[-3:], near[0]) and torch.equal(out[-3:], near[1]) and (acc[-3:] >= 0).all()
    assert (acc[:-3] == -1).all()                                # rows of zeros


def test_slots_past_32_bits():
    lens, add, held = np.array([250, 0, 16]), np.array([20, 700, 1]), np.array([1, 0, 1])
    blocks = 2 ** 31 - 1
    table = np.full((3, 5), -1)
    table[0, 0], table[2, 0] = blocks - 1, 7
    free = blocks - 2 - np.arange(9)
    want = step.block_plan(lens, add, held, free, 0, table, 256, blocks, 800)
    assert want["slot"].max() > 2 ** 38
    assert check_plan(lens, add, held, free, 0, table, 256, blocks, 800) == 0
    st = status()
    cache.block_plan(i32(lens), i32(add), i32(held), i32(free + 2), i32([0]), i32(table), 256, blocks, 800, status=st)
    assert int(st) == binding.ROW_BAD_BLOCK                      # the first of these ids is no block

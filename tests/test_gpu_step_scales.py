"""The cached step's attention over blocks of very small and very large value
scales: smp_cache_append writes scales from 2^-100 on.  A weight enters its
product with 11 bits (22 for binary32 queries), and one far below the largest
is off by at most 2^-25 of the largest weight P v where the scales are below
2^-92 (2^-33 above): the bounds add that floor, n keys times 2^-25 times the
largest scale times the largest code, to the attention's own (2^-9 or 2^-15 of
sum p |v|, 2^-16 of the largest sum |q k|, 2^-8 of a bf16 result)."""

import numpy as np
import pytest

from oracle import step
from spec_verify_gb300 import binding, cache
from tests.test_gpu_step import attention_case, host, i32, status, upload

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def check(arrays, kind, q, start, lens, table, dt, floor=True):
    d, t = q.shape[2], int(start[-1])
    lse, st = torch.zeros(q.shape[:2], device="cuda"), status()
    got = host(cache.cache_attention(upload(arrays, kind), q, i32(start), i32(lens), i32(table), lse=lse, status=st))
    want, wlse, weight, reach = step.attention(*arrays, kind, host(q), start, lens, table, d ** -0.5, 0)
    used = [b for row, n in zip(table, lens) for b in row[:-(-n // arrays[0].shape[2])]]
    lim = (2.0 ** -9 if dt == "bf16" else 2.0 ** -15) * weight + 2.0 ** -16 * reach[..., None] * weight
    if floor:
        lim += max(lens) * 2.0 ** -25 * float(arrays[3][used].max()) * step.TOP[kind]
    if dt == "bf16":
        lim += 2.0 ** -8 * np.abs(want)
    err = np.abs(got.astype(np.float64) - want)[:t]
    assert not np.isnan(got[:t]).any() and (err <= lim[:t]).all(), (err / lim[:t]).max()
    assert (np.abs(host(lse) - wlse)[:t] <= 2.0 ** -16 * (1 + reach[:t])).all()
    assert int(st) == 0
    return want[:t]


CASES = [("e4m3", "bf16"), ("i8", "bf16"), ("e4m3", "f32"), ("i8", "f32")]


@pytest.mark.parametrize("kind,dt", CASES)
@pytest.mark.parametrize("e", [-100, -96, -93, -92, -84, -60, 60, 90])
def test_one_scale(e, kind, dt):
    rng = np.random.default_rng(200 + e)
    arrays, table, start, lens, q = attention_case(rng, [5, 1], [300, 64], 8, 2, 64, 16, kind, dt)
    arrays[3][:] = 2.0 ** e
    assert np.abs(check(arrays, kind, q, start, lens, table, dt)).max() > 2.0 ** e
    q.zero_()                                                    # equal weights
    check(arrays, kind, q, start, lens, table, dt)


@pytest.mark.parametrize("kind,dt", CASES)
@pytest.mark.parametrize("lo,hi", [(-100, -85), (-100, -20), (-100, 30)])
def test_mixed_scales(lo, hi, kind, dt):
    rng = np.random.default_rng(hi - lo)
    arrays, table, start, lens, q = attention_case(rng, [4, 4], [500, 90], 8, 2, 64, 16, kind, dt)
    arrays[3] = (2.0 ** rng.integers(lo, hi + 1, arrays[3].shape)).astype(np.float32)
    check(arrays, kind, q, start, lens, table, dt)
    arrays[0][:] = step.encode(0.1 * step.decode(arrays[0], kind), kind)      # flatter weights
    check(arrays, kind, q, start, lens, table, dt)


@pytest.mark.parametrize("kind,dt", CASES)
@pytest.mark.parametrize("n", [300, 20000])
@pytest.mark.parametrize("e", [0, 30, 70, 90])
def test_blocks_of_zeros_take_their_share_of_the_sum(e, n, kind, dt):
    # three blocks in four hold values of 0, whose scale is the smallest: their keys count in the softmax all the same.
    # 20000 keys are split over CTAs, whose parts may hold such blocks alone
    rng = np.random.default_rng(e + n)
    arrays, table, start, lens, q = attention_case(rng, [3], [n], 4, 1, 64, 16, kind, dt)
    arrays[0][:] = step.encode(0.1 * step.decode(arrays[0], kind), kind)
    arrays[3][:] = 2.0 ** e
    blocks = -(-n // 16)
    zero = table[0, :blocks * 3 // 4]
    arrays[1][zero], arrays[3][zero] = 0, 2.0 ** -100
    check(arrays, kind, q, start, lens, table, dt)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_scores_that_rise_along_small_scales(kind):
    # every key outweighs the ones before: the sum of the weights stays finite though no weight P v passes its limit
    rng = np.random.default_rng(3)
    arrays, table, start, lens, q = attention_case(rng, [1], [4000], 1, 1, 64, 16, kind, "bf16")
    one = step.encode([1.0], kind)[0]
    arrays[0][:] = 0
    arrays[0][..., 0] = one
    for j in range(4000):
        arrays[2][table[0, j // 16]] = 2.0 * (j // 16 + 1)       # scores rise by 2 from block to block, to 500
    arrays[3][:] = 2.0 ** -100
    q.zero_()
    q[:, :, 0] = 8.0
    check(arrays, kind, q, start, lens, table, "bf16")

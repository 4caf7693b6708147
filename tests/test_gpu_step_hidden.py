"""What a query of the cached step's attention does not see has no part in its
result: NaN and infinite scales of hidden blocks, and block ids of pages that
a window has left behind.  Bounds: those of the attention's other tests (bf16
queries: 2^-9 of sum p |v| for the weights' two roundings, 2^-16 of the
largest sum |q k| for the scores, 2^-8 of the result)."""

import numpy as np
import pytest

from oracle import step
from spec_verify_gb300 import binding, cache
from tests.test_gpu_step import attention_case, check_attention, host, i32, status, upload

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


@pytest.mark.parametrize("kind,dt", [("e4m3", "bf16"), ("i8", "bf16"), ("e4m3", "f32"), ("i8", "f32")])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("d,window", [(64, 100), (128, 37), (256, 5)])
def test_scales_of_blocks_before_the_window(bad, d, window, kind, dt):
    rng = np.random.default_rng(d + window)
    arrays, table, start, lens, q = attention_case(rng, [5, 1, 12], [45, 700, 333], 8, 2, d, 16, kind, dt)
    for b, n in enumerate(np.diff(start)):
        first = max(0, lens[b] - n - window + 1)                 # the first position that any query of b sees
        for blk in table[b, :first // 16]:
            arrays[2][blk] = arrays[3][blk] = bad
    check_attention(arrays, kind, q, start, lens, table, dt, window=window)


@pytest.mark.parametrize("kind,dt", [("e4m3", "bf16"), ("i8", "bf16"), ("e4m3", "f32"), ("i8", "f32")])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_scales_of_a_later_drafts_block(which, bad, kind, dt):
    # queries at 60 .. 69; the block of positions 64 .. 79 is seen by the last six alone
    rng = np.random.default_rng(7)
    arrays, table, start, lens, q = attention_case(rng, [10], [70], 8, 2, 64, 16, kind, dt)
    want, _, weight, reach = step.attention(*arrays, kind, host(q), start, lens, table, 0.125, 0)
    arrays[2 if which == "k_scale" else 3][table[0, 4]] = bad
    got = host(cache.cache_attention(upload(arrays, kind), q, i32(start), i32(lens), i32(table))).astype(np.float64)
    rounding = 2.0 ** -8 * np.abs(want[:4]) if dt == "bf16" else 0
    lim = (2.0 ** -9 if dt == "bf16" else 2.0 ** -15) * weight[:4] + 2.0 ** -16 * reach[:4, :, None] * weight[:4] + rounding
    assert (np.abs(got[:4] - want[:4]) <= lim + 1e-30).all()
    if which == "v_scale" or np.isnan(bad):
        assert not np.isfinite(got[4:10]).any()


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("window", [1, 20, 100, 129])
def test_block_ids_before_the_window_are_not_reported(window, kind):
    rng = np.random.default_rng(window)
    arrays, table, start, lens, q = attention_case(rng, [5, 1, 12], [45, 700, 333], 8, 2, 64, 16, kind, "bf16")
    freed = table.copy()
    for b, n in enumerate(np.diff(start)):
        freed[b, :max(0, lens[b] - n - window + 1) // 16] = -1   # pages given back: nobody sees their tokens
    check_attention(arrays, kind, q, start, lens, freed, "bf16", window=window, flags=0)
    b = 1
    freed[b, max(0, lens[b] - 1 - window + 1) // 16] = -1        # the first page that request 1 does see
    st = status()
    cache.cache_attention(upload(arrays, kind), q, i32(start), i32(lens), i32(freed), window=window, status=st)
    assert int(st) == binding.ROW_BAD_BLOCK

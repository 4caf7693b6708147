"""The CUDA calls of the cached speculative step against their plain fp64
forms (oracle/step.py).  Maps, codes, scales and tokens are equal; computed
numbers agree within bounds derived from the roundings that the calls state:

* norm and rotation, binary32: a sum of D squares (a chain of 8 and a
  butterfly), a reciprocal square root, two products and one rotation, at most
  16 roundings of 2^-24 on a pair's |a| + |b|: bound 2^-20.  bf16 adds half a
  unit of 2^-8.
* attention: a weight enters its product rounded to 11 bits (22 for binary32
  queries), twice (in the sum and the product they differ by that), so the
  bound is 2^-9 (2^-15 with the sums' own roundings) of sum p |v|; a score is
  a binary32 sum of D terms, so a weight is off by at most 2^-16 of the
  largest sum |q_d k_d| relative; bf16 results add 2^-8 of the result.
"""

import numpy as np
import pytest

from oracle import step
from spec_verify_gb300 import binding, cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return cuda(np.asarray(a, dtype=np.int32))


def status():
    return torch.full((1,), -7, dtype=torch.int32, device="cuda")


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


# ---------------------------------------------------------------- block plan


def plan_case(rng, batch, top, most, bs, columns=None, extra=9):
    lens, add = rng.integers(0, top + 1, batch), rng.integers(0, most + 1, batch)
    held = -(-lens // bs) + rng.integers(0, 2, batch)
    need = np.maximum(held, -(-(lens + add) // bs))
    columns = int(need.max(initial=0)) + 2 if columns is None else columns
    ids = rng.permutation(int(need.sum()) + extra + 2)
    table = np.full((batch, columns), -1)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return lens, add, held, ids[at:], table, len(ids)


def check_plan(lens, add, held, free, head, table, bs, blocks, cap):
    want = step.block_plan(lens, add, held, free, head, table, bs, blocks, cap)
    t, st = i32(table), status()
    got = cache.block_plan(i32(lens), i32(add), i32(held), i32(free), i32([head]), t, bs, blocks, cap, status=st)
    assert int(st) == want["status"]
    for key in ("lens", "held", "start", "position", "request", "slot"):
        assert np.array_equal(host(getattr(got, key)), want[key]), key
    assert int(got.free_head) == want["free_head"]
    assert np.array_equal(host(t), want["table"])
    return want["status"]


@pytest.mark.parametrize("batch,top,most,bs", [(1, 0, 1, 16), (1, 5000, 1, 16), (32, 300, 5, 16), (33, 0, 3000, 64),
                                               (257, 100, 40, 32), (1500, 50, 3, 256), (3, 40, 0, 16)])
def test_block_plan(batch, top, most, bs):
    rng = np.random.default_rng(batch + most)
    lens, add, held, free, table, blocks = plan_case(rng, batch, top, most, bs)
    for cap in (int(add.sum()), int(add.sum()) + 1077):
        assert check_plan(lens, add, held, free, 0, table, bs, blocks, cap) == 0


def test_block_plan_without_requests_or_room():
    none = np.zeros(0, dtype=np.int64)
    assert check_plan(none, none, none, np.arange(3), 1, np.zeros((0, 4), dtype=np.int64), 16, 8, 5) == 0
    rng = np.random.default_rng(1)
    lens, add, held, free, table, blocks = plan_case(rng, 300, 100, 30, 16)
    assert check_plan(lens, add, held, free, 0, table, 16, blocks, int(add.sum()) // 2) == 32      # tokens run out
    assert check_plan(lens, add, held, free[:70], 3, table, 16, blocks, int(add.sum())) == 32      # blocks run out
    assert check_plan(lens, add, held, free[:0], 0, table, 16, blocks, int(add.sum())) == 32
    assert check_plan(lens, add, held, free, 0, table, 16, blocks, 0) == 32


def test_block_plan_of_half_a_million_tokens():
    rng = np.random.default_rng(7)
    lens, add, held, free, table, blocks = plan_case(rng, 300, 90, 3300, 64)
    cap = int(add.sum())
    assert cap > 400000
    assert check_plan(lens, add, held, free, 0, table, 64, blocks, cap) == 0
    assert check_plan(lens, add, held, free, 0, table, 64, blocks, cap - 1) == 32


def test_block_plan_sums_past_32_bits():
    lens, held = np.zeros(6, dtype=np.int64), np.zeros(6, dtype=np.int64)
    table = np.full((6, 1 << 22), -1, dtype=np.int32)
    for add in ([5, 2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30, 3], [5, 0, 2 ** 30, 2 ** 30, 7, 2 ** 30]):
        assert check_plan(lens, np.array(add), held, np.arange(9), 0, table, 256, 9, 40) == 32


def test_block_plan_bad_inputs():
    rng = np.random.default_rng(2)
    lens, add, held, free, table, blocks = plan_case(rng, 40, 100, 30, 16)
    for change in ("lens", "add", "held", "wide", "huge", "head"):
        l, a, h, head = lens.copy(), add.copy(), held.copy(), 0
        if change == "lens":
            l[7] = -1
        elif change == "add":
            a[0] = -3
        elif change == "held":
            h[5] = -(-l[5] // 16) - 1
        elif change == "wide":
            h[39] = table.shape[1] + 1
        elif change == "huge":
            l[9], h[9] = 2 ** 31 - 1, 3
        else:
            head = len(free) + 1
        assert check_plan(l, a, h, free, head, table, 16, blocks, int(np.abs(a).sum())) & 16
    bad = table.copy()
    full = int(np.flatnonzero((lens % 16 > 0) & (add > 0))[0])
    bad[full, lens[full] // 16] = blocks                                   # an id past the cache
    assert check_plan(lens, add, held, free, 0, bad, 16, blocks, int(add.sum())) == 64


# ---------------------------------------------------------------- norm and rotation


def rope_inputs(rng, t, hq, hk, d, dt, fused=True):
    x = torch.from_numpy(rng.normal(0, 2, (t, hq + 2 * hk, d)).astype(np.float32)).to(DT[dt]).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk]
    return (q, k) if fused else (q.contiguous(), k.contiguous())


def check_rope(q, k, positions, table, qw, kw, eps, inter, dt, **kw_args):
    st = status()
    tab = None if table is None else cuda(table)
    got = cache.qk_norm_rope(q, k, i32(positions), tab, None if qw is None else cuda(qw), None if kw is None else cuda(kw),
                             eps, inter, status=st, **kw_args)
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        if x is None:
            continue
        want, bound = step.norm_rope(host(x), w, positions, table, eps, inter)
        live = np.asarray(positions) >= 0
        err = np.abs(host(y).astype(np.float64) - want)[live]
        lim = 2.0 ** -20 * bound[live] + (2.0 ** -8 * np.abs(want[live]) if dt == "bf16" else 0) + 1e-38
        assert not (err > lim).any(), (err / lim).max()
        assert np.array_equal(np.isnan(host(y)[live]), np.isnan(want[live]))
    return got, int(st)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,rotary", [(1, 1, 1, 64, 64), (160, 32, 8, 128, 128), (7, 9, 3, 80, 80), (5, 4, 4, 96, 32),
                                              (3, 5, 1, 256, 128), (9, 2, 2, 192, 192), (4, 3, 1, 8, 8), (11, 3, 2, 33, 20),
                                              (6, 2, 1, 20, 0), (2, 7, 7, 128, 24), (3, 2, 2, 250, 250), (2, 1, 1, 1, 0)])
def test_norm_rope(t, hq, hk, d, rotary, inter, dt):
    rng = np.random.default_rng(t * d + rotary)
    q, k = rope_inputs(rng, t, hq, hk, d, dt)
    table = host(cache.rope_table(50, rotary, 100.0)) if rotary else None
    w = rng.normal(1, 0.2, (2, d)).astype(np.float32)
    _, st = check_rope(q, k, rng.integers(0, 50, t), table, w[0], w[1], 1e-5, inter, dt)
    assert st == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 36])
def test_norm_rope_in_place_padding_and_bad_positions(d, dt):
    rng = np.random.default_rng(d)
    q, k = rope_inputs(rng, 12, 6, 2, d, dt)
    table = host(cache.rope_table(30, d))
    pos = rng.integers(0, 30, 12)
    pos[[0, 5]] = -1
    want_q, want_k = cache.qk_norm_rope(q, k, i32(np.maximum(pos, 0)), cuda(table))
    before = q.clone()
    cache.qk_norm_rope(q, k, i32(pos), cuda(table), out_q=q, out_k=k)
    assert torch.equal(q[1:5], want_q[1:5]) and torch.equal(k[6:], want_k[6:])
    assert torch.equal(q[[0, 5]], before[[0, 5]])
    pos[3] = 30
    q2, _ = rope_inputs(rng, 12, 6, 2, d, dt)
    got, st = check_rope(q2, None, pos, table, None, None, 1e-6, False, dt)
    assert st == binding.ROW_BAD_LENGTH and got[0][3].isnan().all()


def test_norm_rope_odd_strides_and_addresses():
    rng = np.random.default_rng(8)
    buf = torch.from_numpy(rng.normal(0, 1, 40 * 300).astype(np.float32)).cuda()
    q = buf[1:].as_strided((10, 2, 64), (131, 64, 1))                       # odd stride, 4-byte aligned base
    out = torch.zeros(10 * 131 + 3, device="cuda")[3:].as_strided((10, 2, 64), (131, 64, 1))
    check_rope(q, None, np.arange(10), host(cache.rope_table(10, 64)), None, None, 1e-6, False, "f32", out_q=out)


def test_norm_rope_large_values_and_zeros():
    x = torch.zeros(3, 1, 128, dtype=torch.bfloat16, device="cuda")
    x[1] = 3e18
    x[2, 0, 5] = float("nan")
    y, _ = cache.qk_norm_rope(x, None, i32([0, 1, 2]), cache.rope_table(4, 128))
    assert (y[0] == 0).all() and y[1].isfinite().all() and y[2].isnan().all()
    e, _ = cache.qk_norm_rope(x[:0], None, i32([]), cache.rope_table(4, 128))
    assert e.shape == (0, 1, 128)


# ---------------------------------------------------------------- the cache


def random_cache(rng, blocks, heads, bs, d, kind, poison=False):
    """codes k, v (bytes) and scales; poison: half of the bytes NaN codes."""
    out = []
    for _ in range(2):
        c = step.encode(rng.normal(0, 60 if kind == "e4m3" else 40, (blocks, heads, bs, d)), kind)
        if poison:
            c = np.where(rng.random(c.shape) < 0.5, 0x7F, c).astype(np.uint8)
        out.append(c)
    scale = [(2.0 ** rng.integers(-7, -3, (blocks, heads))).astype(np.float32) for _ in range(2)]
    return out + scale


def upload(arrays, kind):
    k, v, ks, vs = arrays
    return cuda(k).view(CODES[kind]), cuda(v).view(CODES[kind]), cuda(ks), cuda(vs)


def run_slots(rng, bs, blocks, runs):
    """Slots of runs of the given lengths, each starting at a random offset of
    a block of its own and going on in further blocks."""
    ids = list(rng.permutation(blocks))
    out = []
    for n in runs:
        off, block = int(rng.integers(0, bs)), ids.pop()
        for _ in range(n):
            if off == bs:
                off, block = 0, ids.pop()
            out.append(block * bs + off)
            off += 1
    return np.array(out, dtype=np.int64)


def check_append(arrays, kind, x, slots, bs, dt):
    t = [torch.from_numpy(a.astype(np.float32)).to(DT[dt]).cuda() for a in x]
    got, st = upload(arrays, kind), status()
    cache.cache_append(got, t[0], t[1], cuda(slots), status=st)
    flags = 0
    for i in range(2):
        codes, scale, f = step.append(arrays[i], arrays[2 + i], host(t[i]), slots, bs, kind)
        flags |= f
        have = got[i].view(torch.uint8).cpu().numpy()
        assert np.array_equal(host(got[2 + i]), scale, equal_nan=True)
        same = step.decode(have, kind), step.decode(codes, kind)
        assert np.array_equal(*same, equal_nan=True), int((same[0] != same[1]).sum())
    assert int(st) == flags
    return flags


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,d,bs,runs", [(1, 16, 16, [1]), (8, 128, 16, [5] * 20), (2, 80, 32, [1, 2, 100, 33, 7]),
                                             (1, 256, 256, [300, 1, 255]), (3, 64, 64, [0, 64, 65, 200]),
                                             (5, 48, 128, [3, 400])])
def test_append(heads, d, bs, runs, dt, kind):
    rng = np.random.default_rng(sum(runs) + d)
    blocks = sum(-(-n // bs) + 1 for n in runs) + 2
    arrays = random_cache(rng, blocks, heads, bs, d, kind)
    slots = run_slots(rng, bs, blocks, runs)
    x = rng.normal(0, 1, (2, len(slots), heads, d)) * 2.0 ** rng.integers(-12, 6, (2, len(slots), 1, 1))
    assert check_append(arrays, kind, x, slots, bs, dt) == 0


@pytest.mark.parametrize("kind,dt", [("e4m3", "f32"), ("i8", "bf16")])
@pytest.mark.parametrize("heads,d,bs,runs", [(12, 32, 16, [37, 1, 180, 5, 99]), (16, 16, 128, [700, 3, 129, 1000, 1, 64, 700]),
                                             (40, 48, 64, [333, 1, 64, 65, 500, 90])])
def test_append_of_long_steps(heads, d, bs, runs, dt, kind):
    # enough tokens and heads that a CTA looks at 2 to 32 tokens; padding and bad slots among them
    rng = np.random.default_rng(sum(runs) * heads)
    blocks = sum(-(-n // bs) + 1 for n in runs) + 2
    arrays = random_cache(rng, blocks, heads, bs, d, kind)
    slots = run_slots(rng, bs, blocks, runs)
    slots = np.insert(slots, [0, runs[0], len(slots)], [-1, -7, blocks * bs])
    x = rng.normal(0, 1, (2, len(slots), heads, d)) * 2.0 ** rng.integers(-12, 6, (2, len(slots), 1, 1))
    x[0, 5, heads - 1, 3], x[1, -9, 0, d - 1] = np.nan, np.inf
    assert check_append(arrays, kind, x, slots, bs, dt) == binding.ROW_BAD_LENGTH | binding.ROW_NONFINITE


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_append_exact_limits_zeros_and_nonfinite(kind):
    rng = np.random.default_rng(3)
    top = step.TOP[kind]
    arrays = random_cache(rng, 6, 2, 16, 32, kind)
    arrays[2][:], arrays[3][:] = 0.3, 0.1                          # scales that are no powers of two
    slots = np.array([3, 4, 16, 17, 40, 64, 65, 66], dtype=np.int64)
    x = rng.normal(0, 1e-3, (2, 8, 2, 32))
    x[:, 0, :, 0], x[:, 2, :, 1], x[:, 3, :, 2] = top, top * 4, np.nextafter(np.float32(top * 4), np.float32(1e9))
    x[:, 4] = 0.0
    x[:, 5:, :, 3] = 1e-42
    assert check_append(arrays, kind, x, slots, 16, "f32") == 0
    x[0, 0, 0, 1], x[0, 1, 1, 1], x[1, 5, 0, 0], x[1, 2, 0, 5] = np.nan, np.inf, -np.inf, 3e38
    assert check_append(arrays, kind, x, slots, 16, "f32") == binding.ROW_NONFINITE
    x[:, 5:] = np.inf                                               # nothing finite in a run
    assert check_append(arrays, kind, x, slots, 16, "f32") == binding.ROW_NONFINITE


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_append_padding_bad_slots_and_strides(kind):
    rng = np.random.default_rng(4)
    arrays = random_cache(rng, 4, 2, 16, 32, kind)
    slots = np.array([-1, 5, 6, -1, -1, 64, 10 ** 12, 32, 33, -5], dtype=np.int64)
    x = rng.normal(0, 3, (2, 10, 2, 32))
    assert check_append(arrays, kind, x, slots, 16, "bf16") == binding.ROW_BAD_LENGTH
    slots = np.array([48, 49, 50, 51, 14, 15, 16, 17], dtype=np.int64)
    wide = torch.from_numpy(rng.normal(0, 3, (10, 4, 32)).astype(np.float32)).cuda()
    a, b = upload(arrays, kind), upload(arrays, kind)
    odd = torch.empty(10 * 131 + 1, device="cuda")[1:].as_strided((10, 2, 32), (131, 32, 1))
    odd.copy_(wide[:, :2])
    cache.cache_append(a, wide[:8, :2], wide[:8, 2:], cuda(slots))
    cache.cache_append(b, odd[:8], wide[:8, 2:], cuda(slots))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    cache.cache_append(a, wide[:0, :2], wide[:0, 2:], cuda(slots[:0]))


def test_append_step_by_step_stays_near_one_append():
    # one token at a time with growing values: each growth encodes the older codes again
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (40, 1, 64)) * 2.0 ** (np.arange(40) // 4)[:, None, None]
    for kind, unit in (("e4m3", 2.0 ** -4), ("i8", 0.0)):
        c = cache.new_cache(3, 1, 64, 64, CODES[kind])
        t = cuda(x.astype(np.float32))
        for i in range(40):
            cache.cache_append(c, t[i:i + 1], t[i:i + 1], cuda(np.array([64 + i])))
        s = float(c[2][1, 0])
        got = step.decode(c[0].view(torch.uint8).cpu().numpy()[1, 0, :40], kind) * s
        # e4m3: half a unit in the last place, or half the subnormal step once per growth; i8: half a step, at most
        # doubled by the geometric sum of the earlier, finer roundings
        lim = np.maximum(np.abs(x[:, 0]) * unit, 2.0 ** -9 * s) if kind == "e4m3" else np.full((40, 64), s)
        assert (np.abs(got - x[:, 0]) <= lim * (1 + 1e-6)).all()


def attention_case(rng, adds, lens, hq, kv, d, bs, kind, dt, extra=3):
    adds, lens = np.asarray(adds), np.asarray(lens)
    need = -(-lens // bs)
    blocks = int(need.sum()) + extra
    ids = rng.permutation(blocks)
    table = np.full((len(adds), int(need.max(initial=0)) + 1), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    arrays = random_cache(rng, blocks, kv, bs, d, kind)
    poison = random_cache(rng, blocks, kv, bs, d, kind, poison=True) if kind == "e4m3" else arrays
    for b in range(len(adds)):                          # past the length: anything
        for j in range(lens[b], need[b] * bs):
            for i in range(2):
                arrays[i][table[b, j // bs], :, j % bs] = poison[i][table[b, j // bs], :, j % bs]
    start = np.concatenate([[0], np.cumsum(adds)])
    q = torch.from_numpy(rng.normal(0, 1.5, (int(start[-1]) + 2, hq, d)).astype(np.float32)).to(DT[dt]).cuda()
    return arrays, table, start, lens, q


def check_attention(arrays, kind, q, start, lens, table, dt, window=0, scale=None, flags=0, want_len=None, view=None):
    d = q.shape[2]
    out = torch.full_like(q, 77.0) if view is None else view
    lse, st = torch.full(q.shape[:2], 77.0, device="cuda"), status()
    cache.cache_attention(upload(arrays, kind), q, i32(start), i32(lens), i32(table), scale, window, out, lse, status=st)
    sc = d ** -0.5 if scale is None else scale
    want, wlse, weight, reach = step.attention(arrays[0], arrays[1], arrays[2], arrays[3], kind, host(q), start,
                                               lens if want_len is None else want_len, table, sc, window)
    t = int(start[-1])
    got, gl = host(out).astype(np.float64)[:t], host(lse)[:t]
    lim = (2.0 ** -9 if dt == "bf16" else 2.0 ** -15) * weight[:t] + 2.0 ** -16 * reach[:t, :, None] * weight[:t] * (
        1 if dt == "bf16" else 0.25)
    lim += 2.0 ** -8 * np.abs(want[:t]) if dt == "bf16" else 0
    err = np.abs(got - want[:t])
    assert not (err > lim + 1e-30).any() and not np.isnan(got).any(), (err / (lim + 1e-30)).max()
    none = np.isneginf(wlse[:t])
    assert np.array_equal(none, np.isneginf(gl))
    assert (np.abs(gl - wlse[:t])[~none] <= 2.0 ** -16 * (1 + reach[:t][~none])).all()
    assert (host(out)[t:] == 77.0).all() and (host(lse)[t:] == 77.0).all()      # rows past the last request
    assert int(st) == flags


ATTENTION = [
    # adds, lens, q heads, kv heads, head dim, block size
    ([1], [1], 1, 1, 16, 16),
    ([1], [1029], 32, 8, 128, 16),
    ([5] * 6, [5, 17, 64, 333, 700, 16], 32, 8, 128, 16),
    ([1, 3, 0, 8, 2], [130, 3, 50, 8, 0], 8, 1, 64, 32),
    ([17, 1, 9], [200, 1000, 9], 16, 2, 96, 64),
    ([2, 4], [513, 511], 7, 1, 256, 128),
    ([3], [259], 10, 5, 48, 256),
    ([40, 2], [77, 300], 8, 2, 64, 16),
    ([5, 5], [2100, 1999], 64, 8, 128, 32),
    ([1] * 40, list(range(1, 41)), 4, 4, 80, 16),
    ([17], [600], 16, 1, 128, 16),
    ([1], [5000], 8, 8, 192, 64),
]


@pytest.mark.parametrize("kind,dt", [("e4m3", "bf16"), ("i8", "bf16"), ("e4m3", "f32"), ("i8", "f32")])
@pytest.mark.parametrize("adds,lens,hq,kv,d,bs", ATTENTION)
def test_attention(adds, lens, hq, kv, d, bs, kind, dt):
    rng = np.random.default_rng(sum(lens) + hq)
    arrays, table, start, lens, q = attention_case(rng, adds, lens, hq, kv, d, bs, kind, dt)
    check_attention(arrays, kind, q, start, lens, table, dt)


@pytest.mark.parametrize("kind,dt", [("e4m3", "bf16"), ("i8", "f32")])
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
def test_attention_window(window, kind, dt):
    rng = np.random.default_rng(window)
    arrays, table, start, lens, q = attention_case(rng, [5, 1, 12], [40, 700, 333], 8, 2, 64, 16, kind, dt)
    check_attention(arrays, kind, q, start, lens, table, dt, window=window)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_scales_and_large_scores(dt):
    rng = np.random.default_rng(11)
    arrays, table, start, lens, q = attention_case(rng, [4, 4], [300, 64], 8, 2, 64, 16, "e4m3", dt)
    arrays[3] = (arrays[3] * 10.0 ** rng.uniform(-12, 12, arrays[3].shape)).astype(np.float32)   # any positive scale
    arrays[2] = (arrays[2] * rng.uniform(0.5, 2, arrays[2].shape)).astype(np.float32)
    check_attention(arrays, "e4m3", q, start, lens, table, dt)
    q[0] *= 3e4                                                     # beyond 16-bit floats; a single key wins
    q[1] *= 1e-9
    q[2] = 0
    check_attention(arrays, "e4m3", q, start, lens, table, dt)
    check_attention(arrays, "e4m3", q, start, lens, table, dt, scale=-0.03)
    check_attention(arrays, "e4m3", q, start, lens, table, dt, scale=0.0)


def test_attention_nan_value_of_a_later_draft_stays_out_of_earlier_rows():
    rng = np.random.default_rng(12)
    arrays, table, start, lens, q = attention_case(rng, [5], [70], 8, 2, 64, 16, "e4m3", "bf16")
    block, off = table[0, 69 // 16], 69 % 16
    good = step.attention(*arrays, "e4m3", host(q), start, lens, table, 0.125, 0)[0]
    arrays[0][block, :, off, 3] = 0x7F
    arrays[1][block, :, off, 5] = 0xFF
    out = cache.cache_attention(upload(arrays, "e4m3"), q, i32(start), i32(lens), i32(table))
    got = host(out)
    assert np.isfinite(got[:4]).all() and np.abs(got[:4] - good[:4]).max() < 0.05 * np.abs(good).max()
    assert np.isnan(got[4]).all()                                   # the row that sees the NaN key
    # and one that has left the window of the later rows, but not of the first
    arrays, table, start, lens, q = attention_case(rng, [5], [70], 8, 2, 64, 16, "e4m3", "bf16")
    arrays[1][table[0, 3], :, 65 - 9 - 48, 5] = 0x7F                # position 56: only row 0 (position 65) sees it
    out = host(cache.cache_attention(upload(arrays, "e4m3"), q, i32(start), i32(lens), i32(table), window=10))
    assert np.isnan(out[0, :, 5]).all() and np.isfinite(out[0, :, :5]).all() and np.isfinite(out[1:5]).all()


def test_attention_bad_inputs():
    rng = np.random.default_rng(13)
    arrays, table, start, lens, q = attention_case(rng, [3, 3, 3], [50, 60, 70], 8, 2, 64, 16, "e4m3", "bf16")
    bad = table.copy()
    bad[1, 1] = len(arrays[0]) + 5
    bad[2, 0] = -9
    check_attention(arrays, "e4m3", q, start, lens, bad, "bf16", flags=binding.ROW_BAD_BLOCK)
    room = table.shape[1] * 16
    check_attention(arrays, "e4m3", q, start, [50, -4, 70], table, "bf16", flags=binding.ROW_BAD_LENGTH,
                    want_len=[50, 0, 70])
    st, out = status(), torch.full_like(q, 77.0)
    cache.cache_attention(upload(arrays, "e4m3"), q, i32([0, 3, 2, 9]), i32(lens), i32(table), out=out, status=st)
    assert int(st) == binding.ROW_BAD_LENGTH and out[:3].float().abs().max() < 70
    cache.cache_attention(upload(arrays, "e4m3"), q, i32([-1, 3, 6, 900]), i32(lens), i32(table), out=out, status=st)
    assert int(st) == binding.ROW_BAD_LENGTH
    cache.cache_attention(upload(arrays, "e4m3"), q, i32(start), i32([room + 1, 60, 70]), i32(table), status=st)
    assert int(st) & binding.ROW_BAD_LENGTH
    check_attention(arrays, "e4m3", q, [0, 0, 0, 0], lens, table, "bf16")


def test_attention_strides_streams_and_repeats():
    rng = np.random.default_rng(14)
    arrays, table, start, lens, q = attention_case(rng, [5] * 8, rng.integers(5, 900, 8), 16, 4, 64, 16, "i8", "bf16")
    c = upload(arrays, "i8")
    args = (i32(start), i32(lens), i32(table))
    want = cache.cache_attention(c, q, *args)
    wide = torch.zeros(q.shape[0], 21, 64, dtype=q.dtype, device="cuda")
    wide[:, 3:19] = q
    out = torch.full((q.shape[0], 19, 64), 77.0, dtype=q.dtype, device="cuda")
    cache.cache_attention(c, wide[:, 3:19], *args, out=out[:, 1:17])
    t = int(start[-1])
    assert torch.equal(out[:t, 1:17], want[:t]) and (out[:, 0] == 77).all() and (out[:, 17:] == 77).all()
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    odd.copy_(q)
    out_odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    cache.cache_attention(c, odd, *args, out=out_odd)
    assert torch.equal(out_odd[:t], want[:t])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            again = cache.cache_attention(c, q, *args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again[:t], want[:t])                          # no order of arrival changes a result
    e = cache.cache_attention(c, q[:0], i32([0]), i32([]), i32(np.zeros((0, 4))))
    assert e.shape == (0, 16, 64)


# ---------------------------------------------------------------- verification from given numbers


def probs_case(rng, b, k, v, dt, zero=0.0):
    z = rng.normal(0, 2, (b, k + 1, v))
    p, q = np.exp(z + rng.normal(0, 1, z.shape)), np.exp(z[:, :k])
    p[rng.random(p.shape) < zero] = 0
    p, q = p / np.maximum(p.sum(-1, keepdims=True), 1e-9), q / np.maximum(q.sum(-1, keepdims=True), 1e-9)
    t = [torch.from_numpy(x.astype(np.float32)).to(DT[dt]).cuda() for x in (p, q)]
    ids = np.array([[rng.choice(v, p=q[i, j] / q[i, j].sum()) for j in range(k)] for i in range(b)],
                   dtype=np.int32).reshape(b, k)
    return t[0], t[1], ids, rng.random((b, k), dtype=np.float32), rng.exponential(size=(b, v)).astype(np.float32)


def check_probs(p, q, ids, lens, u, noise):
    st = status()
    acc, out = binding.spec_verify_probs(p, q, i32(ids), cuda(u), cuda(noise), None if lens is None else i32(lens), status=st)
    want = step.verify_probs(host(p), None if q is None else host(q), ids, lens, u, noise)
    flags = 0
    for r, w in enumerate(want):
        assert (int(acc[r]), out[r].tolist()) == (w[0], w[1]), r
        flags |= w[2]
    assert int(st) == flags
    return want


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("b,k,v", [(1, 1, 1), (3, 4, 7), (32, 4, 2003), (5, 16, 511), (2, 2, 50021), (300, 1, 64), (1, 3, 128256)])
def test_verify_probs(b, k, v, dt):
    rng = np.random.default_rng(b + v)
    p, q, ids, u, noise = probs_case(rng, b, k, v, dt)
    check_probs(p, q, ids, None, u, noise)
    check_probs(p, None, ids, None, u, noise)
    check_probs(p, q, ids, rng.integers(0, k + 1, b), u, noise)
    check_probs(p, q, ids, None, np.zeros_like(u), noise)                    # every draft kept


def test_verify_probs_edges():
    rng = np.random.default_rng(9)
    p, q, ids, u, noise = probs_case(rng, 12, 3, 301, "f32", zero=0.5)
    check_probs(p, q, ids, None, u, noise)
    p0 = p[:, :1].contiguous()                                               # k = 0: draw from the target alone
    check_probs(p0, q[:, :0], ids[:, :0], None, u[:, :0], noise)
    p[0, 0], q[0, 0] = 0, 0                                                  # nothing to draw from
    p[1, 0] = q[1, 0]
    p[1, 0, ids[1, 0]] = 0                                                   # the rest is p where p - q <= 0 everywhere
    p[2, 0, 5] = float("nan")
    p[3, :, 17] = float("inf")
    noise[4] = 1.0                                                           # ties: the lowest id
    p[4, :] = 0.25
    q[4, :] = 0.125
    u[4] = 1.0 - 2 ** -24
    ids[5, 1], ids[6, 2] = -1, 301
    want = check_probs(p, q, ids, None, u, noise)
    assert want[0][2] == binding.ROW_NONFINITE and want[5][2] == want[6][2] == binding.ROW_BAD_DRAFT
    assert want[4][1][want[4][0]] == 0
    check_probs(p, q, ids, [3, 3, 3, 3, 3, 1, 2, 4, -1, 0, 0, 3], u, noise)  # short rows hide bad ids; lengths 4, -1 are bad


@pytest.mark.parametrize("cluster", ["1", "2", "8", "16"])
def test_verify_probs_does_not_depend_on_the_split(cluster, monkeypatch):
    monkeypatch.setenv("SMP_FORCE_CLUSTER", cluster)
    rng = np.random.default_rng(10)
    p, q, ids, u, noise = probs_case(rng, 6, 3, 40007, "bf16")
    check_probs(p, q, ids, None, u, noise)


# ---------------------------------------------------------------- one step, and graphs


def test_a_step_in_a_graph():
    rng = np.random.default_rng(20)
    hq, kv, d, bs, b, cap = 8, 2, 64, 16, 4, 24
    lens, add = np.array([0, 15, 31, 100]), np.array([5, 5, 1, 5])
    held = -(-lens // bs)
    table = np.full((b, 10), -1)
    table[1, 0], table[2, :2], table[3, :7] = 0, [1, 2], range(3, 10)
    c = cache.new_cache(40, kv, bs, d)
    fill = torch.from_numpy(rng.normal(0, 1, (40, kv, bs, d)).astype(np.float32)).cuda()
    c[0].copy_((fill * 30).to(torch.float8_e4m3fn))
    c[1].copy_((fill.flip(0) * 30).to(torch.float8_e4m3fn))
    c[2].fill_(1 / 32)
    c[3].fill_(1 / 32)
    x = torch.from_numpy(rng.normal(0, 1, (cap, hq + 2 * kv, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    tab, args = cache.rope_table(256, d), [i32(lens), i32(add), i32(held), i32(range(10, 40)), i32([0]), i32(table)]
    st = [status() for _ in range(4)]
    work = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step_once():
        plan = cache.block_plan(*args, bs, 40, cap, status=st[0])
        q, k = cache.qk_norm_rope(x[:, :hq], x[:, hq:hq + kv], plan.position, tab, status=st[1])
        cache.cache_append(c, k, x[:, hq + kv:], plan.slot, status=st[2])
        return cache.cache_attention(c, q, plan.start, plan.lens, args[5], workspace=work, status=st[3]), plan, q

    before = [t.clone() for t in c]
    want, plan, q = step_once()
    after = [t.view(torch.uint8).cpu().numpy() for t in c[:2]] + [host(t) for t in c[2:]]
    ref = step.attention(*after, "e4m3", host(q), host(plan.start), host(plan.lens), host(args[5]), d ** -0.5, 0)[0]
    assert np.abs(host(want)[:16] - ref[:16]).max() < 0.01 * np.abs(ref).max() + 0.01
    for t, o in zip(c, before):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again, _, _ = step_once()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[:16], want[:16]) and all(int(s) == 0 for s in st)

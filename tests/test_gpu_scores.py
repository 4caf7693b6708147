"""The calls on rows of logits against their plain forms in 64 bits.

Tolerances.  A weight 2^y is off by its argument's rounding (y = (z - m) c has
a relative error of 3.5 steps of 2^-24, so the weight one of ln 2 |y| 3.5
2^-24: 3e-6 at |y| = 20, beyond which weights no longer matter to sums) and by
ex2.approx (1.7e-7).  A sum of them adds at most 100 roundings one after another
(a unit of 32 elements, a thread's units, then trees): 6e-6.  So Z, and with it ln Z, p and
mean values, are within 2^-16 relative; values are then off by a few steps of
2^-24 of the numbers they are made from: 2^-21 of those.  A weight of its own
(a gradient's p_j) has |y| up to 126 before it is flushed: ln 2 * 126 * 3.5 *
2^-24 = 1.8e-5, together below 2^-15.  A gradient
whose argument is one fused multiply-add, z c plus a constant below 128 + 150,
has that constant's rounding instead, 278 * 2^-24 ln 2 = 1.1e-5, and c's own of
2^-24 ln 2 * 256 = 1.1e-5: the same 2^-15.  bf16 results: half a step, 2^-8."""

import numpy as np
import pytest

from oracle import scores as oracle
from spec_verify_gb300 import binding, scores

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")]

torch = pytest.importorskip("torch")

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 2.0 ** -120                    # weights below 2^-126 are flushed (times w / T), and the type's own smallest numbers


def single(a):
    """As binary32, which overflows to infinity."""
    with np.errstate(over="ignore"):
        return np.asarray(a).astype(np.float32).astype(np.float64)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def up(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def status():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


def rows_of(rng, rows, vocab, dtype, masked=0.0, spread=3.0, stride=None, offset=0):
    """Logits on the GPU, rows `stride` apart (NaN between them) from an element
    `offset`, and what they hold."""
    stride = stride or vocab
    store = torch.full((rows * stride + offset + 16,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    view = store[offset:offset + rows * stride].view(rows, stride)[:, :vocab]
    z = rng.normal(0, spread, (rows, vocab))
    z[rng.random((rows, vocab)) < masked] = -np.inf
    view.copy_(up(z))
    return view, host(view), store


def check_logprobs(view, z, ids, top, temperature, entropy=True, flags=0, **kw):
    rows = len(z)
    st = status()
    t = temperature if isinstance(temperature, float) else up(temperature)
    got = scores.token_logprobs(view, None if ids is None else up(ids, torch.int32), top=top, entropy=entropy,
                                temperature=t, status=st, **kw)
    torch.cuda.synchronize()
    want, flag = oracle.token_logprobs(z, ids, top, np.float32(temperature))
    assert int(st) == flag == flags
    for r in range(rows):
        given, ent, best, value = want[r]
        given, value = single(given), single(value)
        if ids is not None:
            g = host(got.logprobs[r])
            same = (np.isnan(g) & np.isnan(given)) | (g == given)
            assert (same | (np.abs(g - given) <= 2.0 ** -16 + 2.0 ** -21 * np.abs(given))).all(), (r, g, given)
        if entropy:
            e = float(got.entropy[r])
            assert (np.isnan(e) and np.isnan(ent)) or abs(e - ent) <= 2.0 ** -15 * (1 + ent), (r, e, ent)
        if top:
            assert np.array_equal(got.top_ids[r].cpu().numpy(), best), (r, got.top_ids[r], best)
            g = host(got.top_logprobs[r])
            same = (np.isnan(g) & np.isnan(value)) | (g == value)
            assert (same | (np.abs(g - value) <= 2.0 ** -16 + 2.0 ** -21 * np.abs(value))).all(), (r, g, value)
    return got


def check_grad(got, want, reach, dtype, temperature=1.0):
    tiny = TINY * max(1.0, 1.0 / float(np.min(temperature)))
    g = host(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), np.argwhere(np.isnan(g) != np.isnan(want))[:5]
    fine = ~np.isnan(want)
    err = np.abs(g - want)[fine]
    assert (err <= (2.0 ** -15 * reach + STEP[dtype] * np.abs(want) * (1 + 2.0 ** -7))[fine] + tiny).all(), (
        np.abs(err).max(), np.argmax(err - (2.0 ** -15 * reach + STEP[dtype] * np.abs(want))[fine]))


SHAPES = [(1, 1), (3, 2), (5, 7), (4, 17), (7, 100), (2, 1000), (3, 2049), (33, 8191), (700, 517), (3, 32000), (2, 50021),
          (1, 128256), (2, 152064), (1, 524288)]


def ids_for(rng, rows, vocab, count):
    ids = rng.integers(0, vocab, (rows, count))
    ids[rng.random((rows, count)) < 0.2] = -1
    return ids


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_token_logprobs(rows, vocab, dtype):
    rng = np.random.default_rng(rows * vocab)
    view, z, _ = rows_of(rng, rows, vocab, dtype, masked=0.1 if vocab > 50 else 0.0)
    check_logprobs(view, z, ids_for(rng, rows, vocab, 1), 0, 1.0, entropy=False)
    check_logprobs(view, z, None, 5, 0.7)
    check_logprobs(view, z, ids_for(rng, rows, vocab, 128), 128, rng.uniform(0.3, 3.0, rows).astype(np.float32))
    check_logprobs(view, z, ids_for(rng, rows, vocab, 3), 20, 1.0, entropy=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,stride,offset", [(5, 1001, 1001, 1), (4, 1000, 1003, 3), (6, 50021, 50048, 0),
                                                      (3, 33, 37, 5), (9, 7, 8, 1)])
def test_rows_at_odd_addresses(rows, vocab, stride, offset, dtype):
    rng = np.random.default_rng(stride)
    view, z, store = rows_of(rng, rows, vocab, dtype, stride=stride, offset=offset)
    ids = ids_for(rng, rows, vocab, 2)
    check_logprobs(view, z, ids, 7, 1.0)
    g, h = rng.normal(0, 1, (rows, 2)).astype(np.float32), rng.normal(0, 1, rows).astype(np.float32)
    want, reach, _ = oracle.token_logprobs_grad(z, ids, g, h)
    teach = rng.integers(0, vocab, (rows, 3))
    values = np.log(rng.dirichlet(np.ones(4), rows)[:, :3]).astype(np.float32)
    loss, dwant, lreach, dreach, _ = oracle.distill(z, teach, values, 1)
    other, _, whole = rows_of(rng, rows, vocab, dtype, stride=stride + 2, offset=offset + 1)
    for out, around in ((None, None), (other, whole), (view, store)):      # a new one, one of another alignment, in place
        for kind in ("scores", "distill"):
            view.copy_(up(z))
            if out is not None and out is not view:
                out.fill_(3.0)
            if kind == "scores":
                got = scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), up(h), out=out)
                check_grad(got, want, reach, dtype)
            else:
                _, got = scores.distill_grad(view, up(teach, torch.int32), up(values), tail=True, out=out)
                check_grad(got, dwant, dreach, dtype)
            if around is not None:                                         # what lies between the rows is left alone
                assert int(torch.isnan(around).sum()) == around.numel() - rows * vocab


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits_and_short_masks(dtype):
    rng = np.random.default_rng(3)
    for vocab in (40, 3000, 40000):                      # every token equal: more candidates than a list holds
        z = np.zeros((3, vocab))
        z[1, :] = -np.inf
        z[1, rng.permutation(vocab)[:9]] = 2.0           # nine tokens allowed
        z[2, :] = rng.integers(0, 2, vocab)              # two values
        check_logprobs(up(z, DTYPES[dtype]), z, [[0], [vocab - 1], [5]], 20, 1.0)
    z = np.full((2, 70000), -np.inf)
    z[0, 69999] = -3.0                                   # one token allowed: the last, the first
    z[1, 0] = 5.0
    check_logprobs(up(z, DTYPES[dtype]), z, [[69999, 0], [0, 1]], 3, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [9, 5000, 90000])
def test_hard_rows(vocab, dtype):
    lowest = torch.finfo(DTYPES[dtype]).min
    rng = np.random.default_rng(vocab)
    z = rng.normal(0, 2, (12, vocab))
    z[0] = -np.inf                                       # nothing left
    z[1] = np.nan
    z[2, 3] = np.inf
    z[3, rng.random(vocab) < 0.5] = np.nan               # NaN is -inf
    z[4, 1:] = lowest                                    # masked with the type's lowest value
    z[5] = lowest
    z[6] = lowest
    z[6, 1::2] = -np.inf
    z[7] = 1e30 * rng.choice([-1, 1], vocab)
    z[8] = -z[8] * 1e-40
    z[9] += 3e4                                          # far from zero
    z[10, 1:] = -np.inf
    z[11, : vocab // 2] = lowest
    z[11, vocab // 2] = np.nan
    z = host(up(z, DTYPES[dtype]))
    view = up(z, DTYPES[dtype])
    ids = rng.integers(0, vocab, (12, 4))
    ids[:, 3] = -1
    g, h = rng.normal(0, 1, (12, 4)).astype(np.float32), rng.normal(0, 1, 12).astype(np.float32)
    for t in (1.0, 2.0 ** -30, 1e-3, 50.0, 2.0 ** 30):
        check_logprobs(view, z, ids, 6, t, flags=oracle.NONFINITE)
        want, reach, flags = oracle.token_logprobs_grad(z, ids, g, h, np.float32(t))
        st = status()
        got = scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), up(h), temperature=t, status=st)
        assert int(st) == flags == oracle.NONFINITE
        check_grad(got, want, reach, dtype, t)
        check_distill(view, z, ids, np.log(rng.dirichlet(np.ones(5), 12)[:, :4]).astype(np.float32), dtype, temperature=t,
                      flags=oracle.NONFINITE)


def test_bad_rows_are_marked_and_the_others_right():
    rng = np.random.default_rng(9)
    view, z, _ = rows_of(rng, 6, 3000, "bf16")
    ids = ids_for(rng, 6, 3000, 3)
    ids[1, 2] = 3000
    ids[2] = -1
    t = np.array([1.0, 1.0, 0.0, np.nan, 2.0 ** -31, 2.0], dtype=np.float32)
    check_logprobs(view, z, ids, 4, t, flags=oracle.BAD_PARAMS | oracle.BAD_TOKEN)
    st = status()
    got = scores.token_logprobs(view, up(ids, torch.int32), temperature=up(t), status=st)      # row 2 asks for nothing
    assert int(st) == oracle.BAD_PARAMS | oracle.BAD_TOKEN and not got.logprobs[2].any()
    g = rng.normal(0, 1, (6, 3)).astype(np.float32)
    want, reach, flags = oracle.token_logprobs_grad(z, ids, g, None, t)
    grad = scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), temperature=up(t), status=st)
    assert int(st) == flags == oracle.BAD_PARAMS | oracle.BAD_TOKEN
    check_grad(grad, want, reach, "bf16")
    values = np.full((6, 3), np.log(0.2), dtype=np.float32)
    values[0, 1] = np.nan
    values[5] = -0.1
    t[3] = 1.0
    ids[0, :2], ids[5] = [4, 5], [1, 2, 3]
    check_distill(view, z, ids, values, "bf16", temperature=t, tails=(1,), flags=oracle.BAD_PARAMS | oracle.BAD_TOKEN)
    values[0], values[3] = -np.inf, -np.inf
    ids[3] = [7, 8, -1]
    check_distill(view, z, ids, values, "bf16", temperature=t, tails=(0,), flags=oracle.BAD_PARAMS | oracle.BAD_TOKEN)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_token_logprobs_grad(rows, vocab, dtype):
    rng = np.random.default_rng(rows + vocab)
    view, z, _ = rows_of(rng, rows, vocab, dtype, masked=0.1 if vocab > 50 else 0.0)
    for count, with_entropy, t in ((1, False, 1.0), (128, True, 0.8), (0, True, 1.0), (2, True, None)):
        ids = ids_for(rng, rows, vocab, count)
        if rows > 2:
            ids[1] = -1                                   # padding
        g, h = rng.normal(0, 1, (rows, count)).astype(np.float32), rng.normal(0, 1, rows).astype(np.float32)
        h[1:2] = 0.0
        t = rng.uniform(0.3, 3.0, rows).astype(np.float32) if t is None else t
        want, reach, flags = oracle.token_logprobs_grad(z, ids, g, h if with_entropy else None, np.float32(t))
        st = status()
        got = scores.token_logprobs_grad(view, up(ids, torch.int32) if count else None, up(g) if count else None,
                                         up(h) if with_entropy else None, temperature=t if isinstance(t, float) else up(t),
                                         status=st)
        assert int(st) == flags == 0
        check_grad(got, want, reach, dtype)


def check_distill(view, z, ids, values, dtype, temperature=1.0, weight=None, tails=(0, 1), flags=0):
    t = temperature if isinstance(temperature, float) else up(temperature)
    for tail in tails:
        loss, grad, lreach, reach, flag = oracle.distill(z, ids, values, tail, weight, np.float32(temperature))
        st = status()
        got, dz = scores.distill_grad(view, up(ids, torch.int32), up(values), None if weight is None else up(weight),
                                      tail=bool(tail), temperature=t, status=st)
        assert int(st) == flag == flags
        st = status()
        alone = scores.distill_loss(view, up(ids, torch.int32), up(values), tail=bool(tail), temperature=t, status=st)
        assert int(st) == flag
        loss = single(loss)
        for g in (host(got), host(alone)):
            same = (np.isnan(g) & np.isnan(loss)) | (g == loss)
            # a loss of binary32's largest number, off by what is allowed, may round to infinity: infinity is at least 2^128 - 2^103
            g = np.where((g == np.inf) & np.isfinite(loss), 2.0 ** 128, g)
            with np.errstate(invalid="ignore"):
                near = np.abs(g - loss) <= 2.0 ** -16 * (1 + lreach * 2.0 ** -5)
            assert (same | near).all(), (tail, g - loss, lreach)
        check_grad(dz, grad, reach, dtype, temperature if flags != 1 | 128 else 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_distill(rows, vocab, dtype):
    rng = np.random.default_rng(7 * rows + vocab)
    view, z, _ = rows_of(rng, rows, vocab, dtype)
    for count in (1, 20, 128):
        k = min(count, vocab)
        teacher = z + rng.normal(0, 1, z.shape)
        ids = np.full((rows, count), -1)
        ids[:, :k] = np.argsort(-teacher, 1)[:, :k]
        logt = teacher - np.log(np.exp(teacher).sum(1, keepdims=True))
        values = np.where(ids >= 0, np.take_along_axis(logt, np.maximum(ids, 0), 1), np.nan).astype(np.float32)
        if rows > 3:
            ids[2] = -1
            perm = rng.permutation(count)
            ids[3], values[3] = ids[3][perm], values[3][perm]
        check_distill(view, z, ids, values, dtype, weight=rng.normal(0, 1, rows).astype(np.float32))
    check_distill(view, z, ids, values, dtype, temperature=rng.uniform(0.5, 2.0, rows).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [6, 4000, 100000])
def test_distill_at_the_edges(vocab, dtype):
    rng = np.random.default_rng(vocab)
    z = rng.normal(0, 2, (8, vocab))
    ids = np.stack([rng.permutation(vocab)[:5] for _ in range(8)])
    values = np.log(rng.dirichlet(np.ones(6), 8)[:, :5]).astype(np.float32)
    ids[0, 3] = ids[0, 1]                                # the same id twice
    ids[1] = ids[1, 0]                                   # five times
    z[2, ids[2, 1]] = -np.inf                            # the student rules out what the teacher says: loss +inf
    values[3, 2] = -np.inf                               # a teacher's token of probability 0 ...
    z[3, ids[3, 2]] = -np.inf                            # ... that the student rules out
    z[4] = -np.inf                                       # the student has the ids alone
    z[4, ids[4]] = rng.normal(0, 1, 5)
    z[5, ids[5]] += 300.0                                # hardly anything outside the ids
    z[6, ids[6]] -= 300.0                                # hardly anything on them
    values[7] = np.log(0.2)                              # the teacher has nothing outside
    z = host(up(z, DTYPES[dtype]))
    check_distill(up(z, DTYPES[dtype]), z, ids, values, dtype)


def test_gradients_against_differences_of_the_losses():
    """(loss(z + e d) - loss(z - e d)) / 2e along random directions: the losses are
    within 2^-16 each (above), so the quotient within 2^-16 / e, and the third
    derivative adds e^2 / 6 of a few."""
    rng = np.random.default_rng(21)
    view, z, _ = rows_of(rng, 4, 3001, "f32", spread=1.0)
    ids = up(rng.integers(0, 3001, (4, 6)), torch.int32)
    values = up(np.log(rng.dirichlet(np.ones(7) * 5, 4)[:, :6]))
    hot = ids[:, :1].contiguous()
    e = 2.0 ** -4
    for d in (torch.zeros_like(view).scatter_(1, hot.long(), 1.0), up(rng.choice([-1.0, 1.0], z.shape))):
        for tail in (False, True):
            _, grad = scores.distill_grad(view, ids, values, tail=tail)
            hi, lo = (scores.distill_loss(view + s * e * d, ids, values, tail=tail) for s in (1, -1))
            assert ((hi - lo) / (2 * e) - (grad * d).sum(1)).abs().max() < 2.0 ** -16 / e + e * e
        grad = scores.token_logprobs_grad(view, hot, torch.ones(4, 1, device="cuda"), torch.full((4,), 0.5, device="cuda"))
        hi, lo = (scores.token_logprobs(view + s * e * d, hot, entropy=True) for s in (1, -1))
        want = ((hi.logprobs[:, 0] + 0.5 * hi.entropy) - (lo.logprobs[:, 0] + 0.5 * lo.entropy)) / (2 * e)
        assert (want - (grad * d).sum(1)).abs().max() < 2.0 ** -12 / e + e * e      # an entropy of 8: 2^-15 * 9


@pytest.mark.parametrize("cluster", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_cluster_size(cluster, dtype, monkeypatch):
    monkeypatch.setenv("SMP_FORCE_CLUSTER", str(cluster))
    for rows, vocab in ((3, 5), (4, 1237), (5, 40003)):
        rng = np.random.default_rng(cluster + vocab)
        view, z, _ = rows_of(rng, rows, vocab, dtype)
        ids = ids_for(rng, rows, vocab, 3)
        check_logprobs(view, z, ids, 20, 1.0)
        g, h = rng.normal(0, 1, (rows, 3)).astype(np.float32), rng.normal(0, 1, rows).astype(np.float32)
        want, reach, _ = oracle.token_logprobs_grad(z, ids, g, h)
        check_grad(scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), up(h)), want, reach, dtype)
        values = np.log(rng.dirichlet(np.ones(4), rows)[:, :3]).astype(np.float32)
        check_distill(view, z, ids, values, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,count,top", [(3700, 2300, 1, 1), (3700, 301, 32, 16), (1900, 1203, 33, 5), (1900, 4100, 5, 32),
                                                  (950, 8193, 20, 0), (950, 70, 65, 40), (950, 700, 128, 64), (60, 77003, 2, 1)])
def test_many_rows_by_small_thread_blocks(rows, vocab, count, top, dtype):
    rng = np.random.default_rng(rows + vocab)
    view, z, _ = rows_of(rng, rows, vocab, dtype, masked=0.05, stride=vocab + 3, offset=1)
    view[7], view[11, 5], view[13, ::2], z[7], z[11, 5], z[13, ::2] = -np.inf, np.inf, np.nan, -np.inf, np.inf, np.nan
    view[17, 1:], z[17, 1:] = -np.inf, -np.inf
    ids = ids_for(rng, rows, vocab, count)
    ids[3:5] = -1                                         # padding
    t = rng.uniform(0.3, 3.0, rows).astype(np.float32)
    check_logprobs(view, z, ids, top, t, flags=2)
    check_logprobs(view, z, ids, top, 1.0, entropy=False, flags=2)
    g, h = rng.normal(0, 1, (rows, count)).astype(np.float32), rng.normal(0, 1, rows).astype(np.float32)
    h[::3] = 0.0
    want, reach, flag = oracle.token_logprobs_grad(z, ids, g, h, t)
    st = status()
    got = scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), up(h), temperature=up(t), status=st)
    check_grad(got, want, reach, dtype, t)
    assert int(st) == flag == 2
    values = np.log(rng.dirichlet(np.ones(count + 1), rows)[:, :count]).astype(np.float32)
    check_distill(view, z, ids, values, dtype, temperature=t, weight=h, flags=2)


@pytest.mark.parametrize("rows,vocab,dtype", [(240, 33001, "f32"), (130, 100003, "bf16"), (130, 50021, "f32")])
@pytest.mark.parametrize("count", [20, 64, 65])
def test_distillation_of_long_slices(rows, vocab, dtype, count):
    rng = np.random.default_rng(vocab + count)
    view, z, _ = rows_of(rng, rows, vocab, dtype, masked=0.05, stride=vocab + 5)
    ids = ids_for(rng, rows, vocab, count)
    ids[2], ids[3, 1] = -1, ids[3, 0]
    values = np.log(rng.dirichlet(np.ones(count + 1), rows)[:, :count]).astype(np.float32)
    check_distill(view, z, ids, values, dtype, weight=rng.normal(0, 1, rows).astype(np.float32), tails=(1,))


def all_calls(view, ids, g, h, values, stream=None):
    got = scores.token_logprobs(view, ids, top=5, entropy=True, stream=stream)
    grad = scores.token_logprobs_grad(view, ids, g, h, stream=stream)
    alone = scores.distill_loss(view, got.top_ids, got.top_logprobs, tail=True, stream=stream)
    loss, dz = scores.distill_grad(view, ids, values, tail=True, stream=stream)
    return [*got, grad, alone, loss, dz]


def some_inputs(rows=37, vocab=30001, dtype="bf16", seed=0):
    rng = np.random.default_rng(seed)
    view, _, _ = rows_of(rng, rows, vocab, dtype)
    return (view, up(ids_for(rng, rows, vocab, 3), torch.int32), up(rng.normal(0, 1, (rows, 3))), up(rng.normal(0, 1, rows)),
            up(np.log(rng.dirichlet(np.ones(4), rows)[:, :3])))


def test_the_same_from_run_to_run():
    for rows in (1, 37, 900):
        inputs = some_inputs(rows)
        want = [t.clone() for t in all_calls(*inputs)]
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(all_calls(*inputs), want))


def test_captured_and_replayed_with_new_inputs():
    inputs, other = some_inputs(), some_inputs(seed=1)
    want = [[t.clone() for t in all_calls(*x)] for x in (inputs, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):                        # two graphs over the same inputs
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = all_calls(*inputs)
            graphs.append((graph, out))
    torch.cuda.synchronize()
    for x, expect in ((inputs, want[0]), (other, want[1])):
        for a, b in zip(inputs, x):
            a.copy_(b.clone())
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, expect))


def test_calls_on_a_stream_of_their_own():
    inputs = some_inputs(64)
    want = [t.clone() for t in all_calls(*inputs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = all_calls(*inputs, stream=side)
        for mb in (1, 2, 4, 8, 16, 32, 64):              # what the calls made themselves is not handed out here
            torch.full((mb << 18,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    stride = (1 << 31) + 24                              # the third row starts past 2^32 elements
    store = torch.zeros(2 * stride + 4000, dtype=torch.bfloat16, device="cuda")
    view = store.as_strided((3, 4000), (stride, 1))
    rng = np.random.default_rng(5)
    z = host(up(rng.normal(0, 2, (3, 4000)), torch.bfloat16))
    view.copy_(up(z))
    ids = ids_for(rng, 3, 4000, 2)
    check_logprobs(view, z, ids, 5, 1.0)
    g = rng.normal(0, 1, (3, 2)).astype(np.float32)
    want, reach, _ = oracle.token_logprobs_grad(z, ids, g, None)
    check_grad(scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), out=view), want, reach, "bf16")


def test_more_rows_than_65535():
    g = torch.Generator("cuda").manual_seed(4)
    rows, vocab = 200003, 5
    view = torch.randn(rows, vocab, generator=g, device="cuda") * 3
    ids = torch.randint(-1, vocab, (rows, 2), generator=g, device="cuda").int()
    got = scores.token_logprobs(view, ids, top=3, entropy=True)
    logp = view.double().log_softmax(1)
    live = ids >= 0
    want = logp.gather(1, ids.clamp(min=0).long()) * live
    assert bool(((got.logprobs - want).abs() <= 2.0 ** -16 + 2.0 ** -21 * want.abs()).all())
    entropy = -(logp.exp() * logp).sum(1)
    assert bool(((got.entropy - entropy).abs() <= 2.0 ** -15 * (1 + entropy)).all())
    best, at = logp.sort(dim=1, descending=True, stable=True)
    assert torch.equal(got.top_ids.long(), at[:, :3])
    assert bool(((got.top_logprobs - best[:, :3]).abs() <= 2.0 ** -16 + 2.0 ** -21 * best[:, :3].abs()).all())
    up_g = torch.randn(rows, 2, generator=g, device="cuda")
    hot = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
    hot.scatter_add_(1, ids.clamp(min=0).long(), up_g.double() * live)
    total, reach = (up_g.double() * live).sum(1, keepdim=True), (up_g.double().abs() * live).sum(1, keepdim=True)
    grad = hot - logp.exp() * total
    bound = 2.0 ** -15 * (logp.exp() * reach + (hot.abs() + reach * (hot != 0))) + 2.0 ** -120
    assert bool(((scores.token_logprobs_grad(view, ids, up_g) - grad).abs() <= bound).all())
    loss, dz = scores.distill_grad(view, ids[:, :1].contiguous(), torch.zeros(rows, 1, device="cuda"))
    sure = ids[:, 0] >= 0                                 # a teacher that is sure: the loss is -ln p, its gradient p - 1
    assert bool(((loss + want[:, 0]).abs() <= 2.0 ** -16 * (1 + want[:, 0].abs())).all())
    one = torch.nn.functional.one_hot(ids[:, 0].clamp(min=0).long(), vocab)
    assert bool(((dz - (logp.exp() - one) * sure[:, None]).abs() <= 2.0 ** -15 * (logp.exp() + one)).all())


def test_no_rows_and_no_status():
    empty = torch.empty(0, 500, device="cuda")
    ids = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    st = status()
    got = scores.token_logprobs(empty, ids, top=4, entropy=True, status=st)
    assert int(st) == 0 and got.logprobs.shape == (0, 3) and got.top_ids.shape == (0, 4)
    loss, grad = scores.distill_grad(empty, ids, torch.empty(0, 3, device="cuda"))
    assert loss.shape == (0,) and grad.shape == (0, 500)


@pytest.mark.parametrize("call", ["logprobs", "grad", "distill"])
def test_a_wait_that_runs_out_marks_rows_and_the_next_call_is_right(call, monkeypatch):
    """With a limit of 0 the copy's barrier is looked at once: rows whose copy has
    not landed by then are marked, and the others right."""
    view, ids, g, h, values = some_inputs(300, 20001)
    run = {"logprobs": lambda st: [scores.token_logprobs(view, ids, entropy=True, status=st).entropy[:, None]],
           "grad": lambda st: [scores.token_logprobs_grad(view, ids, g, h, status=st)],
           "distill": lambda st: [t.reshape(300, -1) for t in scores.distill_grad(view, ids.clamp(min=0), values, status=st)]}[call]
    st = status()
    want = [t.clone() for t in run(st)]
    assert int(st) == 0
    monkeypatch.setenv("SMP_WAIT_LIMIT_NS", "0")
    got = run(st)
    late = torch.isnan(got[0]).any(1)
    assert int(st) == (binding.ROW_TIMEOUT if bool(late.any()) else 0)
    assert all(torch.equal(a[~late], b[~late]) for a, b in zip(got, want)) and all(bool(torch.isnan(a[late]).all()) for a in got)
    monkeypatch.delenv("SMP_WAIT_LIMIT_NS")
    assert all(torch.equal(a, b) for a, b in zip(run(st), want)) and int(st) == 0


def test_a_teachers_record_trains_a_student():
    """The calls together: the target's record, the student's loss and gradient on
    it, and steps along the gradient towards the target."""
    rng = np.random.default_rng(2)
    target, t, _ = rows_of(rng, 40, 6001, "bf16")
    record = scores.token_logprobs(target, top=32, temperature=2.0)
    student = up(rng.normal(0, 1, (40, 6001)))
    ids, values = record.top_ids.cpu().numpy(), host(record.top_logprobs).astype(np.float32)
    check_distill(student, host(student), ids, values, "f32", temperature=2.0, tails=(1,))
    for _ in range(50):
        _, grad = scores.distill_grad(student, record.top_ids, record.top_logprobs, tail=True, temperature=2.0)
        student -= 4.0 * grad
    check_distill(student, host(student), ids, values, "f32", temperature=2.0, tails=(1,))
    check_logprobs(student, host(student), ids, 32, 2.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_beside_the_logits_in_wider_rows(dtype):
    rng = np.random.default_rng(9)
    store = torch.full((30, 2011), 7.0, dtype=DTYPES[dtype], device="cuda")
    view, out = store[:, 5:1005], store[:, 1005:2005]
    view.copy_(up(rng.normal(0, 3, (30, 1000))))
    z, ids, g = host(view), ids_for(rng, 30, 1000, 3), rng.normal(0, 1, (30, 3)).astype(np.float32)
    want, reach, _ = oracle.token_logprobs_grad(z, ids, g, None)
    check_grad(scores.token_logprobs_grad(view, up(ids, torch.int32), up(g), out=out), want, reach, dtype)
    assert np.array_equal(host(view), z) and bool((store[:, :5] == 7).all()) and bool((store[:, 2005:] == 7).all())
    for other in (store[:, 6:1006], store[:, 1004:2004], store[:, :1000], store[1:, 5:1005]):
        with pytest.raises(binding.SmpError):
            scores.token_logprobs_grad(view[:len(other)], up(ids[:len(other)], torch.int32), up(g[:len(other)]), out=other)

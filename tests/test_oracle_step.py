"""The plain forms of the cached speculative step (oracle/step.py) against
torch's 8-bit floats, direct formulas and the distribution they promise."""

import numpy as np
import pytest

from oracle import step

torch = pytest.importorskip("torch")


def test_e4m3_codes_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(step.decode(codes, "e4m3"), want, equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(0, 1, 4000), rng.normal(0, 200, 4000), rng.normal(0, 0.01, 4000),
                        (step.E4M3[:126] + step.E4M3[1:127]) / 2]).astype(np.float32)
    x = np.clip(x, -448, 448)
    got = step.encode(x, "e4m3")
    assert np.array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_encode_edges():
    assert list(step.encode([np.inf, -np.inf, np.nan, 1e9, -0.0], "e4m3")) == [0x7E, 0xFE, 0x7F, 0x7E, 0x80]
    assert list(step.encode([np.inf, -np.inf, np.nan, 0.5, 1.5, -2.5], "i8").view(np.int8)) == [127, -127, 0, 0, 2, -2]


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_needed_scale_is_the_smallest_power_of_two(kind):
    top = step.TOP[kind]
    for e in (-60, -3, 0, 1, 40):
        assert step.needed_scale(top * 2.0 ** e, kind) == 2.0 ** e
        assert step.needed_scale(np.nextafter(top * 2.0 ** e, np.inf), kind) == 2.0 ** (e + 1)
    assert step.needed_scale(0.0, kind) == step.needed_scale(1e-40, kind) == 2.0 ** -100


def test_block_plan_partitions_the_free_list():
    rng = np.random.default_rng(2)
    lens, add = rng.integers(0, 100, 20), rng.integers(0, 50, 20)
    held = -(-lens // 16)
    ids = rng.permutation(400)
    table = np.full((20, 12), -1)
    at = 0
    for b in range(20):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    res = step.block_plan(lens, add, held, ids[at:], 0, table, 16, 400, 2000)
    assert res["status"] == 0 and list(res["lens"]) == list(lens + add)
    slots = res["slot"][:add.sum()]
    assert len(set(slots)) == add.sum() and (res["slot"][add.sum():] == -1).all()
    used = res["table"][res["table"] >= 0]
    assert len(set(used)) == len(used) == (-(-(lens + add) // 16)).sum()


def test_norm_rope_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (1, 1, 32))
    pos = np.arange(40)[:, None] * 100.0 ** (-np.arange(16) / 16)
    table = np.concatenate([np.cos(pos), np.sin(pos)], 1)
    for inter in (False, True):
        a, _ = step.norm_rope(np.repeat(x, 4, 0), None, [3, 10, 13, 20], table, 0.0, inter)
        assert np.allclose((a ** 2).sum(-1), 32)
        assert np.isclose((a[0] * a[1]).sum(), (a[2] * a[3]).sum())     # depends on the distance alone


def test_attention_matches_a_direct_softmax():
    rng = np.random.default_rng(4)
    k, v = (rng.integers(0, 0x7F, (4, 2, 16, 16)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.uniform(0.001, 0.01, (4, 2)).astype(np.float32) for _ in range(2))
    q = rng.normal(0, 1, (3, 4, 16))
    table = np.array([[2, 0, -1], [3, 1, -1]])
    out, lse, weight, _ = step.attention(k, v, ks, vs, "e4m3", q, [0, 2, 3], [20, 0], table, 0.25, 0)
    kk = np.concatenate([step.decode(k[2, 1], "e4m3") * ks[2, 1], step.decode(k[0, 1], "e4m3") * ks[0, 1]])[:19]
    vv = np.concatenate([step.decode(v[2, 1], "e4m3") * vs[2, 1], step.decode(v[0, 1], "e4m3") * vs[0, 1]])[:19]
    z = np.exp(0.25 * kk @ q[0, 2])
    assert np.allclose(out[0, 2], z @ vv / z.sum()) and np.isclose(lse[0, 2], np.log(z.sum()))
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all()             # length 0: nothing to see


def test_verify_probs_keeps_the_target_distribution():
    rng = np.random.default_rng(5)
    n, vocab = 20000, 5
    p0, q0 = rng.dirichlet(np.ones(vocab)), rng.dirichlet(np.ones(vocab))
    p = np.broadcast_to(p0.astype(np.float32), (n, 2, vocab))
    q = np.broadcast_to(q0.astype(np.float32), (n, 1, vocab))
    ids = rng.choice(vocab, size=(n, 1), p=q0)
    res = step.verify_probs(p, q, ids, None, rng.random((n, 1), dtype=np.float32),
                            rng.exponential(size=(n, vocab)).astype(np.float32))
    first = np.bincount([r[1][0] for r in res], minlength=vocab)
    assert ((first - n * p0) ** 2 / (n * p0)).sum() < 23.5                # chi-square, 4 degrees, p = 1e-4
    kept = np.mean([r[0] for r in res])
    assert abs(kept - np.minimum(p0, q0).sum()) < 5 * 0.5 / np.sqrt(n)

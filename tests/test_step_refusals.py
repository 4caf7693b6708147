"""Host-side validation of the cached step's entry points: bad arguments are
answered before anything touches a GPU."""

import ctypes

import pytest

from spec_verify_gb300 import binding, build, cache

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)
HALF = ctypes.c_void_p(0x1008)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def call(fn, good, **change):
    args = dict(good, **change)
    return fn(*args.values())


def test_block_plan(lib):
    good = dict(lens=P, add=P, held=P, batch=4, free=P, free_count=9, head=P, table=P, stride=8, bs=16, blocks=64,
                cap=32, olens=P, oheld=P, ohead=P, ostart=P, opos=P, oreq=P, oslot=P, status=NULL, stream=NULL)
    for bad in (dict(lens=NULL), dict(add=NULL), dict(held=NULL), dict(batch=-1), dict(batch=(1 << 24) + 1),
                dict(free=NULL), dict(free_count=-1), dict(head=NULL), dict(table=NULL), dict(stride=-1), dict(bs=8),
                dict(bs=24), dict(bs=512), dict(blocks=0), dict(cap=-1), dict(olens=NULL), dict(oheld=NULL),
                dict(ohead=NULL), dict(ostart=NULL), dict(opos=NULL), dict(oreq=NULL), dict(oslot=NULL),
                dict(cap=2 ** 31 - 1), dict(free_count=2 ** 31 - 1),
                dict(lens=ODD), dict(table=ODD), dict(oslot=ctypes.c_void_p(0x1004)), dict(status=ODD)):
        assert call(lib.smp_block_plan, good, **bad) == 1, bad


def test_norm_rope(lib):
    good = dict(q=P, k=P, tokens=4, hq=8, hk=2, d=64, qs=512, ks=128, dtype=1, qw=P, kw=P, eps=1e-6, table=P, rows=10,
                rotary=64, inter=0, pos=P, oq=P, ok=P, oqs=512, oks=128, status=NULL, stream=NULL)
    for bad in (dict(q=NULL), dict(k=NULL), dict(tokens=-1), dict(hq=0), dict(hk=-1), dict(d=0), dict(d=257),
                dict(qs=511), dict(ks=127), dict(oqs=100), dict(oks=100), dict(eps=-1.0), dict(eps=float("nan")),
                dict(table=NULL), dict(rows=-1), dict(rotary=66), dict(rotary=63), dict(pos=NULL), dict(oq=NULL),
                dict(ok=NULL), dict(q=ODD), dict(qw=ODD), dict(pos=ODD), dict(status=ODD)):
        assert call(lib.smp_qk_norm_rope, good, **bad) == 1, bad
    assert call(lib.smp_qk_norm_rope, good, dtype=2) == 2


class Cache(ctypes.Structure):
    """smp_cache of include/smp_cache.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32)]


def a_cache(**change):
    fields = dict(k=0x1000, v=0x1000, ks=0x1000, vs=0x1000, n=8, h=2, bs=16, d=64, type=0)
    fields.update(change)
    return ctypes.byref(Cache(*fields.values()))


BAD_CACHES = [(dict(k=0), 1), (dict(v=0), 1), (dict(ks=0), 1), (dict(vs=0), 1), (dict(n=0), 1), (dict(h=0), 1),
              (dict(bs=8), 1), (dict(bs=48), 1), (dict(bs=512), 1), (dict(d=72), 1), (dict(d=0), 1), (dict(d=272), 1),
              (dict(k=0x1008), 1), (dict(ks=0x1002), 1), (dict(type=2), 2)]


def test_cache_append(lib):
    good = dict(cache=a_cache(), k=P, v=P, tokens=4, ks=128, vs=128, dtype=1, slots=P, status=NULL, stream=NULL)
    for bad, code in BAD_CACHES:
        assert call(lib.smp_cache_append, good, cache=a_cache(**bad)) == code, bad
    for bad in (dict(cache=None), dict(k=NULL), dict(v=NULL), dict(tokens=-1), dict(ks=127), dict(vs=127),
                dict(slots=NULL), dict(slots=ctypes.c_void_p(0x1004)), dict(k=ODD), dict(status=ODD)):
        assert call(lib.smp_cache_append, good, **bad) == 1, bad
    assert call(lib.smp_cache_append, good, dtype=7) == 2


def test_cache_attention(lib):
    good = dict(cache=a_cache(), q=P, tokens=4, hq=8, qs=512, dtype=1, start=P, lens=P, batch=2, table=P, stride=4,
                scale=0.1, window=0, out=P, os=512, lse=NULL, status=NULL, work=P, work_bytes=64 << 20, stream=NULL)
    for bad, code in BAD_CACHES:
        assert call(lib.smp_cache_attention, good, cache=a_cache(**bad)) == code, bad
    for bad in (dict(q=NULL), dict(out=NULL), dict(start=NULL), dict(lens=NULL), dict(table=NULL), dict(tokens=-1),
                dict(hq=0), dict(hq=7), dict(qs=511), dict(os=511), dict(batch=-1), dict(stride=-1),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1), dict(q=ODD), dict(lse=ODD),
                dict(lens=ODD), dict(status=ODD)):
        assert call(lib.smp_cache_attention, good, **bad) == 1, bad
    assert call(lib.smp_cache_attention, good, dtype=7) == 2
    for bad in (dict(work=NULL), dict(work_bytes=0), dict(work=HALF)):
        assert call(lib.smp_cache_attention, good, **bad) == 5, bad
    assert lib.smp_cache_attention_workspace_bytes(4, 7, 2, 64, 2) == 0
    assert lib.smp_cache_attention_workspace_bytes(4, 8, 2, 65, 2) == 0
    assert 0 < lib.smp_cache_attention_workspace_bytes(4, 8, 2, 64, 2) <= 64 << 20


def test_verify_probs(lib):
    good = dict(p=P, q=P, ids=P, lens=NULL, batch=2, k=3, vocab=100, dtype=0, u=P, noise=P, oacc=P, oids=P,
                status=NULL, stream=NULL)
    for bad in (dict(p=NULL), dict(ids=NULL), dict(u=NULL), dict(noise=NULL), dict(oacc=NULL), dict(oids=NULL),
                dict(batch=-1), dict(batch=(1 << 20) + 1), dict(k=-1), dict(k=17), dict(vocab=0), dict(p=ODD),
                dict(noise=ODD), dict(status=ODD), dict(lens=ODD)):
        assert call(lib.smp_spec_verify_probs, good, **bad) == 1, bad
    assert call(lib.smp_spec_verify_probs, good, dtype=3) == 2
    assert call(lib.smp_spec_verify_probs, good, vocab=(1 << 19) + 1) == 4


def test_the_python_layer_refuses_what_it_can_see():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 4, 16)
    with pytest.raises(binding.SmpError):                       # host tensors
        cache.qk_norm_rope(x, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(binding.SmpError):
        cache.cache_append(tuple(torch.zeros(1) for _ in range(4)), x, x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(binding.SmpError):
        binding.spec_verify_probs(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1),
                                  torch.zeros(1, 8))


def test_tensors_of_two_gpus_are_refused():
    # tensors that only claim a GPU: the answer comes before anything looks at their memory
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode

    if torch.cuda.is_available():
        pytest.skip("claimed devices: only where no GPU is initialised for them")
    i32, f32, i64 = torch.int32, torch.float32, torch.int64
    with FakeTensorMode():
        def t(*shape, dtype=i32):
            return torch.empty(shape, dtype=dtype, device="cuda:0")

        def kv():
            codes = t(4, 2, 16, 32, dtype=torch.int8)
            return codes, t(4, 2, 16, 32, dtype=torch.int8), t(4, 2, dtype=f32), t(4, 2, dtype=f32)

        plan = dict(lens=t(2), add=t(2), held=t(2), free_blocks=t(5), free_head=t(1), block_table=t(2, 4), block_size=16,
                    num_blocks=9, max_tokens=8, status=t(1))
        rope = dict(q=t(4, 8, 32, dtype=f32), k=t(4, 2, 32, dtype=f32), positions=t(4), table=t(9, 32, dtype=f32),
                    q_weight=t(32, dtype=f32), k_weight=t(32, dtype=f32), out_q=t(4, 8, 32, dtype=f32),
                    out_k=t(4, 2, 32, dtype=f32), status=t(1))
        append = dict(k=t(4, 2, 32, dtype=f32), v=t(4, 2, 32, dtype=f32), slots=t(4, dtype=i64), status=t(1))
        attend = dict(q=t(4, 8, 32, dtype=f32), start=t(3), lens=t(2), block_table=t(2, 4), out=t(4, 8, 32, dtype=f32),
                      lse=t(4, 8, dtype=f32), workspace=t(1 << 20, dtype=torch.uint8), status=t(1))
        probs = dict(p=t(2, 4, 50, dtype=f32), q=t(2, 3, 50, dtype=f32), draft_ids=t(2, 3), uniforms=t(2, 3, dtype=f32),
                     noise=t(2, 50, dtype=f32), draft_lens=t(2), out_accepted=t(2), out_ids=t(2, 4), status=t(1))
        calls = [(cache.block_plan, plan), (cache.qk_norm_rope, rope), (lambda **kw: cache.cache_append(kv(), **kw), append),
                 (lambda **kw: cache.cache_attention(kv(), **kw), attend), (binding.spec_verify_probs, probs)]
        for call, good in calls:
            for name, value in list(good.items())[1:]:
                if isinstance(value, int):
                    continue
                other = torch.empty(value.shape, dtype=value.dtype, device="cuda:1")
                with pytest.raises(binding.SmpError, match="must be on one GPU"):
                    call(**dict(good, **{name: other}))


def test_no_outputs_are_made_for_what_is_refused():
    # outputs and scratch left to the call: their shapes come from arguments that have to be looked at first
    torch = pytest.importorskip("torch")
    i32 = torch.int32
    t = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype)  # noqa: E731
    kv = (t(3, 2, 16, 32, dtype=torch.int8), t(3, 2, 16, 32, dtype=torch.int8), t(3, 2), t(3, 2))
    plan = (t(2, dtype=i32), t(2, dtype=i32), t(5, dtype=i32), t(1, dtype=i32), t(2, 4, dtype=i32), 16, 5)
    attend = (t(3, dtype=i32), t(2, dtype=i32), t(2, 4, dtype=i32))
    probs = (t(2, 3, 50), t(2, 3, dtype=i32), t(2, 3), t(2, 50))
    for call in (lambda: cache.block_plan(None, *plan, 8), lambda: cache.block_plan(t(dtype=i32), *plan, 8),
                 lambda: cache.block_plan(t(2, dtype=i32), *plan, -1),
                 lambda: cache.qk_norm_rope(None, None, t(4, dtype=i32)),
                 lambda: cache.qk_norm_rope([[1.0]], None, t(4, dtype=i32)),
                 lambda: cache.qk_norm_rope(t(4, 8, 32), [1.0], t(4, dtype=i32)),
                 lambda: cache.cache_attention(kv, None, *attend), lambda: cache.cache_attention(kv, t(4, 8), *attend),
                 lambda: cache.cache_attention(None, t(4, 8, 32), *attend),
                 lambda: cache.cache_attention(kv[:1], t(4, 8, 32), *attend),
                 lambda: cache.cache_attention(kv, t(4, 8, 32), t(3, dtype=i32), None, t(2, 4, dtype=i32)),
                 lambda: cache.cache_attention(kv, None, *attend, out=t(4, 8, 32), workspace=t(9, dtype=torch.uint8)),
                 lambda: cache.cache_attention(kv, t(4, 8, 0), *attend, out=t(4, 8, 0), workspace=t(9, dtype=torch.uint8)),
                 lambda: binding.spec_verify_probs(None, *probs), lambda: binding.spec_verify_probs(t(2), *probs)):
        with pytest.raises(binding.SmpError):
            call()

"""Host-side validation of the calls on rows of logits: bad arguments are
answered before anything touches a GPU."""

import ctypes

import pytest

from spec_verify_gb300 import binding, build, scores

P = ctypes.c_void_p(0x1000)
Q = ctypes.c_void_p(0x9000)
ODD = ctypes.c_void_p(0x1001)
NULL = ctypes.c_void_p(0)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def call(fn, good, **change):
    args = dict(good, **change)
    return fn(*args.values())


ROWS = dict(logits=P, rows=4, vocab=100, stride=100, dtype=1, temperature=1.0, temperatures=NULL)
BAD_ROWS = [dict(logits=NULL), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=-5), dict(stride=99),
            dict(stride=(1 << 40) + 1), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=NAN),
            dict(temperature=INF), dict(temperature=2.0 ** -31), dict(temperature=2.0 ** 31), dict(logits=ODD),
            dict(temperatures=ODD), dict(status=ODD)]


def check_rows(fn, good):
    for bad in BAD_ROWS:
        assert call(fn, good, **bad) == 1, bad
    assert call(fn, good, dtype=2) == 2
    assert call(fn, good, vocab=(1 << 19) + 1, stride=1 << 20) == 4


def test_token_logprobs(lib):
    good = dict(ROWS, ids=P, count=2, top=3, lp=P, entropy=P, top_ids=P, top_lp=P, status=NULL, stream=NULL)
    check_rows(lib.smp_token_logprobs, good)
    for bad in (dict(ids=NULL), dict(count=-1), dict(count=129), dict(top=-1), dict(top=129), dict(lp=NULL), dict(top_ids=NULL),
                dict(top_lp=NULL), dict(count=0, top=0, entropy=NULL), dict(ids=ODD), dict(lp=ODD), dict(entropy=ODD),
                dict(top_ids=ODD), dict(top_lp=ODD)):
        assert call(lib.smp_token_logprobs, good, **bad) == 1, bad


def test_token_logprobs_grad(lib):
    good = dict(ROWS, ids=P, count=2, g=P, h=P, grad=Q, gs=100, status=NULL, stream=NULL)
    check_rows(lib.smp_token_logprobs_grad, good)
    for bad in (dict(ids=NULL), dict(count=-1), dict(count=129), dict(g=NULL), dict(count=0, h=NULL), dict(grad=NULL),
                dict(gs=99), dict(gs=(1 << 40) + 1), dict(grad=P, gs=104), dict(ids=ODD), dict(g=ODD), dict(h=ODD),
                dict(grad=ODD)):
        assert call(lib.smp_token_logprobs_grad, good, **bad) == 1, bad


def test_distill(lib):
    good = dict(ROWS, ids=P, values=P, count=2, tail=1, w=P, loss=P, grad=Q, gs=100, status=NULL, stream=NULL)
    check_rows(lib.smp_distill, good)
    for bad in (dict(ids=NULL), dict(values=NULL), dict(count=0), dict(count=129), dict(loss=NULL), dict(gs=99),
                dict(gs=(1 << 40) + 1), dict(grad=P, gs=104), dict(ids=ODD), dict(values=ODD), dict(w=ODD), dict(loss=ODD),
                dict(grad=ODD)):
        assert call(lib.smp_distill, good, **bad) == 1, bad


def test_gradients_over_the_logits(lib):
    """Rows lie in the logits' place or share no element with them."""
    at = lambda elements: ctypes.c_void_p((1 << 20) + 2 * elements)  # noqa: E731
    good = dict(ROWS, logits=at(0), vocab=100, stride=300, ids=P, count=2, g=P, h=P, grad=P, gs=300, status=NULL, stream=NULL)
    for elements, gs in ((1, 300), (99, 300), (-1, 300), (-99, 300), (201, 300), (299, 300), (301, 300), (600, 300), (150, 301),
                         (0, 301), (-500, 400), (900, 300 - 1)):
        assert call(lib.smp_token_logprobs_grad, good, grad=at(elements), gs=gs) == 1, (elements, gs)
    for elements in (1, 99, -99, 50):
        assert call(lib.smp_token_logprobs_grad, dict(good, rows=1), grad=at(elements)) == 1, elements


def test_no_rows_are_no_work(lib):
    assert lib.smp_token_logprobs(NULL, 0, 100, 100, 0, 1.0, NULL, NULL, 2, 0, NULL, NULL, NULL, NULL, NULL, NULL) == 0
    assert lib.smp_token_logprobs_grad(NULL, 0, 100, 100, 0, 1.0, NULL, NULL, 2, NULL, NULL, NULL, 100, NULL, NULL) == 0
    assert lib.smp_distill(NULL, 0, 100, 100, 0, 1.0, NULL, NULL, NULL, 2, 1, NULL, NULL, NULL, 0, NULL, NULL) == 0


def fakes():
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode

    if torch.cuda.is_available():
        pytest.skip("claimed devices: only where no GPU is initialised for them")
    return torch, FakeTensorMode()


def good_calls(torch):
    def t(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda:0")

    i32 = torch.int32
    out = (t(4, 2), t(4), t(4, 3, dtype=i32), t(4, 3))
    return [(scores.token_logprobs, dict(logits=t(4, 50), ids=t(4, 2, dtype=i32), top=3, entropy=True, temperature=t(4),
                                         out=out, status=t(1, dtype=i32))),
            (scores.token_logprobs_grad, dict(logits=t(4, 50), ids=t(4, 2, dtype=i32), grad_logprobs=t(4, 2),
                                              grad_entropy=t(4), temperature=t(4), out=t(4, 50), status=t(1, dtype=i32))),
            (scores.distill_loss, dict(logits=t(4, 50), teacher_ids=t(4, 2, dtype=i32), teacher_logprobs=t(4, 2),
                                       temperature=t(4), out=t(4), status=t(1, dtype=i32))),
            (scores.distill_grad, dict(logits=t(4, 50), teacher_ids=t(4, 2, dtype=i32), teacher_logprobs=t(4, 2), weight=t(4),
                                       temperature=t(4), out_loss=t(4), out=t(4, 50), status=t(1, dtype=i32)))]


def test_tensors_of_two_gpus_are_refused():
    # tensors that only claim a GPU: the answer comes before anything looks at their memory
    torch, mode = fakes()
    with mode:
        for fn, good in good_calls(torch):
            for name, value in list(good.items())[1:]:
                if name == "out" and isinstance(value, tuple):
                    others = [tuple(torch.empty_like(x, device="cuda:1") if i == j else x for j, x in enumerate(value))
                              for i in range(4)]
                elif isinstance(value, torch.Tensor):
                    others = [torch.empty_like(value, device="cuda:1")]
                else:
                    continue
                for other in others:
                    with pytest.raises(binding.SmpError, match="must be on one GPU"):
                        fn(**dict(good, **{name: other}))


def test_shapes_and_types_are_refused():
    torch, mode = fakes()
    with mode:
        t = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda:0")  # noqa: E731
        i32, i64 = torch.int32, torch.int64
        for fn, good in good_calls(torch):
            bad = [dict(logits=t(4, 50, dtype=torch.float16)), dict(logits=t(200)), dict(logits=t(50, 4).t()),
                   dict(logits=t(1, 50).expand(4, 50)), dict(logits=t(4, 100)[:, ::2]), dict(temperature=t(3)),
                   dict(temperature=t(4, dtype=torch.float64)), dict(status=t(1))]
            for name, value in good.items():
                if name in ("logits", "status", "temperature") or not isinstance(value, torch.Tensor):
                    continue
                other = {i32: i64, torch.float32: torch.float64}[value.dtype]
                bad += [{name: t(*value.shape, dtype=other)}, {name: t(5, *value.shape[1:], dtype=value.dtype)}, {name: 3.0}]
            if fn is scores.token_logprobs:
                out = good["out"]
                bad += [dict(entropy=False), dict(out=out[:3]), dict(out=(None, *out[1:])), dict(out=(*out[:2], None, out[3])),
                        dict(top=0), dict(top=2), dict(ids=None), dict(out=(out[0], out[1], out[2], t(4, 4)))]
            if fn is scores.token_logprobs_grad:
                bad += [dict(ids=None), dict(grad_logprobs=None)]
            for change in bad:
                with pytest.raises(binding.SmpError):
                    fn(**dict(good, **change))


def test_no_outputs_are_made_for_what_is_refused():
    torch = pytest.importorskip("torch")
    t = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype)  # noqa: E731
    ids = t(4, 2, dtype=torch.int32)
    for fn in (lambda: scores.token_logprobs(None, ids), lambda: scores.token_logprobs(t(50), ids),
               lambda: scores.token_logprobs(t(4, 50), t(4)), lambda: scores.token_logprobs(t(4, 50), top=-1),
               lambda: scores.token_logprobs(t(4, 50), ids),                     # host tensors
               lambda: scores.token_logprobs_grad(None, ids, t(4, 2)), lambda: scores.token_logprobs_grad(t(4, 50), ids, t(4, 2)),
               lambda: scores.distill_loss(t(50), ids, t(4, 2)), lambda: scores.distill_loss(t(4, 50), ids, t(4, 2)),
               lambda: scores.distill_grad([1.0], ids, t(4, 2)), lambda: scores.distill_grad(t(4, 50), ids, t(4, 2))):
        with pytest.raises(binding.SmpError):
            fn()

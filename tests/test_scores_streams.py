"""Tensors that the calls on rows of logits make themselves belong to the stream
that the call is launched on, and lie as the documentation says.  Host logic
alone: the native calls are replaced by a recorder, torch by a stand-in that
notes the current stream of each allocation."""

import contextlib

import pytest

from spec_verify_gb300 import binding, scores

torch = pytest.importorskip("torch")


class Stream:
    cuda_stream = 0x5000


class Recorder:
    def __getattr__(self, name):
        def call(*args):
            self.args = args
        return call


class Cuda:
    def __init__(self):
        self.current = "the caller's"

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before


class Torch:
    int32, float32 = torch.int32, torch.float32

    def __init__(self):
        self.cuda, self.made = Cuda(), []

    def empty(self, shape, dtype, device):
        t = torch.empty(shape, dtype=dtype)
        self.made.append((t, self.cuda.current))
        return t


@pytest.fixture
def stand_in(monkeypatch):
    fake, native = Torch(), Recorder()
    for module in (scores, binding):
        monkeypatch.setattr(module, "_torch", lambda: fake)
        monkeypatch.setattr(module, "step_module", lambda: native)
    return fake, native


LOGITS, IDS, VALUES = torch.zeros(4, 50), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 3)
CALLS = {
    "token_logprobs": (lambda **kw: scores.token_logprobs(LOGITS, IDS, top=2, entropy=True, **kw), 4),
    "token_logprobs_grad": (lambda **kw: scores.token_logprobs_grad(LOGITS, IDS, VALUES, **kw), 1),
    "distill_loss": (lambda **kw: scores.distill_loss(LOGITS, IDS, VALUES, **kw), 1),
    "distill_grad": (lambda **kw: scores.distill_grad(LOGITS, IDS, VALUES, **kw), 2),
}


@pytest.mark.parametrize("name", CALLS)
def test_own_tensors_belong_to_the_stream_of_the_launch(name, stand_in):
    fake, native = stand_in
    call, count = CALLS[name]
    s = Stream()
    call(stream=s)
    assert native.args[-1] == s.cuda_stream
    assert len(fake.made) == count and all(on is s for _, on in fake.made)
    assert fake.cuda.current == "the caller's"
    given = {a.data_ptr() for a in native.args if isinstance(a, torch.Tensor)}
    assert all(t.data_ptr() in given for t, _ in fake.made)                  # they are what the call was given
    fake.made.clear()
    call()
    assert native.args[-1] is None and all(on == "the caller's" for _, on in fake.made)


@pytest.mark.parametrize("dtype,per", [(torch.float32, 4), (torch.bfloat16, 8)])
@pytest.mark.parametrize("rows,vocab,stride", [(3, 50, 50), (3, 50, 64), (5, 33, 36), (4, 7, 4000), (1, 9, 9), (0, 9, 9)])
def test_a_gradients_own_rows(rows, vocab, stride, dtype, per, stand_in):
    """As far from 16-byte boundaries as the logits' rows, and hardly further apart than they are long."""
    logits = torch.zeros(max(rows, 1), stride, dtype=dtype)[:rows, :vocab]
    grad = scores.token_logprobs_grad(logits, None, None, torch.zeros(rows))
    assert grad.shape == logits.shape and grad.dtype == dtype
    if rows > 1:
        assert vocab <= grad.stride(0) < vocab + per and (grad.stride(0) - stride) % per == 0

"""Tensors that the cached step's calls make themselves belong to the stream
that the call is launched on: with `stream=` given, every allocation happens
while that stream is the current one.  Host logic alone: the native calls are
replaced by a recorder, torch by a stand-in that notes the current stream of
each allocation."""

import contextlib

import pytest

from spec_verify_gb300 import binding, cache

torch = pytest.importorskip("torch")


class Stream:
    cuda_stream = 0x5000


class Recorder:
    """In place of the native module: keeps the arguments of the last call."""

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
    """torch with `empty` on the host, noting the stream it was called on."""

    int32, int64, uint8 = torch.int32, torch.int64, torch.uint8

    def __init__(self):
        self.cuda, self.made = Cuda(), []

    def empty(self, shape, dtype, device):
        t = torch.empty(shape, dtype=dtype)
        self.made.append((t, self.cuda.current))
        return t


@pytest.fixture
def stand_in(monkeypatch):
    fake, native = Torch(), Recorder()
    for module in (cache, binding):
        monkeypatch.setattr(module, "_torch", lambda: fake)
        monkeypatch.setattr(module, "step_module", lambda: native)
    monkeypatch.setattr(cache, "attention_workspace_bytes", lambda *sizes: 4096)
    return fake, native


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def kv():
    codes, scale = torch.zeros(3, 2, 16, 32, dtype=torch.int8), torch.ones(3, 2)
    return codes, codes.clone(), scale, scale.clone()


CALLS = {
    "block_plan": (lambda **kw: cache.block_plan(i32(2), i32(2), i32(2), i32(5), i32(1), i32(2, 4), 16, 5, 8, **kw), 7),
    "qk_norm_rope": (lambda **kw: cache.qk_norm_rope(torch.zeros(4, 8, 32), torch.zeros(4, 2, 32), i32(4), **kw), 2),
    "cache_append": (lambda **kw: cache.cache_append(kv(), torch.zeros(4, 2, 32), torch.zeros(4, 2, 32),
                                                     torch.zeros(4, dtype=torch.int64), **kw), 0),
    "cache_attention": (lambda **kw: cache.cache_attention(kv(), torch.zeros(4, 8, 32), i32(3), i32(2), i32(2, 4), **kw), 2),
    "spec_verify_probs": (lambda **kw: binding.spec_verify_probs(torch.zeros(2, 4, 50), torch.zeros(2, 3, 50), i32(2, 3),
                                                                 torch.zeros(2, 3), torch.zeros(2, 50), **kw), 2),
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
    assert all(any(t is a for a in native.args) for t, _ in fake.made)       # they are what the call was given
    fake.made.clear()
    call()
    assert native.args[-1] is None and all(on == "the caller's" for _, on in fake.made)

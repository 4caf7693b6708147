"""Tensors that the sampler's, the verifier's and the beam step's calls make
themselves (outputs, status words, scratch, parameter records) belong to the
stream that the call is launched on.  Host logic alone: the library is
replaced by a recorder, torch by a stand-in that notes the current stream of
each allocation."""

import contextlib

import numpy as np
import pytest

from spec_verify_gb300 import binding, workloads

torch = pytest.importorskip("torch")


class Stream:
    cuda_stream = 0x5000


class Library:
    """In place of libsmp: every call succeeds; the last argument of the last one is kept."""

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 4096
            self.stream = args[-1].value
            return 0
        return call


class Device(torch.Tensor):
    """A host tensor that passes for one on the GPU."""
    is_cuda = property(lambda self: True)


class Cuda:
    def __init__(self):
        self.current = Stream()
        self.current.cuda_stream = 0x7000

    def current_stream(self):
        return self.current

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before


class Torch:
    """torch, with `empty` noting the stream it was called on."""

    def __init__(self):
        self.cuda, self.made = Cuda(), []

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *shape, dtype, device):
        self.made.append(self.cuda.current)
        return torch.empty(*shape, dtype=dtype)


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Device)


def params(b):
    return workloads.make_params(b)


LOGITS, P, Q, IDS = (3, 40), (3, 5, 40), (3, 4, 40), (3, 4)
CALLS = {
    "sample": lambda **kw: binding.sample(on_gpu(*LOGITS), params(3), **kw),
    "sample_processed": lambda **kw: binding.sample_processed(on_gpu(*LOGITS), params(3), **kw),
    "sample_rows": lambda **kw: binding.sample_rows(on_gpu(*LOGITS), params(3), **kw),
    "logit_prepass": lambda **kw: binding.logit_prepass(on_gpu(*LOGITS), **kw),
    "filter_debug": lambda **kw: binding.filter_debug(on_gpu(*LOGITS), params(3), **kw),
    "spec_verify": lambda **kw: binding.spec_verify(on_gpu(*P), on_gpu(*Q), on_gpu(*IDS, dtype=torch.int32), **kw),
    "spec_verify_params": lambda **kw: binding.spec_verify_params(on_gpu(*P), on_gpu(*Q), on_gpu(*IDS, dtype=torch.int32),
                                                                  params(3), **kw),
    "spec_verify_rows": lambda **kw: binding.spec_verify_rows(on_gpu(*P), on_gpu(*Q), on_gpu(*IDS, dtype=torch.int32),
                                                              params(3), **kw),
    "spec_verify_static": lambda **kw: binding.spec_verify_static(on_gpu(*P), on_gpu(*Q), on_gpu(*IDS, dtype=torch.int32),
                                                                  **kw),
    "beam_topk": lambda **kw: binding.beam_topk(on_gpu(2, 3, 40), on_gpu(2, 3, dtype=torch.float64), **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_own_tensors_belong_to_the_stream_of_the_launch(name, monkeypatch):
    fake, lib, copied = Torch(), Library(), []
    monkeypatch.setattr(binding, "_torch", lambda: fake)
    monkeypatch.setattr(binding, "load", lambda: lib)
    to_device = lambda p, device: copied.append(fake.cuda.current) or torch.from_numpy(  # noqa: E731
        np.ascontiguousarray(p).view(np.uint8).copy())
    monkeypatch.setattr(binding, "params_to_device", to_device)
    s, default = Stream(), fake.cuda.current
    CALLS[name](stream=s)
    assert lib.stream == s.cuda_stream
    assert fake.made and all(on is s for on in fake.made + copied)
    assert fake.cuda.current is default
    fake.made.clear(), copied.clear()
    CALLS[name]()
    assert lib.stream == default.cuda_stream and all(on is default for on in fake.made + copied)

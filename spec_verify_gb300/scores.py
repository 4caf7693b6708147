"""Binding of libsmp's calls on rows of logits (include/smp_scores.h): log
probabilities of tokens, entropies and likeliest tokens, and the losses that a
draft model is trained on, with their gradients.  The checks and the
marshalling are native (csrc/step_binding.cpp).

Logits are [rows, vocab], float32 or bfloat16, rows contiguous, any distance
apart (a padded projection cut to its vocabulary).  `temperature` is a number,
or a float32 [rows] tensor of one per row, by which the logits are divided.
Every call takes `status`, an int32 [1] CUDA tensor that is cleared and gets
the ROW_* flags of binding.py, or None (no status word), and `stream`, a
torch.cuda.Stream, or None for the current one.  Tensors that a call makes
itself belong to the stream it is launched on.  What a call cannot take is
refused with SmpError before anything is launched.

Nothing here is recorded by autograd: a gradient is a call of its own, which
keeps nothing from the forward call, and goes on with `logits.backward(grad)`:

    record = scores.token_logprobs(target_logits, top=64)          # the teacher's, once
    loss, grad = scores.distill_grad(logits.detach(), record.top_ids, record.top_logprobs, weight, tail=True)
    logits.backward(grad)                                          # weight: d total / d loss of each row
"""

import collections

from .binding import SmpError, _needs, _on, _torch, step_module

TokenLogprobs = collections.namedtuple("TokenLogprobs", "logprobs entropy top_ids top_logprobs")


def _queue(stream):
    return None if stream is None else stream.cuda_stream


def _beside(logits, stream):
    """A gradient's tensor: its rows end where they begin, but for what lets them
    lie to 16-byte boundaries as the logits' rows do (both then go by bulk copies)."""
    _needs(logits, "logits", 2)
    rows, vocab = logits.shape
    stride = vocab + (logits.stride(0) - vocab) % (16 // logits.element_size()) if rows > 1 else vocab
    with _on(stream):
        return _torch().empty((rows, stride), dtype=logits.dtype, device=logits.device)[:, :vocab]


def token_logprobs(logits, ids=None, top=0, entropy=False, temperature=1.0, out=None, status=None, stream=None):
    """smp_token_logprobs.  ids: int32 [rows, count], negative ones padding, or
    None; top: how many of the likeliest tokens are wanted; entropy: whether it
    is.  Returns TokenLogprobs(logprobs [rows, count], entropy [rows], top_ids
    [rows, top] (int32), top_logprobs [rows, top]) with None for what was not
    asked for, in the tensors of `out`, such a tuple, if given."""
    native = step_module()
    if out is None:
        torch = _torch()
        _needs(logits, "logits", 2)
        if ids is not None:
            _needs(ids, "ids", 2)
        if top < 0:
            raise SmpError("top must not be negative")
        rows, dev = logits.shape[0], logits.device
        with _on(stream):
            out = (None if ids is None else torch.empty((rows, ids.shape[1]), dtype=torch.float32, device=dev),
                   torch.empty((rows,), dtype=torch.float32, device=dev) if entropy else None,
                   torch.empty((rows, top), dtype=torch.int32, device=dev) if top else None,
                   torch.empty((rows, top), dtype=torch.float32, device=dev) if top else None)
    elif len(out) != 4 or (out[1] is not None) != bool(entropy):
        raise SmpError("out must be (logprobs, entropy, top_ids, top_logprobs), with None for what is not asked for")
    native.token_logprobs(logits, ids, top, temperature, *out, status, _queue(stream))
    return TokenLogprobs(*out)


def token_logprobs_grad(logits, ids, grad_logprobs, grad_entropy=None, temperature=1.0, out=None, status=None,
                        stream=None):
    """smp_token_logprobs_grad: the gradient in the logits of a loss whose
    gradients in the log probabilities (float32 [rows, count], as ids; both
    None: no ids) and the entropies (float32 [rows], or None) are given.  out:
    a tensor like the logits (the logits themselves: in place), or None for a
    new one, whose rows lie to 16-byte boundaries as the logits' do: others, as
    torch.empty_like makes them for logits cut from wider rows, take up to 1.4
    times as long.  Returns it."""
    native = step_module()
    if out is None:
        out = _beside(logits, stream)
    native.token_logprobs_grad(logits, ids, grad_logprobs, grad_entropy, temperature, out, status, _queue(stream))
    return out


def _losses(logits, out, stream):
    if out is not None:
        return out
    _needs(logits, "logits", 2)
    with _on(stream):
        return _torch().empty((logits.shape[0],), dtype=_torch().float32, device=logits.device)


def distill_loss(logits, teacher_ids, teacher_logprobs, tail=False, temperature=1.0, out=None, status=None,
                 stream=None):
    """smp_distill without its gradient: the divergence of each row from a
    teacher's likeliest tokens, teacher_ids (int32 [rows, count], negative ones
    unused) with teacher_logprobs (float32), as token_logprobs gives them at
    the same temperature.  tail: what the teacher has outside its ids counts as
    one more outcome; without it the ids' probabilities are renormalised.
    Returns float32 [rows] (`out`, if given)."""
    native = step_module()
    out = _losses(logits, out, stream)
    native.distill(logits, teacher_ids, teacher_logprobs, tail, temperature, None, out, None, status, _queue(stream))
    return out


def distill_grad(logits, teacher_ids, teacher_logprobs, weight=None, tail=False, temperature=1.0, out_loss=None,
                 out=None, status=None, stream=None):
    """smp_distill: distill_loss and, in the same pass, the gradient in the
    logits of sum(weight * loss); weight: float32 [rows], or None for ones.
    out: as for token_logprobs_grad.  Returns (loss, gradient)."""
    native = step_module()
    out_loss = _losses(logits, out_loss, stream)
    if out is None:
        out = _beside(logits, stream)
    native.distill(logits, teacher_ids, teacher_logprobs, tail, temperature, weight, out_loss, out, status,
                   _queue(stream))
    return out_loss, out

"""Binding of libsmp's cached speculative step (include/smp_cache.h): the
checks and the marshalling are native (csrc/step_binding.cpp), since a step
makes several of these calls and each is a few microseconds of kernel.

A cache is a tuple (k, v, k_scale, v_scale): codes [blocks, kv_heads,
block_size, head_dim] of torch.float8_e4m3fn or torch.int8, contiguous, and
float32 scales [blocks, kv_heads].  `new_cache` makes one.

Every call takes `status`, an int32 [1] CUDA tensor that is cleared and gets
the ROW_* flags of binding.py, or None (no status word), and `stream`, a
torch.cuda.Stream, or None for the current one.  Tensors that a call makes
itself (outputs not given, scratch) belong to the stream it is launched on.
What a call cannot take is refused with SmpError before anything is launched.
"""

import collections

from .binding import SmpError, _needs, _on, _torch, load, step_module

BlockPlan = collections.namedtuple("BlockPlan", "lens held free_head start position request slot")


def new_cache(num_blocks, kv_heads, block_size, head_dim, dtype=None, device="cuda"):
    """An empty cache (k, v, k_scale, v_scale) of float8_e4m3fn codes, or of
    `dtype` torch.int8."""
    torch = _torch()
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    codes = [torch.zeros(num_blocks, kv_heads, block_size, head_dim, dtype=torch.uint8, device=device).view(dtype)
             for _ in range(2)]
    scales = [torch.ones(num_blocks, kv_heads, dtype=torch.float32, device=device) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def rope_table(rows, rotary_dim, theta=10000.0, device="cuda"):
    """The [rows, rotary_dim] float32 table of qk_norm_rope: for position t and
    pair j, cos and sin of t * theta^(-2j / rotary_dim), computed in 64 bits."""
    torch = _torch()
    pos = torch.arange(rows, dtype=torch.float64, device=device)[:, None]
    freq = theta ** (-2.0 * torch.arange(rotary_dim // 2, dtype=torch.float64, device=device) / max(1, rotary_dim))
    return torch.cat([(pos * freq).cos(), (pos * freq).sin()], 1).float()


def _queue(stream):
    return None if stream is None else stream.cuda_stream


def block_plan(lens, add, held, free_blocks, free_head, block_table, block_size, num_blocks, max_tokens, out=None,
               status=None, stream=None):
    """smp_block_plan.  lens, add, held: int32 [B]; free_blocks: int32 [F];
    free_head: int32 [1]; block_table: int32 [B, columns], extended in place.
    Returns BlockPlan(lens [B], held [B], free_head [1], start [B + 1],
    position [max_tokens], request [max_tokens] (int32) and slot [max_tokens]
    (int64)), in the tensors of `out` if given."""
    native = step_module()
    if out is None:
        torch = _torch()
        _needs(lens, "lens", 1)
        if max_tokens < 0:
            raise SmpError("max_tokens must not be negative")
        b, i32 = lens.shape[0], torch.int32
        new = lambda n, t=i32: torch.empty(n, dtype=t, device=lens.device)  # noqa: E731
        with _on(stream):
            out = (new(b), new(b), new(1), new(b + 1), new(max_tokens), new(max_tokens), new(max_tokens, torch.int64))
    native.block_plan(lens, add, held, free_blocks, free_head, block_table, block_size, num_blocks, max_tokens, *out,
                      status, _queue(stream))
    return BlockPlan(*out)


def qk_norm_rope(q, k, positions, table=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out_q=None,
                 out_k=None, status=None, stream=None):
    """smp_qk_norm_rope.  q [T, Hq, D] and k [T, Hk, D] (or None), float32 or
    bfloat16, views of a fused projection allowed; positions: int32 [T];
    table: float32 [rows, rotary_dim] (rope_table), or None for the norm
    alone; weights: float32 [D] or None.  out_q, out_k: tensors to write (q
    and k themselves: in place), or None for new ones.  Returns (out_q,
    out_k)."""
    native = step_module()
    if out_q is None or (k is not None and out_k is None):
        _needs(q, "q", 3)
        if k is not None:
            _needs(k, "k", 3)
        with _on(stream):
            if out_q is None:
                out_q = _torch().empty(q.shape, dtype=q.dtype, device=q.device)
            if k is not None and out_k is None:
                out_k = _torch().empty(k.shape, dtype=k.dtype, device=k.device)
    native.qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps, interleaved, out_q, out_k, status,
                        _queue(stream))
    return out_q, out_k


def cache_append(cache, k, v, slots, status=None, stream=None):
    """smp_cache_append: k and v [T, kv_heads, head_dim] (float32 or bfloat16)
    into the cache's slots (int64 [T], BlockPlan.slot)."""
    step_module().cache_append(cache, k, v, slots, status, _queue(stream))


def attention_workspace_bytes(tokens, q_heads, kv_heads, head_dim, batch):
    return int(load().smp_cache_attention_workspace_bytes(tokens, q_heads, kv_heads, head_dim, batch))


def cache_attention(cache, q, start, lens, block_table, scale=None, window=0, out=None, lse=None, workspace=None,
                    status=None, stream=None):
    """smp_cache_attention: q [T, Hq, D] over the cache; start: int32 [B + 1]
    (BlockPlan.start), lens: int32 [B], the lengths with the step's tokens
    (BlockPlan.lens), block_table: int32 [B, columns].  scale defaults to
    D^-0.5; window 0 sees every earlier key.  lse: a float32 [T, Hq] tensor to
    fill, or None; workspace: a uint8 CUDA tensor of
    attention_workspace_bytes(...) that no overlapping call uses, or None to
    allocate one.  Returns out [T, Hq, D]."""
    native = step_module()
    if out is None or workspace is None:
        torch = _torch()
        _needs(q, "q", 3)
        _needs(lens, "lens", 1)
        if not isinstance(cache, tuple) or len(cache) != 4:
            raise SmpError("a cache is a tuple (k, v, k_scale, v_scale)")
        _needs(cache[0], "k", 4)
        with _on(stream):
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if workspace is None:
                need = attention_workspace_bytes(q.shape[0], q.shape[1], cache[0].shape[1], q.shape[2], lens.shape[0])
                workspace = torch.empty(max(16, need), dtype=torch.uint8, device=q.device)
    native.cache_attention(cache, q, start, lens, block_table, scale, window, out, lse, workspace, status,
                           _queue(stream))
    return out

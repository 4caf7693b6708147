"""Binding of libsmp's cached speculative step (include/smp_cache.h): argument
checks and marshalling only, as in binding.py.

A cache is a tuple (k, v, k_scale, v_scale): codes [blocks, kv_heads,
block_size, head_dim] of torch.float8_e4m3fn or torch.int8, contiguous, and
float32 scales [blocks, kv_heads].  `new_cache` makes one.

Every call takes `status`, an int32 [1] CUDA tensor that is cleared and gets
the ROW_* flags of binding.py, or None (no status word), and `stream`, a
torch.cuda.Stream, or None for the current one.
"""

import collections
import ctypes

from .binding import SMP_BF16, SMP_F32, SmpError, _check, _torch, load

SMP_CACHE_E4M3 = 0
SMP_CACHE_I8 = 1

BlockPlan = collections.namedtuple("BlockPlan", "lens held free_head start position request slot")


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32)]


def _at(t):
    return None if t is None else t.data_ptr()


def _queue(stream):
    torch = _torch()
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _flat(name, t, dtype, *shape):
    """t is a contiguous CUDA tensor of this dtype and shape (None: any size)."""
    if t.dtype != dtype or t.dim() != len(shape) or not t.is_cuda or not t.is_contiguous() or \
            any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise SmpError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {list(shape)}, got {t.dtype} "
                       f"{list(t.shape)}")


def _status(status):
    if status is not None:
        _flat("status", status, _torch().int32, None)
        if status.numel() < 1:
            raise SmpError("status must hold one int32")


def _heads(name, t, dtype=None, shape=None):
    """Token stride, in elements, of a [tokens, heads, dim] CUDA tensor whose
    heads are contiguous; tokens may be further apart."""
    torch = _torch()
    if t.dim() != 3 or not t.is_cuda:
        raise SmpError(f"{name} must be a [tokens, heads, dim] CUDA tensor")
    if t.dtype not in (torch.float32, torch.bfloat16) or (dtype is not None and t.dtype != dtype):
        raise SmpError(f"{name} must be float32 or bfloat16, the same as the others, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise SmpError(f"{name} must have the shape {list(shape)}, got {list(t.shape)}")
    n, h, d = t.shape
    token, head, element = t.stride()
    if (element != 1 and d > 1) or (head != d and h > 1) or (token < h * d and n > 1):
        raise SmpError(f"the heads of {name} must be contiguous and its tokens in order")
    return max(token, h * d)


def _code(t):
    return SMP_BF16 if t.dtype == _torch().bfloat16 else SMP_F32


def _cache_arg(cache):
    torch = _torch()
    k, v, ks, vs = cache
    if k.dtype == torch.float8_e4m3fn:
        kind = SMP_CACHE_E4M3
    elif k.dtype == torch.int8:
        kind = SMP_CACHE_I8
    else:
        raise SmpError(f"cache codes must be float8_e4m3fn or int8, got {k.dtype}")
    if k.dim() != 4:
        raise SmpError("cache codes must be [blocks, kv_heads, block_size, head_dim]")
    n, h, bs, d = k.shape
    _flat("k", k, k.dtype, n, h, bs, d)
    _flat("v", v, k.dtype, n, h, bs, d)
    _flat("k_scale", ks, torch.float32, n, h)
    _flat("v_scale", vs, torch.float32, n, h)
    return _Cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n, h, bs, d, kind)


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


def block_plan(lens, add, held, free_blocks, free_head, block_table, block_size, num_blocks, max_tokens, out=None,
               status=None, stream=None):
    """smp_block_plan.  lens, add, held: int32 [B]; free_blocks: int32 [F];
    free_head: int32 [1]; block_table: int32 [B, columns], extended in place.
    Returns BlockPlan(lens [B], held [B], free_head [1], start [B + 1],
    position [max_tokens], request [max_tokens] (int32) and slot [max_tokens]
    (int64)), in the tensors of `out` if given."""
    torch = _torch()
    lib = load()
    i32 = torch.int32
    b = lens.shape[0]
    _flat("lens", lens, i32, b)
    _flat("add", add, i32, b)
    _flat("held", held, i32, b)
    _flat("free_blocks", free_blocks, i32, None)
    _flat("free_head", free_head, i32, 1)
    _flat("block_table", block_table, i32, b, None)
    _status(status)
    if out is None:
        new = lambda n, t=i32: torch.empty(n, dtype=t, device=lens.device)  # noqa: E731
        out = BlockPlan(new(b), new(b), new(1), new(b + 1), new(max_tokens), new(max_tokens),
                        new(max_tokens, torch.int64))
    else:
        out = BlockPlan(*out)
        for name, t, n in (("out.lens", out.lens, b), ("out.held", out.held, b), ("out.free_head", out.free_head, 1),
                           ("out.start", out.start, b + 1), ("out.position", out.position, max_tokens),
                           ("out.request", out.request, max_tokens)):
            _flat(name, t, i32, n)
        _flat("out.slot", out.slot, torch.int64, max_tokens)
    _check(lib.smp_block_plan(_at(lens), _at(add), _at(held), b, _at(free_blocks), free_blocks.shape[0],
                              _at(free_head), _at(block_table), block_table.shape[1], block_size, num_blocks,
                              max_tokens, _at(out.lens), _at(out.held), _at(out.free_head), _at(out.start),
                              _at(out.position), _at(out.request), _at(out.slot), _at(status), _queue(stream)))
    return out


def qk_norm_rope(q, k, positions, table=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out_q=None,
                 out_k=None, status=None, stream=None):
    """smp_qk_norm_rope.  q [T, Hq, D] and k [T, Hk, D] (or None), float32 or
    bfloat16, views of a fused projection allowed; positions: int32 [T];
    table: float32 [rows, rotary_dim] (rope_table), or None for the norm
    alone; weights: float32 [D] or None.  out_q, out_k: tensors to write (q
    and k themselves: in place), or None for new ones.  Returns (out_q,
    out_k)."""
    torch = _torch()
    lib = load()
    qs = _heads("q", q)
    t, hq, d = q.shape
    hk = ks = oks = 0
    out_q = torch.empty((t, hq, d), dtype=q.dtype, device=q.device) if out_q is None else out_q
    oqs = _heads("out_q", out_q, q.dtype, q.shape)
    if k is not None:
        hk = k.shape[1]
        ks = _heads("k", k, q.dtype, (t, hk, d))
        out_k = torch.empty((t, hk, d), dtype=q.dtype, device=q.device) if out_k is None else out_k
        oks = _heads("out_k", out_k, q.dtype, k.shape)
    _flat("positions", positions, torch.int32, t)
    rows = rotary = 0
    if table is not None:
        _flat("table", table, torch.float32, None, None)
        rows, rotary = table.shape
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _flat(name, w, torch.float32, d)
    _status(status)
    _check(lib.smp_qk_norm_rope(_at(q), _at(k), t, hq, hk, d, qs, ks, _code(q), _at(q_weight), _at(k_weight), eps,
                                _at(table), rows, rotary, int(interleaved), _at(positions), _at(out_q),
                                _at(out_k) if k is not None else None, oqs, oks, _at(status), _queue(stream)))
    return out_q, out_k


def cache_append(cache, k, v, slots, status=None, stream=None):
    """smp_cache_append: k and v [T, kv_heads, head_dim] (float32 or bfloat16)
    into the cache's slots (int64 [T], BlockPlan.slot)."""
    torch = _torch()
    lib = load()
    c = _cache_arg(cache)
    ks = _heads("k", k)
    t = k.shape[0]
    if tuple(k.shape) != (t, c.kv_heads, c.head_dim):
        raise SmpError("k must be [tokens, kv_heads, head_dim] of the cache")
    vs = _heads("v", v, k.dtype, k.shape)
    _flat("slots", slots, torch.int64, t)
    _status(status)
    _check(lib.smp_cache_append(ctypes.byref(c), _at(k), _at(v), t, ks, vs, _code(k), _at(slots), _at(status),
                                _queue(stream)))


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
    torch = _torch()
    lib = load()
    c = _cache_arg(cache)
    qs = _heads("q", q)
    t, h, d = q.shape
    if d != c.head_dim:
        raise SmpError("q must have the cache's head_dim")
    b = lens.shape[0]
    _flat("lens", lens, torch.int32, b)
    _flat("start", start, torch.int32, b + 1)
    _flat("block_table", block_table, torch.int32, b, None)
    out = torch.empty((t, h, d), dtype=q.dtype, device=q.device) if out is None else out
    os_ = _heads("out", out, q.dtype, q.shape)
    if lse is not None:
        _flat("lse", lse, torch.float32, t, h)
    if workspace is None:
        workspace = torch.empty(max(16, attention_workspace_bytes(t, h, c.kv_heads, d, b)), dtype=torch.uint8,
                                device=q.device)
    _flat("workspace", workspace, torch.uint8, None)
    _status(status)
    _check(lib.smp_cache_attention(ctypes.byref(c), _at(q), t, h, qs, _code(q), _at(start), _at(lens), b,
                                   _at(block_table), block_table.shape[1], d ** -0.5 if scale is None else scale,
                                   window, _at(out), os_, _at(lse), _at(status), _at(workspace), workspace.numel(),
                                   _queue(stream)))
    return out

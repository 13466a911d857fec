"""Binding of the operators around the paged FP8 KV cache (``include/nvfp4_attention.h``): block
tables and slot maps from request lengths, attention of prompts and single tokens over the cache, and
attention of trees of drafted tokens.

Argument marshalling only, like the rest of the binding: the HIP kernels of libnvfp4.so compute, on
the current stream of the tensors' device; PyTorch provides device memory.
"""

from __future__ import annotations

import ctypes
import functools
import operator

import bit_block_scaled_nvfp4_amd as _base

#: every symbol include/nvfp4_attention.h declares
ATTENTION_SYMBOLS = ("nvfp4_kv_block_tables", "nvfp4_kv_fp8_attention", "nvfp4_kv_fp8_tree_attention",
                     "nvfp4_kv_fp8_attention_workspace")

MAX_REQUESTS = 8192
MAX_TREE_WORDS = 64

_declared = None  # the library whose signatures are declared


def _lib():
    """The loaded library with the signatures of the attention operators declared (once)."""
    global _declared
    lib = _base.load_library()
    if _declared is lib:
        return lib
    declare(lib)
    _declared = lib
    return lib


def declare(lib: ctypes.CDLL) -> None:
    """Declare the C signatures of ``ATTENTION_SYMBOLS`` on ``lib``."""
    i64, vp, f32, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int
    lib.nvfp4_kv_block_tables.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp, i64, i64, vp, vp, i64, vp,
                                          vp, vp, vp]
    lib.nvfp4_kv_block_tables.restype = c_int
    head = [vp, c_int, i64, i64, i64, i64, i64, i64, vp, vp, vp, vp, i64, i64, vp, i64, i64, i64, i64,
            vp, vp, f32, f32, vp]
    tail = [i64, i64, vp, i64, i64, vp, i64, vp]
    lib.nvfp4_kv_fp8_attention.argtypes = head + [vp, vp] + tail
    lib.nvfp4_kv_fp8_attention.restype = c_int
    lib.nvfp4_kv_fp8_tree_attention.argtypes = head + [vp, i64, i64, vp] + tail
    lib.nvfp4_kv_fp8_tree_attention.restype = c_int
    lib.nvfp4_kv_fp8_attention_workspace.argtypes = [i64] * 7
    lib.nvfp4_kv_fp8_attention_workspace.restype = i64


def _vector(t, n, dtype, device, name):
    """``t`` must be a contiguous ``dtype`` vector of ``n`` elements on ``device``; returns its address."""
    if t.dtype is dtype and t.shape == (n,) and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must hold {n} contiguous values, got shape {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    return t.data_ptr()


def _row_pitch(t, name):
    """Elements from one row of the 2-D ``t`` to the next.  A dimension of one row has none that counts, and
    rows that share elements (an expanded row) have none that the library could take."""
    rows, width = t.shape
    if rows <= 1:
        return max(1, width)
    pitch = t.stride(0)
    if pitch < width:
        raise ValueError(f"{name} must have rows of their own (strides {list(t.stride())}, {width} a row): "
                         "an expanded or overlapping view needs .contiguous()")
    return max(1, pitch)


def _table(t, rows, device, name):
    torch = _base._torch()
    if t.dtype != torch.int32:
        raise ValueError(f"{name} must be int32, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != rows or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{rows}, width] with contiguous rows, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    return _row_pitch(t, name)


def _call(device, fn, *args):
    """Run one library call on ``device`` and its current stream, whichever device is current."""
    torch = _base._torch()
    # the stream's handle without a Stream object: 0.05 us instead of 1.8
    raw_stream, index = torch._C._cuda_getCurrentRawStream, device.index
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw_stream(index))
    if status:
        _base._check(status)


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    return t.device


def _refuse_overlaps(results, inputs, table):
    """Raise ValueError where a result or the table shares memory with another result or with an input.

    ``results``, ``inputs``: ``(name, address, bytes)``, address 0 without memory; ``table``: address, rows,
    bytes of a row and bytes from one row to the next (what lies between its rows is not its own)."""
    at, rows, width, pitch = table
    for i, (name, p, size) in enumerate(results):
        for other, q, n in (*results[:i], *inputs):
            if p and q and size and n and p < q + n and q < p + size:
                raise ValueError(f"{name} must not share memory with {other}")
    for name, p, size in (*results, *inputs):
        if p and at and size and rows * width and p < at + (rows - 1) * pitch + width and at < p + size:
            row, offset = divmod(max(p - at, 0), pitch)
            if offset < width or (row + 1 < rows and p + size > at + (row + 1) * pitch):
                raise ValueError(f"block_table must not share memory with {name}")


def nvfp4_kv_block_tables(context_lens, query_lens, free_blocks, block_table, block_size,
                          max_tokens=None, free_start=None, slot_mapping=None, positions=None,
                          query_start=None, seq_lens=None, blocks_needed=None):
    """Bookkeeping of one serving step, on the GPU, from request lengths alone.

    ``context_lens``, ``query_lens``: int32 ``[requests]``, tokens in the cache and new tokens of each
    request.  New blocks are taken in request order from ``free_blocks`` (int32), beginning at
    ``free_start`` (1-element int32; None: 0), and entered in ``block_table`` (int32 ``[requests,
    width]``, in place).  Returns ``(slot_mapping int64[max_tokens], positions int32[max_tokens],
    query_start int32[requests + 1], seq_lens int32[requests], blocks_needed int32[1])``; each may be
    given to be written in place, but shares no memory with another one, with ``block_table`` or with an
    input (``seq_lens`` of this step can be ``context_lens`` of the next, in a buffer of its own).  Tokens without a block, and padding up to ``max_tokens``, have slot
    -1, which :func:`nvfp4_kv_fp8_store` skips.  ``blocks_needed`` above the free blocks says that
    they did not suffice."""
    torch = _base._torch()
    lib = _lib()
    dev = _cuda(context_lens, "context_lens")
    i32, i64 = torch.int32, torch.int64
    if context_lens.dim() != 1 or free_blocks.dim() != 1:
        raise ValueError("context_lens and free_blocks must be 1-D")
    R = context_lens.shape[0]
    if R > MAX_REQUESTS:
        raise ValueError(f"at most {MAX_REQUESTS} requests, got {R}")
    block_size = int(block_size)
    if not 1 <= block_size <= 1 << 24:
        raise ValueError(f"block_size must lie in [1, 2^24], got {block_size}")
    c = _vector(context_lens, R, i32, dev, "context_lens")
    n = _vector(query_lens, R, i32, dev, "query_lens")
    F = free_blocks.shape[0]
    f = _vector(free_blocks, F, i32, dev, "free_blocks")
    fs = None if free_start is None else _vector(free_start, 1, i32, dev, "free_start")
    ld = _table(block_table, R, dev, "block_table")
    if max_tokens is None:
        if slot_mapping is None:
            raise ValueError("max_tokens or slot_mapping must be given")
        max_tokens = slot_mapping.shape[0]
    max_tokens = int(max_tokens)
    if max_tokens < 0:
        raise ValueError(f"max_tokens must not be negative, got {max_tokens}")
    if slot_mapping is None:
        slot_mapping = torch.empty(max_tokens, dtype=i64, device=dev)
    if positions is None:
        positions = torch.empty(max_tokens, dtype=i32, device=dev)
    if query_start is None:
        query_start = torch.empty(R + 1, dtype=i32, device=dev)
    if seq_lens is None:
        seq_lens = torch.empty(R, dtype=i32, device=dev)
    if blocks_needed is None:
        blocks_needed = torch.empty(1, dtype=i32, device=dev)
    table, W = block_table.data_ptr(), block_table.shape[1]
    sm = _vector(slot_mapping, max_tokens, i64, dev, "slot_mapping")
    ps = _vector(positions, max_tokens, i32, dev, "positions")
    qs = _vector(query_start, R + 1, i32, dev, "query_start")
    sl = _vector(seq_lens, R, i32, dev, "seq_lens")
    bn = _vector(blocks_needed, 1, i32, dev, "blocks_needed")
    # Workgroups read the lengths while others write results.  Ranges are disjoint if and only if, both in
    # rising order, each ends before the next begins; inputs that share memory, and what lies between a
    # table's rows, are sorted out afterwards.
    fs0, span = fs or 0, 4 * ((R - 1) * ld + W) if R * W else 0
    starts = sorted((c, n, f, fs0, table, sm, ps, qs, sl, bn))
    ends = sorted((c + 4 * R, n + 4 * R, f + 4 * F, fs0 + 4 if fs0 else 0, table + span, sm + 8 * max_tokens,
                   ps + 4 * max_tokens, qs + 4 * R + 4, sl + 4 * R, bn + 4))
    if any(map(operator.gt, ends, starts[1:])):
        _refuse_overlaps((("slot_mapping", sm, 8 * max_tokens), ("positions", ps, 4 * max_tokens),
                          ("query_start", qs, 4 * R + 4), ("seq_lens", sl, 4 * R), ("blocks_needed", bn, 4)),
                         (("context_lens", c, 4 * R), ("query_lens", n, 4 * R), ("free_blocks", f, 4 * F),
                          ("free_start", fs0, 4 if fs0 else 0)), (table, R, 4 * W, 4 * ld))
    _call(dev, lib.nvfp4_kv_block_tables, c, n, R, block_size, f, F, fs, table, W, ld, sm, ps, max_tokens, qs,
          sl, bn)
    return slot_mapping, positions, query_start, seq_lens, blocks_needed


def _rows(t, shape, dtype, device, name):
    """Check ``t [tokens, heads, head_dim]``; returns its token and head strides."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    ts, hs, ds = t.stride()
    if ds != 1 and t.numel() > 0:
        raise ValueError(f"{name} must have contiguous head vectors (stride(2) == 1)")
    # the stride of a dimension of one element addresses nothing
    return (ts if shape[0] > 1 else shape[1] * shape[2]), (hs if shape[1] > 1 else shape[2])


def _refuse_overlap_of_rows(q, q_strides, out, out_strides):
    """Raise ValueError where ``out [tokens, heads, head_dim]`` shares elements with ``q`` and is not ``q`` itself (the
    same elements in the same places: an item's rows are read before they are written)."""
    T, H, D = q.shape
    if T == 0:
        return
    ahead, size = out.data_ptr() - q.data_ptr(), q.element_size()
    spans = [(T - 1) * ts + (H - 1) * hs + D for ts, hs in (q_strides, out_strides)]
    if ahead >= spans[0] * size or -ahead >= spans[1] * size or (ahead == 0 and q_strides == out_strides):
        return
    if ahead % size == 0:
        # windows side by side in rows of one pitch (a fused row; head-major storage: heads for tokens)
        for pitch, inner, n in ((q_strides[0], 1, H), (q_strides[1], 0, T)):
            if pitch and pitch == out_strides[1 - inner]:
                widths = [(n - 1) * s[inner] + D for s in (q_strides, out_strides)]
                begin = (ahead // size) % pitch
                if max(widths) <= pitch and begin >= widths[0] and begin + widths[1] <= pitch:
                    return
        torch = _base._torch()
        t, h = torch.arange(T, device="cpu")[:, None], torch.arange(H, device="cpu")[None, :]
        mine = torch.unique(t * q_strides[0] + h * q_strides[1])
        at = ahead // size + (t * out_strides[0] + h * out_strides[1]).flatten()
        place = torch.searchsorted(mine, at)  # the vectors of q before and behind each one of out
        before, behind = mine[(place - 1).clamp(min=0)], mine[place.clamp(max=len(mine) - 1)]
        if not bool((((at - before).abs() < D) | ((at - behind).abs() < D)).any()):
            return
    raise ValueError("out must be q itself or share no memory with it")


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(*sizes):
    """Workspace of a call of these sizes (a function of them alone)."""
    return _lib().nvfp4_kv_fp8_attention_workspace(*sizes)


def _attention(fn_name, q, key_cache, value_cache, key_scale, value_scale, block_table, query_start,
               seq_lens, block_size, num_kv_heads, scale, softcap, slopes, extra, max_query_len,
               max_seq_len, out):
    torch = _base._torch()
    lib = _lib()
    dev = _cuda(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be 3-D [tokens, heads, head_dim]")
    if q.dtype != torch.bfloat16 and q.dtype != torch.float16:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    T, H, D = q.shape
    if D != 64 and D != 128 and D != 256:
        raise ValueError(f"head_dim must be 64, 128 or 256, got {D}")
    num_kv_heads = int(num_kv_heads)
    if num_kv_heads < 1 or H < 1 or H > 1024 or H % num_kv_heads:
        raise ValueError(f"{H} heads (1 to 1024) must be a multiple of {num_kv_heads} KV heads")
    block_size = int(block_size)
    if not 1 <= block_size <= 1 << 24:
        raise ValueError(f"block_size must lie in [1, 2^24], got {block_size}")
    q_ts, q_hs = _rows(q, (T, H, D), q.dtype, dev, "q")
    width = num_kv_heads * D
    for c, name in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        if c.dtype != torch.uint8 or c.dim() != 2 or c.shape[1] < width or c.stride(1) != 1:
            raise ValueError(f"{name} must be uint8 [num_slots, >= {width}] with contiguous rows")
        if c.device != dev:
            raise ValueError(f"{name} must live on {dev}, got {c.device}")
    if value_cache.shape[0] != key_cache.shape[0] or (key_cache.shape[0] > 1 and value_cache.stride(0) != key_cache.stride(0)):
        raise ValueError("value_cache must have key_cache's slots and row pitch")
    slots = key_cache.shape[0]
    cache_ld = key_cache.stride(0) if slots > 1 else max(width, key_cache.shape[1] // 16 * 16)
    for s, name in ((key_scale, "key_scale"), (value_scale, "value_scale")):
        if s.dtype != torch.float32 or s.numel() != 1 or s.device != dev:
            raise ValueError(f"{name} must be one float32 value on {dev}")
    if seq_lens.dim() != 1:
        raise ValueError("seq_lens must be 1-D")
    R = seq_lens.shape[0]
    if R > MAX_REQUESTS:
        raise ValueError(f"at most {MAX_REQUESTS} requests, got {R}")
    table_ld = _table(block_table, R, dev, "block_table")
    qs = _vector(query_start, R + 1, torch.int32, dev, "query_start")
    sl = _vector(seq_lens, R, torch.int32, dev, "seq_lens")
    sp = None if slopes is None else _vector(slopes, H, torch.float32, dev, "slopes")
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=dev)
        out_ts, out_hs = H * D, D
    else:
        out_ts, out_hs = _rows(out, (T, H, D), q.dtype, dev, "out")
        _refuse_overlap_of_rows(q, (q_ts, q_hs), out, (out_ts, out_hs))
    W = block_table.shape[1]
    # without a word from the caller: every request has one token at least
    max_query_len = max(1, T - R + 1 if max_query_len is None else int(max_query_len))
    max_seq_len = max(1, min(W * block_size, 2**31 - 1) if max_seq_len is None else int(max_seq_len))
    need = _workspace_bytes(T, H, num_kv_heads, D, R, max_query_len, max_seq_len)
    # from the caching allocator on the current stream: no two calls that may run at once share one
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, getattr(lib, fn_name), q.data_ptr(), _base.NVFP4_BF16 if q.dtype == torch.bfloat16 else _base.NVFP4_F16,
          T, H, num_kv_heads, D, q_ts, q_hs, key_cache.data_ptr(), value_cache.data_ptr(),
          key_scale.data_ptr(), value_scale.data_ptr(), slots, cache_ld, block_table.data_ptr(), R, W,
          table_ld, block_size, qs, sl, D ** -0.5 if scale is None else float(scale), float(softcap), sp,
          *extra(T, R, dev), max_query_len, max_seq_len, out.data_ptr(), out_ts, out_hs,
          None if ws is None else ws.data_ptr(), need)
    return out


def nvfp4_kv_fp8_attention(q, key_cache, value_cache, key_scale, value_scale, block_table, query_start,
                           seq_lens, *, block_size, num_kv_heads, scale=None, softcap=0.0, slopes=None,
                           doc_start=None, prefix_lens=None, max_query_len=None, max_seq_len=None,
                           out=None):
    """Attention of each request's new tokens (whole prompts, chunks, single tokens) over the paged FP8
    cache that :func:`nvfp4_kv_fp8_store` fills.

    ``q``: bfloat16 or float16 ``[tokens, heads, head_dim]`` (head_dim 64, 128 or 256), any token and
    head strides.  Request r's queries are rows ``query_start[r]`` to ``query_start[r + 1]`` and the last
    positions of its ``seq_lens[r]``, whose rows the cache already holds; ``block_table`` says where.
    Causal; ``softcap`` > 0 caps scores by ``softcap * tanh(x / softcap)``, ``slopes`` (float32
    ``[heads]``) adds ``slope * (key position - query position)``, ``doc_start`` (int32 ``[tokens]``)
    hides the positions before each token's document, ``prefix_lens`` (int32 ``[requests]``) shows the
    positions below it ahead of the causal order too: by itself, each request's prefix to all its tokens;
    with ``doc_start``, what of it does not lie before the token's document, so that the two belong together
    where the prefix ends within the first document (one that reaches further shows a document's tokens the
    beginning of the next one, and none is shared by all documents).  Rows that see nothing are zero; rows of no request are left as
    they were.  ``max_query_len`` and ``max_seq_len`` (bounds of the requests' lengths) only choose how
    the work is divided.  Single tokens in a call with prompts cost as much as 256 rows each over their
    context: many of them over long contexts are faster in a call of their own.  Returns ``out`` in q's
    type (given, it is ``q`` itself or shares no memory with it)."""
    torch = _base._torch()

    def extra(T, R, dev):
        return (None if doc_start is None else _vector(doc_start, T, torch.int32, dev, "doc_start"),
                None if prefix_lens is None else _vector(prefix_lens, R, torch.int32, dev, "prefix_lens"))

    return _attention("nvfp4_kv_fp8_attention", q, key_cache, value_cache, key_scale, value_scale,
                      block_table, query_start, seq_lens, block_size, num_kv_heads, scale, softcap,
                      slopes, extra, max_query_len, max_seq_len, out)


def nvfp4_kv_fp8_tree_attention(q, key_cache, value_cache, key_scale, value_scale, block_table,
                                query_start, seq_lens, tree_mask, *, block_size, num_kv_heads, scale=None,
                                softcap=0.0, slopes=None, positions=None, max_query_len=None,
                                max_seq_len=None, out=None):
    """Attention of trees of drafted tokens over the paged FP8 cache.  Request r's n query rows are
    drafted tokens stored at its last n positions; each sees the whole context before them, and the
    drafted tokens whose bits are set in its row of ``tree_mask`` (int64 ``[tokens, words]``, bit d % 64
    of word d // 64 for drafted token d, its own bit included).  ``positions`` (int32 ``[tokens]``) are
    the positions that drafted tokens count at in the distance bias (default: context + index).  Other
    arguments as :func:`nvfp4_kv_fp8_attention`."""
    torch = _base._torch()

    def extra(T, R, dev):
        if tree_mask.dtype != torch.int64 or tree_mask.dim() != 2 or tree_mask.shape[0] != T:
            raise ValueError(f"tree_mask must be int64 [{T}, words]")
        words = tree_mask.shape[1]
        if not 1 <= words <= MAX_TREE_WORDS or (words > 1 and tree_mask.stride(1) != 1):
            raise ValueError(f"tree_mask must have 1 to {MAX_TREE_WORDS} contiguous words a row")
        if tree_mask.device != dev:
            raise ValueError(f"tree_mask must live on {dev}, got {tree_mask.device}")
        return (tree_mask.data_ptr(), words, _row_pitch(tree_mask, "tree_mask"),
                None if positions is None else _vector(positions, T, torch.int32, dev, "positions"))

    return _attention("nvfp4_kv_fp8_tree_attention", q, key_cache, value_cache, key_scale, value_scale,
                      block_table, query_start, seq_lens, block_size, num_kv_heads, scale, softcap,
                      slopes, extra, max_query_len, max_seq_len, out)

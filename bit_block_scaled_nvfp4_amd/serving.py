"""Binding of the other operators of a serving step (``include/nvfp4_serving.h``): norms and position
rotation of queries and keys, appending keys and values to the paged caches, attention over the 4-bit cache,
and verification of drafted tokens.

Argument marshalling only, like the rest of the binding: the HIP kernels of libnvfp4.so compute, on
the current stream of the tensors' device; PyTorch provides device memory.
"""

from __future__ import annotations

import ctypes
import functools
import operator

import bit_block_scaled_nvfp4_amd as _base

from .attention import (
    MAX_REQUESTS,
    _call,
    _cuda,
    _refuse_overlap_of_rows,
    _rows,
    _table,
    _tree_arguments,
    _vector,
)

#: every symbol include/nvfp4_serving.h declares
SERVING_SYMBOLS = ("nvfp4_qk_norm_rope", "nvfp4_kv_fp8_append", "nvfp4_kv_fp4_append", "nvfp4_kv_fp4_load",
                   "nvfp4_kv_fp4_attention", "nvfp4_kv_fp4_tree_attention", "nvfp4_kv_fp4_attention_workspace",
                   "nvfp4_verify_drafted", "nvfp4_verify_drafted_workspace")

MAX_HEAD_DIM = 512

_declared = None  # the library whose signatures are declared


def _lib():
    """The loaded library with the signatures of the serving operators declared (once)."""
    global _declared
    lib = _base.load_library()
    if _declared is lib:
        return lib
    declare(lib)
    _declared = lib
    return lib


def declare(lib: ctypes.CDLL) -> None:
    """Declare the C signatures of ``SERVING_SYMBOLS`` on ``lib``."""
    i64, vp, f32, f64, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double, ctypes.c_int
    turn = [vp, vp, i64, c_int]
    lib.nvfp4_qk_norm_rope.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64, c_int, i64, i64, *turn, vp, vp, c_int,
                                       f64, f64, vp, i64, i64, vp, i64, i64, vp]
    lib.nvfp4_qk_norm_rope.restype = c_int
    head = [vp, vp, c_int, i64, i64, i64, i64, i64, i64, i64, *turn, vp, c_int, f64, f64, vp, vp, vp]
    lib.nvfp4_kv_fp8_append.argtypes = head + [vp, vp, i64, i64, vp]
    lib.nvfp4_kv_fp8_append.restype = c_int
    lib.nvfp4_kv_fp4_append.argtypes = head + [vp, vp, vp, vp, i64, i64, vp]
    lib.nvfp4_kv_fp4_append.restype = c_int
    lib.nvfp4_kv_fp4_load.argtypes = [vp, vp, i64, i64, i64, i64, vp, vp, i64, vp, c_int, vp]
    lib.nvfp4_kv_fp4_load.restype = c_int
    head = [vp, c_int, i64, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, i64, i64, vp, i64, i64, i64, vp, vp, f32,
            f32, vp]
    tail = [i64, i64, vp, i64, i64, vp, i64, vp]
    lib.nvfp4_kv_fp4_attention.argtypes = head + [vp, vp] + tail
    lib.nvfp4_kv_fp4_attention.restype = c_int
    lib.nvfp4_kv_fp4_tree_attention.argtypes = head + [vp, i64, i64, vp] + tail
    lib.nvfp4_kv_fp4_tree_attention.restype = c_int
    lib.nvfp4_kv_fp4_attention_workspace.argtypes = [i64] * 7
    lib.nvfp4_kv_fp4_attention_workspace.restype = i64
    lib.nvfp4_verify_drafted.argtypes = [vp, i64, vp, i64, i64, i64, vp, vp, i64, vp, vp, vp, vp, vp, i64, vp]
    lib.nvfp4_verify_drafted.restype = c_int
    lib.nvfp4_verify_drafted_workspace.argtypes = [i64, i64]
    lib.nvfp4_verify_drafted_workspace.restype = i64


# ---- head vectors -----------------------------------------------------------------------------


def _strides(t, shape, dtype, device, name):
    """Check ``t [tokens, heads, head_dim]``; returns its token and head strides."""
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head_dim], got {list(shape)}")
    if t.shape == shape and t.dtype is dtype and t.device == device:
        ts, hs, one = t.stride()
        if one == 1:
            T, H, D = shape
            # (the stride of a dimension of one element addresses nothing)
            return (ts if T > 1 else H * D, hs if H > 1 else D)
    elif t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head_dim], got {list(t.shape)}")
    return _rows(t, tuple(shape), dtype, device, name)


def _meet(a, b):
    """Whether two sets of vectors ``(address, tokens, heads, bytes of a vector, token stride, head stride)`` (bytes)
    share memory."""
    (p, T, H, w, ts, hs), (q, U, G, x, us, gs) = a, b
    if not (T and H and w and U and G and x):
        return False
    ends = p + (T - 1) * ts + (H - 1) * hs + w, q + (U - 1) * us + (G - 1) * gs + x
    if q >= ends[0] or p >= ends[1]:
        return False
    # windows side by side in rows of one pitch: a fused row, or head-major storage
    for pitch, n, inner, m, other, same in ((ts, H, hs, G, gs, ts == us), (hs, T, ts, U, us, hs == gs)):
        if pitch and same:
            wide, far = (n - 1) * inner + w, (m - 1) * other + x
            begin = (q - p) % pitch
            if max(wide, far) <= pitch and begin >= wide and begin + far <= pitch:
                return False
    torch = _base._torch()
    upto = functools.partial(torch.arange, device="cpu")
    mine = torch.unique((p + upto(T)[:, None] * ts + upto(H)[None, :] * hs).flatten())
    its = (q + upto(U)[:, None] * us + upto(G)[None, :] * gs).flatten()
    place = torch.searchsorted(mine, its)  # the vectors before and behind each one
    before, behind = mine[(place - 1).clamp(min=0)], mine[place.clamp(max=len(mine) - 1)]
    return bool((((its >= before) & (its < before + w)) | ((behind >= its) & (behind < its + x))
                 | ((its >= behind) & (its < behind + w))).any())


def _turn(positions, inv_freq, tokens, head_dim, device, interleaved, step, torch):
    """Arguments of the rotation: positions, frequencies, their number, the flag."""
    if interleaved is not False and interleaved is not True:
        if interleaved not in (0, 1):
            raise ValueError(f"interleaved must be True or False, got {interleaved!r}")
        interleaved = int(interleaved)
    if positions is None or inv_freq is None:
        if positions is not None or inv_freq is not None:
            raise ValueError("positions and inv_freq come together")
        return None, None, 0, interleaved
    shape = inv_freq.shape
    if len(shape) != 1 or shape[0] % step or 2 * shape[0] > head_dim:
        raise ValueError(f"inv_freq must hold a multiple of {step} values, at most {head_dim // 2}, got shape {list(shape)}")
    n = shape[0]
    return (_vector(positions, tokens, torch.int32, device, "positions"),
            _vector(inv_freq, n, torch.float32, device, "inv_freq"), n, interleaved)


def _weight(t, head_dim, device, name):
    """Address and type of a norm's weight (None: no norm)."""
    if t is None:
        return None, _base.NVFP4_F32
    return _vector(t, head_dim, t.dtype, device, name), _base._dtype_code(t.dtype)


def _extent(shape, strides, size):
    """Bytes from the first to past the last element of head vectors."""
    T, H, D = shape
    return size * ((T - 1) * strides[0] + (H - 1) * strides[1] + D) if T and H else 0


def nvfp4_qk_norm_rope(q, k=None, positions=None, inv_freq=None, *, q_weight=None, k_weight=None, eps=1e-6,
                       weight_offset=0.0, interleaved=False, q_out=None, k_out=None):
    """Norm and position rotation of the head vectors of queries and keys, in one pass.

    ``q``, ``k`` (or None): float32, bfloat16 or float16 ``[tokens, heads, head_dim]`` (heads of their own; head_dim a
    multiple of 16 up to 512), any token and head strides of whole 16 bytes: views of a fused row will do.
    ``q_weight``, ``k_weight`` (``[head_dim]``, one type): ``x / sqrt(mean(x^2) + eps) * (weight_offset + weight)``; None:
    no norm.  ``positions`` (int32 ``[tokens]``) and ``inv_freq`` (float32, a multiple of 8 values up to head_dim / 2):
    element i and its partner (``len(inv_freq)`` further on, or with ``interleaved`` the neighbour) are rotated by
    ``position * inv_freq[i]``; None: no rotation.  Formed in binary64 and rounded once.  Returns ``(q_out, k_out)`` in
    the inputs' type; each may be given, and be its own input (in place)."""
    torch = _base._torch()
    lib = _lib()
    dev, shape, dtype = _cuda(q, "q"), q.shape, q.dtype
    q_strides = _strides(q, shape, dtype, dev, "q")
    T, H, D = shape
    if H < 1 or H > 1024:
        raise ValueError(f"q must have 1 to 1024 heads, got {H}")
    if D % 16 or not 16 <= D <= MAX_HEAD_DIM:
        raise ValueError(f"head_dim must be a multiple of 16 up to {MAX_HEAD_DIM}, got {D}")
    code = _base._dtype_code(dtype)
    p, f, n, pairs = _turn(positions, inv_freq, T, D, dev, interleaved, 8, torch)
    qw, wt = _weight(q_weight, D, dev, "q_weight")
    kw, kt = _weight(k_weight, D, dev, "k_weight")
    if q_weight is None:
        wt = kt
    elif k_weight is not None and kt != wt:
        raise ValueError("q_weight and k_weight must have one type")
    qp, size = q.data_ptr(), 4 if code == _base.NVFP4_F32 else 2
    kp, ko, Hk, k_strides, ko_strides, ko_end, k_end = None, None, 0, (0, 0), (0, 0), 0, 0
    if k is not None:
        k_shape = k.shape
        if len(k_shape) != 3 or k_shape[0] != T or k_shape[2] != D or k_shape[1] > 1024:
            raise ValueError(f"k must have shape [{T}, heads up to 1024, {D}], got {list(k_shape)}")
        Hk = k_shape[1]
        k_strides = _strides(k, k_shape, dtype, dev, "k")
        kp = k.data_ptr()
        if k_out is None:
            k_out, ko_strides = torch.empty(k_shape, dtype=dtype, device=dev), (Hk * D, D)
            ko = k_out.data_ptr()
        else:
            ko_strides = _strides(k_out, k_shape, dtype, dev, "k_out")
            ko = k_out.data_ptr()
            ko_end = ko + _extent(k_shape, ko_strides, size)
        k_end = kp + _extent(k_shape, k_strides, size)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight come with k")
    q_end = qp + _extent(shape, q_strides, size)
    if q_out is None:
        q_out, qo_strides = torch.empty(shape, dtype=dtype, device=dev), (H * D, D)
        qo, qo_end = q_out.data_ptr(), 0
    else:
        qo_strides = _strides(q_out, shape, dtype, dev, "q_out")
        qo = q_out.data_ptr()
        qo_end = qo + _extent(shape, qo_strides, size)
    # (an output made here has no end: it meets nothing)
    if ((qo < q_end and qp < qo_end) or (ko_end and (kp < ko_end and ko < k_end or qp < ko_end and ko < q_end or ko < qo_end and qo < ko_end))
            or (kp is not None and kp < qo_end and qo < k_end)):
        _refuse_meeting(q, q_strides, k, k_strides, q_out if qo_end else None, qo_strides, k_out if ko_end else None, ko_strides)
    _call(dev, lib.nvfp4_qk_norm_rope, qp, H, *q_strides, kp, Hk, *k_strides, code, T, D, p, f, n, pairs, qw, kw, wt, float(eps),
          float(weight_offset), qo, *qo_strides, ko, *ko_strides)
    return q_out, k_out


def _refuse_meeting(q, q_strides, k, k_strides, q_out, qo_strides, k_out, ko_strides):
    """Raise ValueError where a given output shares memory with another one or with an input that is not itself."""
    given = [(x, s, name, mine) for x, s, name, mine in ((q, q_strides, "q", 0), (k, k_strides, "k", 1),
                                                         (q_out, qo_strides, "q_out", 0), (k_out, ko_strides, "k_out", 1))
             if x is not None]
    as_bytes = [(x.data_ptr(), *x.shape[:2], x.shape[2] * x.element_size(), *(n * x.element_size() for n in s))
                for x, s, _, _ in given]
    for i, (x, s, name, mine) in enumerate(given):
        if name not in ("q_out", "k_out"):
            continue
        for j, (y, t, other, its) in enumerate(given):
            if j >= i or (other in ("q", "k") and its == mine and x.data_ptr() == y.data_ptr() and s == t):
                continue  # (pairs of outputs once; in place)
            if _meet(as_bytes[i], as_bytes[j]):
                raise ValueError(f"{name} must share no memory with {other}"
                                 + (", or be it" if other in ("q", "k") and its == mine else ""))


# ---- appending --------------------------------------------------------------------------------


def _refuse_ranges(outs, ins):
    """Raise ValueError where a byte range ``(name, begin, end)`` of ``outs`` meets another one or one of ``ins``."""
    ins = list(ins)
    for i, (name, p, e) in enumerate(outs):
        for other, q, f in (*outs[:i], *ins):
            if p < f and q < e and e > p and f > q:
                raise ValueError(f"{name} must not share memory with {other}")


def _append(key, value, positions, inv_freq, k_scale, v_scale, scale_names, slots, k_weight, eps, weight_offset,
            interleaved, step, torch):
    """What both appends check; returns the common arguments, the device, sizes and the byte ranges read."""
    dev, shape, dtype = _cuda(key, "key"), key.shape, key.dtype
    k_strides = _strides(key, shape, dtype, dev, "key")
    T, Hk, D = shape
    if Hk < 1 or Hk > 1024:
        raise ValueError(f"key must have 1 to 1024 heads, got {Hk}")
    if D != 64 and D != 128 and D != 256:
        raise ValueError(f"head_dim must be 64, 128 or 256, got {D}")
    code = _base._dtype_code(dtype)
    v_strides = _strides(value, shape, dtype, dev, "value")
    p, f, n, pairs = _turn(positions, inv_freq, T, D, dev, interleaved, step, torch)
    kw, wt = _weight(k_weight, D, dev, "k_weight")
    for s, name in ((k_scale, scale_names[0]), (v_scale, scale_names[1])):
        if s.dtype is not torch.float32 or s.numel() != 1 or s.device != dev:
            raise ValueError(f"{name} must be one float32 value on {dev}")
    sm = None if slots is None else _vector(slots, T, torch.int64, dev, "slot_mapping")
    k, v, size = key.data_ptr(), value.data_ptr(), 4 if code == _base.NVFP4_F32 else 2
    args = (k, v, code, T, Hk, D, *k_strides, *v_strides, p, f, n, pairs, kw, wt, float(eps), float(weight_offset),
            k_scale.data_ptr(), v_scale.data_ptr(), sm)
    ke, ve = k + _extent(shape, k_strides, size), v + _extent(shape, v_strides, size)
    if k < ve and v < ke:  # (of one fused row: one range)
        k, ke = min(k, v), max(ke, ve)
        v = ve = k
    return args, dev, (T, Hk, D), (k, v, sm or 0), (ke, ve, sm + 8 * T if sm else 0)


def nvfp4_kv_fp8_append(key, value, positions, inv_freq, key_scale, value_scale, key_cache, value_cache,
                        slot_mapping=None, *, k_weight=None, eps=1e-6, weight_offset=0.0, interleaved=False):
    """Norm and rotate the new tokens' keys and write keys and values into the FP8 cache: bit for bit what
    :func:`nvfp4_qk_norm_rope` of the keys and then :func:`nvfp4_kv_fp8_store` give, in one pass.

    ``key``, ``value``: ``[tokens, kv_heads, head_dim]`` (head_dim 64, 128 or 256) as :func:`nvfp4_qk_norm_rope`'s; the
    rotation and the norm of the keys as there (``positions`` and ``inv_freq`` None: no rotation).  Scales, caches
    ``[num_slots, >= kv_heads * head_dim]`` and ``slot_mapping`` as :func:`nvfp4_kv_fp8_store`; a cache shares no memory
    with an input or the other cache."""
    torch = _base._torch()
    lib = _lib()
    args, dev, (T, Hk, D), begin, end = _append(key, value, positions, inv_freq, key_scale, value_scale,
                                                ("key_scale", "value_scale"), slot_mapping, k_weight, eps, weight_offset,
                                                interleaved, 8, torch)
    width, shape, strides = Hk * D, key_cache.shape, key_cache.stride()
    for c, name in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        if c.dtype is not torch.uint8 or c.dim() != 2 or c.shape[1] < width or c.stride(1) != 1:
            raise ValueError(f"{name} must be uint8 [num_slots, >= {width}] with contiguous rows")
        if c.device != dev:
            raise ValueError(f"{name} must live on {dev}, got {c.device}")
    slots = shape[0]
    if value_cache.shape[0] != slots or (slots > 1 and value_cache.stride(0) != strides[0]):
        raise ValueError("value_cache must have key_cache's slots and row pitch")
    ld = strides[0] if slots > 1 else max(width, shape[1] // 16 * 16)
    if ld < width:
        raise ValueError(f"caches must have rows of their own (row pitch {ld}, {width} a row): no expanded or overlapping views")
    kp, vp = key_cache.data_ptr(), value_cache.data_ptr()
    extent = (slots - 1) * ld + width if slots else 0
    if kp < vp + extent and vp < kp + extent and not width <= (vp - kp) % ld <= ld - width:
        raise ValueError("value_cache must not share memory with key_cache")
    for i, e in zip(begin, end):
        if kp < e and i < kp + extent or vp < e and i < vp + extent:
            _refuse_ranges([("key_cache", kp, kp + extent)], [("key, value or slot_mapping", i, e)])
            _refuse_ranges([("value_cache", vp, vp + extent)], [("key, value or slot_mapping", i, e)])
    _call(dev, lib.nvfp4_kv_fp8_append, *args, kp, vp, slots, ld)


def _cache4(codes, scales, dev, names, torch, like=None):
    """Check one tensor of the 4-bit cache and its scales; returns ``(num_blocks, kv_heads, block_size, head_dim)``.
    ``like``: what this gave for the keys."""
    u8, shape = torch.uint8, codes.shape
    if not (codes.dtype is u8 and scales.dtype is u8 and len(shape) == 4 and codes.device == dev and scales.device == dev
            and codes.is_contiguous() and scales.is_contiguous()):
        for t, name in ((codes, names[0]), (scales, names[1])):
            if t.dtype != u8 or t.dim() != 4:
                raise ValueError(f"{name} must be uint8 [num_blocks, kv_heads, block_size, ...], got {t.dtype} {list(t.shape)}")
            if t.device != dev:
                raise ValueError(f"{name} must live on {dev}, got {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    B, Hk, bs, half = shape
    if scales.shape != (B, Hk, bs, half // 8) or half % 8:
        raise ValueError(f"{names[1]} must have shape {[B, Hk, bs, half // 8]}, got {list(scales.shape)}")
    got = (B, Hk, bs, 2 * half)
    if like is None:
        if half not in (32, 64, 128):
            raise ValueError(f"head_dim must be 64, 128 or 256, got {2 * half}")
        if Hk < 1 or not 1 <= bs <= 1 << 24 or B * Hk * bs >= 2 ** 31:
            raise ValueError(f"{names[0]} must have KV heads, blocks of 1 to 2^24 slots and fewer than 2^31 rows")
    elif got != like:
        raise ValueError(f"{names[0]} must have the keys' shape")
    return got


def nvfp4_kv_fp4_append(key, value, positions, inv_freq, key_gscale, value_gscale, key_codes, key_scales, value_codes,
                        value_scales, slot_mapping=None, *, k_weight=None, eps=1e-6, weight_offset=0.0,
                        interleaved=False):
    """Norm and rotate the new tokens' keys and write keys and values into the 4-bit cache, each head's row encoded as
    NVFP4 under the static scale ``key_gscale`` or ``value_gscale`` (the block scale's factor is ``g * fl(1/6)``, not the
    ``g / 6`` of :func:`nvfp4_quantize`, a neighbour at most: maxima in the middle between two scales may take the other; the same
    where ``g`` is six times a float32 number).

    Codes: uint8 ``[num_blocks, kv_heads, block_size, head_dim / 2]``, scales: uint8 ``[..., head_dim / 16]``, contiguous.
    ``slot_mapping`` (int64 ``[tokens]``; None: token t in slot t) counts ``block * block_size + place``, as
    :func:`nvfp4_kv_block_tables` gives it; slots outside the cache are skipped.  Without ``interleaved``, ``inv_freq``
    holds a multiple of 16 values.  Other arguments as :func:`nvfp4_kv_fp8_append`."""
    torch = _base._torch()
    lib = _lib()
    args, dev, (T, Hk, D), begin, end = _append(key, value, positions, inv_freq, key_gscale, value_gscale,
                                                ("key_gscale", "value_gscale"), slot_mapping, k_weight, eps, weight_offset,
                                                interleaved, 8 if interleaved else 16, torch)
    shape = _cache4(key_codes, key_scales, dev, ("key_codes", "key_scales"), torch)
    _cache4(value_codes, value_scales, dev, ("value_codes", "value_scales"), torch, shape)
    B, heads, bs, dim = shape
    if heads != Hk or dim != D:
        raise ValueError(f"the cache holds {heads} heads of {dim}, keys have {Hk} of {D}")
    at = key_codes.data_ptr(), key_scales.data_ptr(), value_codes.data_ptr(), value_scales.data_ptr()
    n = B * Hk * bs * (D // 16)
    # ranges are disjoint if and only if, both in rising order, each ends before the next begins
    starts, ends = sorted((*at, *begin)), sorted((at[0] + 8 * n, at[1] + n, at[2] + 8 * n, at[3] + n, *end))
    if any(map(operator.gt, ends, starts[1:])):
        _refuse_ranges([(name, p, p + m) for name, p, m in zip(
            ("key_codes", "key_scales", "value_codes", "value_scales"), at, (8 * n, n, 8 * n, n))],
            [("key, value or slot_mapping", i, e) for i, e in zip(begin, end)])
    _call(dev, lib.nvfp4_kv_fp4_append, *args, *at, B, bs)


def nvfp4_kv_fp4_load(codes, scales, gscale, slot_mapping=None, out_dtype=None, out=None):
    """Gather slots of the 4-bit cache (keys or values) and decode them: ``[tokens, kv_heads, head_dim]`` float32
    (default) or bfloat16.  ``slot_mapping``: int64 ``[tokens]`` (None: every slot in order); slots outside the cache give
    zeros."""
    torch = _base._torch()
    lib = _lib()
    dev = _cuda(codes, "codes")
    B, Hk, bs, D = _cache4(codes, scales, dev, ("codes", "scales"), torch)
    if gscale.dtype != torch.float32 or gscale.numel() != 1 or gscale.device != dev:
        raise ValueError(f"gscale must be one float32 value on {dev}")
    T = B * bs
    sm = None
    if slot_mapping is not None:
        if slot_mapping.dim() != 1:
            raise ValueError("slot_mapping must be 1-D")
        T = slot_mapping.shape[0]
        sm = _vector(slot_mapping, T, torch.int64, dev, "slot_mapping")
    if out is None:
        out_dtype = out_dtype or torch.float32
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("out_dtype must be float32 or bfloat16")
        out = torch.empty((T, Hk, D), dtype=out_dtype, device=dev)
    else:
        if out.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"out must be float32 or bfloat16, got {out.dtype}")
        if out.shape != (T, Hk, D) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous [{T}, {Hk}, {D}], got {list(out.shape)}")
        if out.device != dev:
            raise ValueError(f"out must live on {dev}, got {out.device}")
        o, c, s, n, m = out.data_ptr(), codes.data_ptr(), scales.data_ptr(), B * Hk * bs * (D // 16), sm or 0
        end = o + T * Hk * D * (4 if out.dtype is torch.float32 else 2)
        if o < c + 8 * n and c < end or o < s + n and s < end or o < m + 8 * T and m < end:
            _refuse_ranges([("out", o, end)], [("codes", c, c + 8 * n), ("scales", s, s + n), ("slot_mapping", m, m + 8 * T if m else 0)])
    _call(dev, lib.nvfp4_kv_fp4_load, codes.data_ptr(), scales.data_ptr(), B, Hk, bs, D, gscale.data_ptr(), sm, T,
          out.data_ptr(), _base._dtype_code(out.dtype))
    return out


# ---- attention over the 4-bit cache -----------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(*sizes):
    """Workspace of a call of these sizes (a function of them alone)."""
    return _lib().nvfp4_kv_fp4_attention_workspace(*sizes)


def _attention(fn, q, key_codes, key_scales, value_codes, value_scales, key_gscale, value_gscale, block_table,
               query_start, seq_lens, scale, softcap, slopes, extra, max_query_len, max_seq_len, out):
    torch = _base._torch()
    dev = _cuda(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be 3-D [tokens, heads, head_dim]")
    dtype = q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise ValueError(f"q must be bfloat16 or float16, got {dtype}")
    T, H, D = q.shape
    shape = _cache4(key_codes, key_scales, dev, ("key_codes", "key_scales"), torch)
    _cache4(value_codes, value_scales, dev, ("value_codes", "value_scales"), torch, shape)
    B, Hk, bs, dim = shape
    if dim != D:
        raise ValueError(f"the cache holds heads of {dim}, q has {D}")
    if H < 1 or H > 1024 or H % Hk:
        raise ValueError(f"{H} heads (1 to 1024) must be a multiple of {Hk} KV heads")
    q_ts, q_hs = _strides(q, q.shape, dtype, dev, "q")
    for s, name in ((key_gscale, "key_gscale"), (value_gscale, "value_gscale")):
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
    max_seq_len = max(1, min(W * bs, 2**31 - 1) if max_seq_len is None else int(max_seq_len))
    need = _workspace_bytes(T, H, Hk, D, R, max_query_len, max_seq_len)
    # from the caching allocator on the current stream: no two calls that may run at once share one
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, fn, q.data_ptr(), _base.NVFP4_BF16 if dtype is torch.bfloat16 else _base.NVFP4_F16,
          T, H, Hk, D, q_ts, q_hs, key_codes.data_ptr(), key_scales.data_ptr(), value_codes.data_ptr(),
          value_scales.data_ptr(), key_gscale.data_ptr(), value_gscale.data_ptr(), B, bs, block_table.data_ptr(), R, W,
          table_ld, qs, sl, D ** -0.5 if scale is None else float(scale), float(softcap), sp, *extra(T, R, dev),
          max_query_len, max_seq_len, out.data_ptr(), out_ts, out_hs, None if ws is None else ws.data_ptr(), need)
    return out


def _document_arguments(doc_start, prefix_lens, T, R, dev):
    """Arguments of the documents' and the prefixes' masks."""
    if doc_start is None and prefix_lens is None:
        return None, None
    i32 = _base._torch().int32
    return (None if doc_start is None else _vector(doc_start, T, i32, dev, "doc_start"),
            None if prefix_lens is None else _vector(prefix_lens, R, i32, dev, "prefix_lens"))


def nvfp4_kv_fp4_attention(q, key_codes, key_scales, value_codes, value_scales, key_gscale, value_gscale, block_table,
                           query_start, seq_lens, *, scale=None, softcap=0.0, slopes=None, doc_start=None,
                           prefix_lens=None, max_query_len=None, max_seq_len=None, out=None):
    """:func:`nvfp4_kv_fp8_attention` over the 4-bit cache that :func:`nvfp4_kv_fp4_append` fills: the same definition,
    masks and arguments, but for the cache, whose shape gives ``block_size`` and the number of KV heads, and its scales
    (encode direction, as given to the append)."""
    return _attention(_lib().nvfp4_kv_fp4_attention, q, key_codes, key_scales, value_codes, value_scales, key_gscale,
                      value_gscale, block_table, query_start, seq_lens, scale, softcap, slopes,
                      functools.partial(_document_arguments, doc_start, prefix_lens), max_query_len, max_seq_len, out)


def nvfp4_kv_fp4_tree_attention(q, key_codes, key_scales, value_codes, value_scales, key_gscale, value_gscale,
                                block_table, query_start, seq_lens, tree_mask, *, scale=None, softcap=0.0, slopes=None,
                                positions=None, max_query_len=None, max_seq_len=None, out=None):
    """:func:`nvfp4_kv_fp8_tree_attention` over the 4-bit cache; the cache's arguments as
    :func:`nvfp4_kv_fp4_attention`."""
    return _attention(_lib().nvfp4_kv_fp4_tree_attention, q, key_codes, key_scales, value_codes, value_scales, key_gscale,
                      value_gscale, block_table, query_start, seq_lens, scale, softcap, slopes,
                      functools.partial(_tree_arguments, tree_mask, positions), max_query_len, max_seq_len, out)


# ---- verification -----------------------------------------------------------------------------


def _probabilities(t, rows, vocab, dev, name):
    """Check ``t [rows, vocab]``; returns its row pitch."""
    torch = _base._torch()
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32, got {t.dtype}")
    if t.dim() != 2 or t.shape != (rows, vocab) or (vocab > 1 and rows > 0 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{rows}, {vocab}] with contiguous rows, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must live on {dev}, got {t.device}")
    if rows <= 1:
        return vocab
    if t.stride(0) < vocab:
        raise ValueError(f"{name} must have rows of their own (strides {list(t.stride())}): "
                         "an expanded or overlapping view needs .contiguous()")
    return t.stride(0)


def nvfp4_verify_drafted(target_probs, draft_probs, tokens, query_start, accept_u, sample_u, *, accepted=None, out=None):
    """Verify drafted tokens against the target's probabilities, from given random numbers of [0, 1).

    Request r owns rows ``query_start[r]`` to ``query_start[r + 1]`` (int32 ``[requests + 1]``) of the step: its last
    accepted token and then its drafted ones, one after another.  Row i of ``target_probs`` (float32 ``[rows, vocab]``)
    holds the probabilities of the token behind input token ``tokens[i]`` (int32 ``[rows]``), row i of ``draft_probs``
    those that the next input token was drawn from (None: the drafted tokens were certain).  A drafted token x is
    accepted while ``accept_u * draft(x) < target(x)`` (``accept_u``: float32 ``[rows]``); the first that is not is
    replaced by a sample of ``max(target - draft, 0)``, and behind the last one, if all are accepted, comes a sample of
    the target's row (``sample_u``: float32 ``[requests]``, by the running sum in the vocabulary's order).  Chains only:
    drafted trees are not verified by this call.

    Returns ``(accepted int32[requests], out int32[rows])``: per request its accepted tokens, the sampled one, and -1."""
    torch = _base._torch()
    lib = _lib()
    dev = _cuda(target_probs, "target_probs")
    if target_probs.dim() != 2 or target_probs.shape[1] < 1:
        raise ValueError(f"target_probs must be 2-D [rows, vocab], got {list(target_probs.shape)}")
    rows, V = target_probs.shape
    ld = _probabilities(target_probs, rows, V, dev, "target_probs")
    dld = 0 if draft_probs is None else _probabilities(draft_probs, rows, V, dev, "draft_probs")
    if sample_u.dim() != 1:
        raise ValueError("sample_u must be 1-D")
    R = sample_u.shape[0]
    if R > MAX_REQUESTS:
        raise ValueError(f"at most {MAX_REQUESTS} requests, got {R}")
    i32, f32 = torch.int32, torch.float32
    tk = _vector(tokens, rows, i32, dev, "tokens")
    qs = _vector(query_start, R + 1, i32, dev, "query_start")
    au = _vector(accept_u, rows, f32, dev, "accept_u")
    su = _vector(sample_u, R, f32, dev, "sample_u")
    if accepted is None:
        accepted = torch.empty(R, dtype=i32, device=dev)
    # (entries of no request are left as they were: a new tensor has none of a caller's)
    if out is None:
        out = torch.full((rows,), -1, dtype=i32, device=dev)
    ac = _vector(accepted, R, i32, dev, "accepted")
    to = _vector(out, rows, i32, dev, "out")
    tp = target_probs.data_ptr()
    dp = None if draft_probs is None else draft_probs.data_ptr()
    wide, far = (4 * ((rows - 1) * x + V) if rows else 0 for x in (ld, dld))
    begin, end = (tk, qs, au, su, tp, dp or 0), (tk + 4 * rows, qs + 4 * R + 4, au + 4 * rows, su + 4 * R, tp + wide, dp + far if dp else 0)
    starts, ends = sorted((ac, to, *begin)), sorted((ac + 4 * R, to + 4 * rows, *end))
    if any(map(operator.gt, ends, starts[1:])):
        _refuse_ranges([("accepted", ac, ac + 4 * R), ("out", to, to + 4 * rows)],
                       zip(("tokens", "query_start", "accept_u", "sample_u", "target_probs", "draft_probs"), begin, end))
    need = lib.nvfp4_verify_drafted_workspace(R, V)
    # from the caching allocator on the current stream: no two calls that may run at once share one
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, lib.nvfp4_verify_drafted, tp, ld, dp, dld, rows, V, tk, qs, R, au, su, ac, to,
          None if ws is None else ws.data_ptr(), need)
    return accepted, out

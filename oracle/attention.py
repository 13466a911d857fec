"""CPU oracle of the operators around the paged FP8 KV cache (test infrastructure only): block tables
and slot maps, attention of prompts and of drafted trees over the cache.

This module is test infrastructure: only ``tests/`` may import it, and it imports nothing from the
product path.  Plain loops over requests, heads and tokens, in binary64 and Python integers.

Definitions (this library's; the pages name an FP8 cache under attention layers and give no formula):

T1  request r with c cached and n new tokens holds ceil(c / bs) blocks and needs ceil((c + n) / bs)
    (both at most the table's width); new blocks come from the free list in request order, -1 when
    it is used up; token c + i goes to slot block * bs + (c + i) % bs, -1 without a block.
A1  query row i of the n of a request stands at position p = len - n + i; x_j = scale * q . K_j,
    then cap * tanh(x / cap), then + slope * (pos_j - p); out = sum exp(x_j) V_j / sum exp(x_j) over
    the visible j, zeros when none is.
A2  prompts: doc_start <= j and (j <= p or j < prefix), so documents bound the prefix.
    Trees: j < len - n, or bit j - (len - n) set.
A3  positions whose table column, block or slot is outside the table or the cache are not visible.
"""

from __future__ import annotations

import numpy as np

from .nvfp4_oracle import e4m3_decode


def block_tables(context_lens, query_lens, free_blocks, block_table, block_size, max_tokens,
                 free_start=0):
    """``(slot_mapping, positions, query_start, seq_lens, blocks_needed, block_table)``."""
    table = np.array(block_table, dtype=np.int64)
    width = table.shape[1]
    slots, pos, starts, lens, used = [], [], [0], [], 0
    for r, (c, n) in enumerate(zip(context_lens, query_lens)):
        c, n = max(int(c), 0), max(int(n), 0)
        have, need = min(-(-c // block_size), width), min(-(-(c + n) // block_size), width)
        for col in range(have, need):
            at = free_start + used
            table[r, col] = int(free_blocks[at]) if 0 <= at < len(free_blocks) else -1
            used += 1
        for p in range(c, c + n):
            col = p // block_size
            b = table[r, col] if col < width else -1
            slots.append(int(b) * block_size + p % block_size if b >= 0 else -1)
            pos.append(p)
        starts.append(starts[-1] + n)
        lens.append(c + n)
    slots, pos = slots[:max_tokens], pos[:max_tokens]
    pad = max_tokens - len(slots)
    return (np.array(slots + [-1] * pad, np.int64), np.array(pos + [0] * pad, np.int64),
            np.array(starts, np.int64), np.array(lens, np.int64), used, table)


def _decode(codes, scale):
    c = np.asarray(codes, np.uint8)
    nan = (c & 0x7F) == 0x7F
    v = np.where(c & 0x80, -1.0, 1.0) * e4m3_decode(np.where(nan, 0, c & 0x7F)).astype(np.float64)
    return np.where(nan, np.nan, v) * float(scale)


def slots_of(table_row, length, block_size, num_slots):
    """Slot of every position below ``length``, or -1 (rule A3)."""
    out = np.full(length, -1, np.int64)
    for j in range(length):
        col = j // block_size
        if col < len(table_row) and table_row[col] >= 0:
            s = int(table_row[col]) * block_size + j % block_size
            out[j] = s if s < num_slots else -1
    return out


def attention(q, key_cache, value_cache, key_scale, value_scale, block_table, query_start, seq_lens,
              block_size, kv_heads, scale, softcap=0.0, slopes=None, doc_start=None, prefix_lens=None,
              tree=None, positions=None, out=None, out_eps=0.0, decode=_decode):
    """``(out, tolerance)`` in binary64.  ``tree``: bool ``[tokens, drafted]`` (drafted trees), else
    prompts.  ``decode``: ``(cache rows, scale)`` to values, the FP8 cache's unless given.  ``out``: initial
    contents, kept where no request owns a row.  The tolerance of an element
    counts the roundings of an FP32 computation whose exponentials are rounded to FP16 (half steps
    2^-24 and 2^-11; below 2^-14 an absolute 2^-25, where a row's largest weight is 2^4 at least) and whose
    result is rounded with relative step ``out_eps``:

      out_eps / 2 |o|, 2^-25 at least for FP16     the last rounding (FP16 numbers below 2^-14 lie 2^-24
                                                   apart: 8.518 2^-24 is rounded to 9 2^-24, off by
                                                   0.48 steps; BF16's 2^-133 count as nothing)
      + A 2^-11 + 2^-29 sum|v| / sum p'            exponentials to FP16; A = sum p |v| / sum p, and
                                                   p' = p / max p (the kernel's reference is at most
                                                   2^-4 of the maximum, so its sum is at least 2^4
                                                   times this one)
      + 2 A dx                                     scores off by dx: p changes by exp(dx), above and
                                                   below the fraction
      + 2 A (N + 64) 2^-23                         sums over N keys, in any order, and their joining

    dx = 2^-23 ((head_dim + 8) X + 8 min(cap, max(128, X)) + 4 |bias|max + 8),  X = max_j scale sum|q k|."""
    q = np.asarray(q, np.float64)
    T, H, D = q.shape
    G = H // kv_heads
    o = np.zeros((T, H, D)) if out is None else np.array(out, np.float64)
    tol = np.zeros((T, H, D))
    num_slots = key_cache.shape[0]
    for r in range(len(seq_lens)):
        t0, t1 = (int(np.clip(query_start[r + e], 0, T)) for e in (0, 1))
        n, L = t1 - t0, max(int(seq_lens[r]), 0)
        if n <= 0:
            continue
        ctx = L - n
        slot = slots_of(block_table[r], L, block_size, num_slots)
        there = slot >= 0
        j = np.arange(L)
        kpos = j.astype(np.float64)
        if positions is not None:
            for d in range(n):
                if 0 <= ctx + d < L:
                    kpos[ctx + d] = positions[t0 + d]
        for h in range(H):
            cols = slice((h // G) * D, (h // G) * D + D)
            K = decode(key_cache[np.maximum(slot, 0), cols], key_scale)
            V = decode(value_cache[np.maximum(slot, 0), cols], value_scale)
            for i in range(n):
                t, p = t0 + i, ctx + i
                if tree is not None:
                    see = j < ctx
                    d = j - ctx
                    ok = (d >= 0) & (d < tree.shape[1])
                    see = see | (ok & tree[t][np.clip(d, 0, tree.shape[1] - 1)])
                    at = float(positions[t]) if positions is not None else float(p)
                else:
                    see = j <= p
                    if prefix_lens is not None:
                        see = see | (j < prefix_lens[r])
                    if doc_start is not None:
                        see = see & (j >= doc_start[t])
                    at = float(p)
                see = see & there
                if not see.any():
                    o[t, h] = 0.0
                    continue
                k, v = K[see], V[see]
                x = scale * (k @ q[t, h])
                mag = np.max(np.abs(scale) * (np.abs(k) @ np.abs(q[t, h])))
                big = 0.0
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    b = float(slopes[h]) * (kpos[see] - at)
                    big = np.max(np.abs(b))
                    x = x + b
                w = np.exp(x - np.max(x))
                total = w.sum()
                o[t, h] = (w @ v) / total
                A = (w @ np.abs(v)) / total
                dx = 2.0 ** -23 * ((D + 8) * mag + 8 * min(softcap, max(128.0, mag)) + 4 * big + 8)
                least = 2.0 ** -25 if out_eps == 2.0 ** -10 else 0.0
                tol[t, h] = (np.maximum(out_eps / 2 * np.abs(o[t, h]), least) + A * (2.0 ** -11 + 2 * dx + 2 * (len(w) + 64) * 2.0 ** -23)
                             + 2.0 ** -29 * np.abs(v).sum(0) / total)
    return o, tol

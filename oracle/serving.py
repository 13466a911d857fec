"""CPU oracle of the serving operators (test infrastructure only): norms and position rotation of head
vectors, the 4-bit cache, verification of drafted tokens.

This module is test infrastructure: only ``tests/`` may import it, and it imports nothing from the product
path.  Head vectors in 64-bit significands (``numpy.longdouble``), verification in exact rationals.

Definitions (this library's; the pages give none):

H1  n_i = x_i / sqrt(mean(x^2) + eps) * (offset + w_i), or x_i without a weight.
H2  pairs (n_i, n_{i + f}) or (n_2i, n_{2i + 1}), i < f, are rotated by positions[t] * inv_freq[i]; the rest is kept.
H3  the result is rounded once, to nearest even, to the input's type.
Q1  a 4-bit cache row is the head vector's NVFP4 encoding under a static global scale g, decoded as V * sd / g; the
    block scale is E4M3(fl(amax * fl(g * fl(1/6)))), a product where the tensor encoder forms fl(g / 6).
V1  token x_i is accepted while u_i q_i(x_i) < p_i(x_i); then the lowest v with w(v) > 0 and
    sum_{u <= v} w(u) > u' sum w, w = max(p - q, 0), or p behind the last drafted token, or where all w are 0.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from .nvfp4_oracle import E2M1_VALUES, e2m1_encode_magnitude, e4m3_decode, e4m3_encode, unpack_codes

#: lowest exponent of a normal number and bits behind the point
TYPES = {"f32": (-126, 23), "bf16": (-126, 7), "f16": (-14, 10)}


def round_to(x, dtype):
    """``x`` (longdouble) to the nearest number of ``dtype``, ties to even (no number overflows in the tests)."""
    low, bits = TYPES[dtype]
    _, e = np.frexp(np.where(x == 0, np.longdouble(1), x))
    step = np.ldexp(np.longdouble(1), np.maximum(e - 1, low) - bits)
    return np.rint(x / step) * step


def turn(x, positions=None, inv_freq=None, interleaved=False, weight=None, eps=0.0, offset=0.0):
    """``(value, size)``: the head vectors of ``x [tokens, heads, head_dim]`` by H1 and H2, before H3, and
    |a| + |b| of each element's pair (an error bound's unit)."""
    n = np.array(x, np.longdouble)
    if weight is not None:
        mean = (n * n).sum(-1, keepdims=True) / n.shape[-1]
        n = n / np.sqrt(mean + np.longdouble(eps)) * (np.longdouble(offset) + np.asarray(weight, np.longdouble))
    out, size = n.copy(), np.abs(n)
    if positions is not None:
        f = len(inv_freq)
        i = np.arange(f)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + f)
        w = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)
        c, s = np.cos(w)[:, None], np.sin(w)[:, None]
        out[..., a] = n[..., a] * c - n[..., b] * s
        out[..., b] = n[..., b] * c + n[..., a] * s
        size[..., a] = size[..., b] = np.abs(n[..., a]) + np.abs(n[..., b])
    return out, size


def encode4(rows, g):
    """4-bit ``(codes, scales)`` of ``rows [..., head_dim]`` (float32 values) under the static scale ``g`` (Q1): the
    encoder's steps in binary32, but for the block scale's factor."""
    rows, g = np.asarray(rows, np.float32), np.float32(g)
    v = rows.reshape(*rows.shape[:-1], rows.shape[-1] // 16, 16)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        factor = g * (np.float32(1.0) / np.float32(6.0))
        scales = e4m3_encode((np.abs(v).max(-1) * factor).astype(np.float32)).astype(np.uint8)
        sd = e4m3_decode(scales).astype(np.float32)
        r = np.where(sd > 0, g / np.where(sd > 0, sd, np.float32(1.0)), np.float32(0.0)).astype(np.float32)
        y = (np.abs(v) * r[..., None]).astype(np.float32)
    code = np.where((sd > 0)[..., None], e2m1_encode_magnitude(y), 0) | np.signbit(v).astype(np.int64) << 3
    code = code.reshape(rows.shape)
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8), scales


def decode4(codes, scales):
    """Exact V(code) * scale of codes and scale bytes (bit 7 of a scale ignored, 0x7F as 480), in binary64."""
    codes, scales = np.asarray(codes, np.uint8), np.asarray(scales, np.uint8) & 0x7F
    flat = unpack_codes(codes.reshape(-1, codes.shape[-1]))
    v = np.asarray(E2M1_VALUES, np.float64)[flat & 7] * np.where(flat & 8, -1.0, 1.0)
    sd = np.where(scales == 0x7F, 480.0, e4m3_decode(np.minimum(scales, 0x7E)).astype(np.float64))
    return v.reshape(*codes.shape[:-1], -1) * np.repeat(sd, 16, axis=-1)


def verify(target, draft, tokens, query_start, accept_u, sample_u, out):
    """``(accepted, out)`` by V1, request by request in exact arithmetic; ``out``: initial contents."""
    rows, V = target.shape
    accepted, out = [], np.array(out)
    whole = lambda x: int(Fraction(float(x)) * 2 ** 160)  # noqa: E731  (every float32 is a multiple of 2^-149)
    for r in range(len(sample_u)):
        s, e = (int(np.clip(query_start[r + k], 0, rows)) for k in (0, 1))
        if e <= s:
            accepted.append(0)
            continue
        row = s
        while row < e - 1:
            x = int(tokens[row + 1])
            if not 0 <= x < V:
                break
            q = Fraction(1) if draft is None else Fraction(float(draft[row, x]))
            if not Fraction(float(accept_u[row])) * q < Fraction(float(target[row, x])):
                break
            row += 1
        accepted.append(row - s)
        p = [max(whole(x), 0) for x in target[row]]
        w = list(p)
        if row < e - 1:
            if draft is None:
                if 0 <= int(tokens[row + 1]) < V:
                    w[int(tokens[row + 1])] = 0
            else:
                w = [max(a - whole(b), 0) for a, b in zip(p, draft[row])]
        if not any(w):
            w = p
        token, last, upto = -1, -1, 0
        aim = Fraction(float(sample_u[r])) * sum(w)
        for v, x in enumerate(w):
            upto += x
            if x > 0:
                last = v
                if upto > aim:
                    token = v
                    break
        out[s:e] = -1
        out[s:row] = tokens[s + 1:row + 1]
        out[row] = token if token >= 0 else last
    return np.array(accepted), out

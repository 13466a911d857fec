"""Pins of the serving operators' oracle (oracle/serving.py): rotation against complex numbers, norms against their
definition, rounding against numpy's and torch's own types, the 4-bit rows against the encoder, verification against the
law that it keeps."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle import attention as oa
from oracle import serving as osv

from .fp4_scale_util import SIXTH, middle_maxima, scale_code


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rounding_is_the_types_own(dtype):
    import torch

    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-30, 12, 20000), [0.0, -0.0, 1.0, -2.5]]).astype(np.float32)
    if dtype == "f32":  # from 64 bits: numpy rounds to nearest even
        y = rng.standard_normal(20000)
        assert np.array_equal(osv.round_to(y, "f32").astype(np.float32), y.astype(np.float32))
        return
    td = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    want = torch.from_numpy(x).to(td).to(torch.float32).numpy()
    assert np.array_equal(osv.round_to(x.astype(np.longdouble), dtype).astype(np.float32), want)
    # a value just past the middle between two numbers, which rounding by way of 32 bits would lose
    step = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}[dtype]
    assert osv.round_to(np.longdouble(1 + step / 2) + np.longdouble(2.0) ** -40, dtype) == 1 + step
    assert osv.round_to(np.longdouble(1 + step / 2) - np.longdouble(2.0) ** -40, dtype) == 1


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_product_of_complex_numbers(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 3, 40))
    pos, f = np.array([0, 1, 5, 100, 4096, 100000, 1 << 20]), (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    got, size = osv.turn(x, pos, f, interleaved)
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * np.outer(pos, f.astype(np.float64)))[:, None]
    assert np.allclose(got[..., a].astype(float), z.real, atol=1e-9) and np.allclose(got[..., b].astype(float), z.imag, atol=1e-9)
    assert np.array_equal(got[..., 32:].astype(float), x[..., 32:]) and np.array_equal(got[0].astype(float), x[0])
    # lengths are kept, and position p + 1 is one more turn
    assert np.allclose((got ** 2).sum(-1).astype(float), (x ** 2).sum(-1))
    again, _ = osv.turn(got, np.ones(7), f, interleaved)
    one, _ = osv.turn(x, pos + 1, f, interleaved)
    assert np.allclose(again.astype(float), one.astype(float), atol=1e-12)
    assert np.all(size >= np.abs(got) - 1e-12)


def test_norm():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((4, 2, 64)) * 5, rng.standard_normal(64)
    got, _ = osv.turn(x, weight=np.zeros(64), offset=1.0, eps=0.0)
    assert np.allclose((got ** 2).mean(-1).astype(float), 1.0)
    got, _ = osv.turn(x, weight=w, offset=0.5, eps=0.25)
    want = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 0.25) * (0.5 + w)
    assert np.allclose(got.astype(float), want)
    assert not osv.turn(np.zeros((1, 1, 64)), weight=w, eps=1e-6)[0].any()


def test_rows_of_the_cache():
    """The tensor encoder's codes under the same scales; scales next to its own, and only where the maximum lies in the
    middle between two."""
    rng = np.random.default_rng(3)
    for g in (200.0, 56.0, 448.0, 3.0):
        x = (rng.standard_normal((300, 2, 64)) * np.exp2(rng.integers(-4, 3, (300, 2, 64)))).astype(np.float32)
        x = np.round(x * 32) / 32  # few bits: maxima on the middle between two scales are common
        c, s = osv.encode4(x, g)
        assert c.shape == (300, 2, 32) and s.shape == (300, 2, 4)
        qc, qs, _ = oracle.quantize(x.reshape(600, 64), np.float32(g))
        qc, qs = qc.reshape(c.shape), qs.reshape(s.shape)
        alike = np.repeat(qs == s, 8, axis=-1)
        assert np.array_equal(qc[alike], c[alike])
        scaled = np.abs(x).reshape(300, 2, 4, 16).max(-1).astype(np.float64) * g / 6
        lo, hi = (np.minimum, np.maximum)
        values = [oracle.e4m3_decode(f(qs, s)).astype(np.float64) for f in (lo, hi)]
        off = qs != s
        assert np.all(np.abs(qs.astype(int) - s)[off] == 1)
        assert np.all(np.abs(scaled - (values[0] + values[1]) / 2)[off] <= 2.0 ** -22 * scaled[off])
    back = osv.decode4(*osv.encode4(x, 3.0)) / 3.0
    assert np.abs(back - x).max() <= np.abs(x).max() / 5  # E2M1's widest step, 4 to 6, less a scale's rounding
    assert osv.decode4(np.array([[0x77] * 8], np.uint8), np.array([[0xFF]], np.uint8)).max() == 6 * 480


@pytest.mark.parametrize("g", [56.0, 448.0, 200.0, 140.0, 300.0, 3.0])
def test_scales_of_the_cache_at_the_middles(g):
    """Blocks whose maximum lies next to the middle between two scale codes: the code by the definition alone, step by
    step (fp4_scale_util)."""
    maxima = middle_maxima(g)
    x = np.zeros((len(maxima), 1, 16), np.float32)
    x[:, 0, 3] = -maxima
    got = osv.encode4(x, g)[1][:, 0, 0]
    assert np.array_equal(got, [scale_code(a, g) for a in maxima])
    # the tensor encoder's factor is the quotient: the same codes where it is the same number, else next to them
    other = oracle.quantize(x[:, 0], np.float32(g))[1].reshape(-1)
    alike = np.float32(g) / np.float32(6) == np.float32(g) * (np.float32(1) / np.float32(6))
    assert alike == (g in (140.0, 300.0, 3.0))
    assert np.array_equal(got, other) if alike else 0 < np.sum(got != other) and np.abs(got.astype(int) - other).max() == 1


def test_a_global_scale_of_six_times_a_number_has_one_factor():
    """g = 6 x, exactly: fl(g / 6) = x, and g fl(1/6) = x (1 + 2^-25), less than half a place from x."""
    assert Fraction(SIXTH) * 6 == 1 + Fraction(1, 2 ** 25)
    x = np.random.default_rng(6).uniform(1, 2, 100000).astype(np.float32)
    x = x.view(np.uint32) & ~np.uint32(7)  # three bits for the product with 6
    x = np.concatenate([x.view(np.float32), np.float32([1.0, 2.0 - 2.0 ** -20])])
    g = x * np.float32(6)
    assert np.array_equal(g.astype(np.float64), x.astype(np.float64) * 6)
    assert np.array_equal(g / np.float32(6), x) and np.array_equal(g * np.float32(SIXTH), x)


def test_scales_of_the_cache_by_hand():
    """2.25 * 56 / 6 is 21, the middle between 20 (0x5A) and 22 (0x5B): fl(56 / 6) is below 56 / 6 and the product rounds to 21
    itself, a tie (even: 20); fl(56 fl(1/6)) is the next number, above it, and the product 21 + 2^-19: 22."""
    x = np.zeros((1, 1, 16), np.float32)
    x[0, 0, 0] = 2.25
    assert scale_code(2.25, 56.0) == 0x5B and osv.encode4(x, 56.0)[1].item() == 0x5B
    assert oracle.quantize(x[0], np.float32(56.0))[1].item() == 0x5A


def test_attention_takes_decoded_rows():
    """The attention's oracle on rows decoded beforehand is the one on FP8 codes."""
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 0x78, (32, 64)).astype(np.uint8)
    q = rng.standard_normal((3, 2, 64))
    rest = ([[0, 1]], [0, 3], [20], 16, 1, 0.125)
    a, ta = oa.attention(q, codes, codes, 0.5, 0.25, *rest)
    k, v = oa._decode(codes, 0.5), oa._decode(codes, 0.25)
    b, tb = oa.attention(q, k, v, 1.0, 1.0, *rest, decode=lambda x, s: x * s)
    assert np.allclose(a, b) and np.allclose(ta, tb)


@pytest.mark.parametrize("certain", [False, True])
def test_what_is_emitted_follows_the_target(certain):
    """One drafted token, all values of both random numbers on a grid on which every weight is a whole number: the
    first emitted token's frequency is the target's probability exactly."""
    p = np.array([[8, 1, 4, 3, 0], [2, 2, 4, 4, 4]], np.float32) / 16
    q = None if certain else np.array([[2, 4, 8, 2, 0], [0, 0, 0, 0, 0]], np.float32) / 16
    draft = [Fraction(1, 2), 0, Fraction(1, 2), 0, 0] if certain else [Fraction(float(x)) for x in q[0]]
    # (drafts that are certain: one token or another, by a coin that the verification does not see)
    n = 240
    mass = [Fraction(0)] * 5
    for x in range(5):
        if not draft[x]:
            continue
        for i in range(n):
            u = np.float32((i + 0.5) / n)
            accepted, out = osv.verify(p, q, [0, x], [0, 2], [u, 0.0], [0.0], np.zeros(2, int))
            if accepted[0]:
                mass[int(out[0])] += draft[x] / n
                continue
            weights = [Fraction(float(a)) for a in p[0]]
            if certain:
                weights[x] = Fraction(0)
            else:
                weights = [max(a - Fraction(float(b)), 0) for a, b in zip(weights, q[0])]
            total = sum(weights)
            for k in range(48):
                _, out = osv.verify(p, q, [0, x], [0, 2], [u, 0.0], [np.float32((k + 0.5) / 48)], np.zeros(2, int))
                mass[int(out[0])] += draft[x] / n / 48
            assert total > 0
    # the grid of 240 values of u meets p / q in whole steps; that of 48 meets the weights within half a step
    for v in range(5):
        assert abs(mass[v] - Fraction(float(p[0, v]))) <= Fraction(1, 48), (v, float(mass[v]))


def test_verification_by_hand():
    p = np.array([[0.5, 0.5, 0], [0.25, 0, 0.75], [0, 0.125, 0.875]], np.float32)
    q = np.array([[0.25, 0.75, 0], [0.5, 0.25, 0.25], [1, 0, 0]], np.float32)
    run = lambda tokens, u, w, draft=q: [x.tolist() for x in osv.verify(p, draft, tokens, [0, 3], u, [w], np.full(3, -7))]  # noqa: E731
    # 0.5 * 0.75 < 0.5; then 0.4 * 0.25 < 0.75; then the last row
    assert run([9, 1, 2], [0.5, 0.4, 0.0], 0.1) == [[2], [1, 2, 1]]
    assert run([9, 1, 2], [0.5, 0.4, 0.0], 0.125) == [[2], [1, 2, 2]]  # on the border: the next
    # 0.7 * 0.75 >= 0.5: weights (0.25, 0, 0)
    assert run([9, 1, 2], [0.7, 0.4, 0.0], 0.99) == [[0], [0, -1, -1]]
    # the second is token 1, which the target excludes: weights (0, 0, 0.5)
    assert run([9, 1, 1], [0.5, 0.0, 0.0], 0.0) == [[1], [1, 2, -1]]
    # certain drafts: 0.6 >= 0.5; the rest without token 1
    assert run([9, 1, 2], [0.6, 0.0, 0.0], 0.9, None) == [[0], [0, -1, -1]]
    assert run([9, 5, 2], [0.0, 0.0, 0.0], 0.9, None) == [[0], [1, -1, -1]]


def test_a_row_of_several_requests_is_the_last_ones():
    rng = np.random.default_rng(5)
    p, q = (x / x.sum(1, keepdims=True) for x in rng.random((2, 12, 9)).astype(np.float32))
    tokens, u = rng.integers(0, 9, 12), rng.random(12).astype(np.float32)
    for start in ([0, 6, 2, 9, 0, 4], [0, 3, 7, 12, 0, 0, 0], [-4, 3, 2, 100]):
        w = rng.random(len(start) - 1).astype(np.float32)
        accepted, out = osv.verify(p, q, tokens, start, u, w, np.full(12, -7))
        alone = [osv.verify(p, q, tokens, start[r:r + 2], u, w[r:r + 1], np.full(12, -7)) for r in range(len(w))]
        assert accepted.tolist() == [a[0] for a, _ in alone]
        for t in range(12):
            owners = [r for r in range(len(w)) if max(start[r], 0) <= t < min(start[r + 1], 12)]
            assert out[t] == (alone[owners[-1]][1][t] if owners else -7)

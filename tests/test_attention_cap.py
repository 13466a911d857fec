"""The two forms in which the attention kernels cap a score, emulated in binary32 with the hardware's exp2 and
reciprocal one unit off either way, against cap tanh(x / cap) in binary64: the error is within the term
that the oracle's tolerance and the header count for it, 2^-20 min(cap, max(128, |x|)), at every cap."""

import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "bit_block_scaled_nvfp4_amd", "csrc", "kv_attention_common.h")
LOG2E = np.float32(1.44269504088896340736)
f32 = np.float32


def _off(v, units):
    """Binary32 of v, some units in the last place away from the nearest."""
    v = np.asarray(v, np.float64).astype(f32)
    return v if units == 0 else np.nextafter(v, f32(np.inf if units > 0 else -np.inf))


def _fma(a, b, c):
    return (a.astype(np.float64) * np.float64(b) + np.float64(c)).astype(f32)


def _cap_term(x, to_r, e, r):
    with np.errstate(over="ignore"):
        t = _off(np.exp2((x * to_r).astype(f32).astype(np.float64)), e)
        return _off(1.0 / (t + f32(1.0)).astype(f32).astype(np.float64), r)


def _small(x, cap, e, r):
    top = f32(cap) * LOG2E
    to_r = (LOG2E * (f32(1.0) / f32(cap))) * f32(2.0)  # one raw product counts as one score
    return _fma(_cap_term(x, to_r, e, r), f32(-2.0) * top, top)


def _wide(x, cap, e, r):
    top = f32(cap) * LOG2E
    to_y = LOG2E / top
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        y = (x * to_y).astype(f32)
        z = (y * y).astype(f32)
        den = _fma(z, (z + f32(45.0)).astype(f32).astype(np.float64), 105.0)
        near = ((x * LOG2E).astype(f32) * (_fma(z, 10.0, 105.0) * _off(1.0 / den.astype(np.float64), r)).astype(f32)).astype(f32)
        far = _fma(_cap_term(x, (f32(2.0) * LOG2E) * to_y, e, r), f32(-2.0) * top, top)
    return np.where(np.abs(y) < 0.5, near, far)


def _scores(cap):
    rng = np.random.default_rng(7)
    x = np.concatenate([rng.standard_normal(20000) * s for s in (1e-3, 0.3, 4.0, 60.0)]
                       + [cap * rng.uniform(-8, 8, 20000), cap * rng.uniform(0.49, 0.51, 20000) * rng.choice([-1, 1], 20000), [0.0]])
    return x.astype(f32)


@pytest.mark.parametrize("exp_off", [-1, 0, 1])
@pytest.mark.parametrize("rcp_off", [-1, 0, 1])
@pytest.mark.parametrize("cap", [1e-3, 0.5, 5.0, 30.0, 50.0, 64.0, 128.0, 128.01, 200.0, 1e3, 1e4, 1e5, 1e6, 1e7, 1e9, 1e20, 1e37])
def test_error_of_the_capped_score(cap, exp_off, rcp_off):
    x = _scores(cap)
    small = float(re.search(r"kSmallCap = ([\d.]+)f;", open(SRC).read()).group(1))
    got = (_small if cap <= small else _wide)(x, cap, exp_off, rcp_off).astype(np.float64) / np.float64(LOG2E)
    c = np.float64(f32(cap))
    want = c * np.tanh(x.astype(np.float64) / c)
    err = np.abs(got - want)
    lim = 2.0 ** -20 * np.minimum(c, np.maximum(128.0, np.abs(x))) + 2.0 ** -22 * np.abs(want)
    assert np.all(err <= lim), (cap, x[np.argmax(err - lim)], (err / lim).max())
    if cap > small:  # and relative to the score itself, whatever the cap
        ok = np.abs(x) > 0
        assert np.max(err[ok] / np.abs(want[ok])) < 2.0 ** -20


def test_the_form_for_small_caps_would_not_do_for_large_ones():
    x = _scores(1e6)[:80000]
    got = _small(x, 1e6, 0, 0).astype(np.float64) / np.float64(LOG2E)
    assert np.max(np.abs(got - 1e6 * np.tanh(x / 1e6))) > 100 * 2.0 ** -20 * 128

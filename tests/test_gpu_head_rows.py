"""GPU parity of the head vectors' operators (nvfp4_qk_norm_rope, nvfp4_kv_fp8_append, nvfp4_kv_fp4_append,
nvfp4_kv_fp4_load) against the oracle in 64-bit significands.

The operators' contract is one rounding of a value formed in binary64, off by at most 2^-48 (|a| + |b|) before it: a
result must lie between the roundings of the oracle's value less and plus that (which are the same number but for one
element in about 2^38).  Codes and decoded values must be equal bit for bit to the unfused operators', and through them to
the oracle's."""

import numpy as np
import pytest

import bit_block_scaled_nvfp4_amd as nv
import oracle
from oracle import serving as osv

from .attention_util import to_type
from .fp4_scale_util import middle_maxima, scale_code
from .gpu_util import DEV, log

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
SENTINEL = 7.5


def _td(dtype):
    import torch

    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]


def _up(x, dtype="f32"):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(_td(dtype)).to(DEV)


def _values(x, dtype):
    """float32 holding numbers of ``dtype``."""
    return np.asarray(x, np.float32) if dtype == "f32" else to_type(x, dtype)


def _host(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, tokens, heads, kv_heads, head_dim, freqs, dtype="bf16", seed=0, weights=None, first=0,
                 interleaved=False, eps=1e-6, offset=0.0):
        rng = np.random.default_rng(seed)
        self.dtype, self.eps, self.offset, self.interleaved = dtype, eps, offset, interleaved
        mk = lambda h: _values(rng.standard_normal((tokens, h, head_dim)) * 3.0, dtype)  # noqa: E731
        self.q, self.k, self.v = mk(heads), mk(kv_heads), mk(kv_heads)
        self.positions = (first + rng.permutation(max(tokens, 1) * 2)[:tokens]).astype(np.int64)
        self.inv_freq = (10000.0 ** (-np.arange(freqs) / max(freqs, 1))).astype(np.float32)
        self.weight_type = weights
        self.qw, self.kw = (None, None) if weights is None else (_values(rng.standard_normal(head_dim) * 0.5, weights) for _ in range(2))

    def turned(self, x, w):
        kw = dict(positions=self.positions, inv_freq=self.inv_freq) if len(self.inv_freq) else {}
        return osv.turn(x, interleaved=self.interleaved, weight=w, eps=self.eps, offset=self.offset, **kw)

    def words(self):
        import torch

        i32 = torch.from_numpy(self.positions).to(torch.int32).to(DEV)
        return ((i32, _up(self.inv_freq)) if len(self.inv_freq) else (None, None),
                dict(eps=self.eps, weight_offset=self.offset, interleaved=self.interleaved))

    def weight(self, w):
        return None if w is None else _up(w, self.weight_type)


def same(got, value, size, dtype, what):
    got = np.asarray(got, np.longdouble)
    slack = size * np.longdouble(2.0) ** -48
    low, high = osv.round_to(value - slack, dtype), osv.round_to(value + slack, dtype)
    bad = np.argwhere(~((got >= low) & (got <= high)))
    assert bad.size == 0, (f"{what}: {len(bad)} of {got.size} differ, first {bad[0].tolist()}: got {got[tuple(bad[0])]!r}, "
                           f"expected {low[tuple(bad[0])]!r} of {value[tuple(bad[0])]!r}")


def rope(c, **kw):
    at, words = c.words()
    k = kw.pop("k", _up(c.k, c.dtype))
    return nv.nvfp4_qk_norm_rope(kw.pop("q", _up(c.q, c.dtype)), k, *at, q_weight=c.weight(c.qw),
                                 k_weight=None if k is None else c.weight(c.kw), **words, **kw)


def check(c, what):
    log(f"rope {what}")
    q, k = rope(c)
    same(_host(q), *c.turned(c.q, c.qw), c.dtype, what + " q")
    same(_host(k), *c.turned(c.k, c.kw), c.dtype, what + " k")


@TYPES
@pytest.mark.parametrize("weights", [None, "f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("head_dim,freqs", [(64, 32), (128, 64), (256, 32), (256, 128), (80, 40), (96, 16), (16, 8), (512, 256), (128, 0)])
def test_types_norms_pairs_and_head_sizes(dtype, weights, interleaved, head_dim, freqs):
    c = Case(5, 3, 2, head_dim, freqs, dtype, seed=head_dim + freqs, weights=weights, interleaved=interleaved, offset=1.0)
    check(c, f"{dtype} w={weights} pairs={interleaved} D={head_dim} f={freqs}")


@pytest.mark.parametrize("tokens", [1, 2, 7, 64, 65, 513, 2049])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (24, 4), (7, 1), (32, 8)])
def test_lengths_and_head_counts(tokens, heads, kv_heads):
    if tokens > 600 and heads > 7:
        heads, kv_heads = 5, 2
    check(Case(tokens, heads, kv_heads, 64, 32, seed=tokens, weights="bf16"), f"T={tokens} H={heads}/{kv_heads}")


@pytest.mark.parametrize("first", [0, 4000, 131000, 1048576, 2 ** 30])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(first, interleaved):
    check(Case(40, 2, 1, 128, 64, "f32", seed=3, first=first, interleaved=interleaved), f"positions from {first}")


def test_negative_positions_and_large_frequencies():
    c = Case(30, 2, 1, 64, 32, "f32", seed=4)
    c.positions = -c.positions - 5
    check(c, "negative positions")
    c.inv_freq = np.linspace(0.0, 30.0, 32).astype(np.float32)
    check(c, "frequencies up to 30")


@TYPES
def test_small_and_large_values(dtype):
    """Subnormal results, zeros of both signs, and rows of the type's largest numbers."""
    c = Case(6, 2, 1, 64, 16, dtype, seed=5)
    tiny = {"bf16": 2.0 ** -130, "f16": 2.0 ** -20, "f32": 2.0 ** -140}[dtype]
    c.q[0] = _values(c.q[0] * tiny, dtype)
    c.q[1] = 0.0
    c.q[2, :, ::2] = -0.0
    c.q[3] = _values(np.sign(c.q[3]) * {"bf16": 1e38, "f16": 30000.0, "f32": 1e38}[dtype], dtype)
    check(c, f"small and large {dtype}")
    n = Case(4, 2, 1, 64, 0, dtype, seed=6, weights="f32", eps=1e-5)
    n.q[0] = 0.0  # the norm of zeros is zero
    n.q[1] = _values(n.q[1] * 1e-4, dtype)
    check(n, f"norm of small rows {dtype}")


def test_not_finite_values_stay_in_their_head():
    import torch

    c = Case(4, 3, 1, 64, 32, "bf16", seed=7, weights="f32")
    clean = rope(c)[0]
    c.q[1, 2, 5] = np.inf
    c.q[2, 0, 9] = np.nan
    got = rope(c)[0]
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[1, 2] = keep[2, 0] = False
    assert bool((got[keep] == clean[keep]).all()) and bool(got[2, 0].isnan().all()) and not bool(got[1, 2].isfinite().all())


def test_strides_in_place_and_windows():
    """Views of a fused row, written in place and into windows of wider rows; head-major storage; one head for all."""
    import torch

    T, H, Hk, D = 19, 6, 2, 128
    c = Case(T, H, Hk, D, 32, seed=8, weights="bf16", offset=1.0)
    want = rope(c)
    fused = torch.full((T, (H + 2 * Hk) * D), SENTINEL, dtype=torch.bfloat16, device=DEV)
    q, k = fused[:, : H * D].unflatten(1, (H, D)), fused[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    q.copy_(_up(c.q, "bf16"))
    k.copy_(_up(c.k, "bf16"))
    log("windows and in place")
    wide = torch.full((T, H + Hk + 3, D + 8), SENTINEL, dtype=torch.bfloat16, device=DEV)
    got = rope(c, q=q, k=k, q_out=wide[:, 1:H + 1, :D], k_out=wide[:, H + 2:H + 2 + Hk, :D])
    assert all(bool((a == b).all()) for a, b in zip(got, want))
    rest = wide.clone()
    rest[:, 1:H + 1, :D] = SENTINEL
    rest[:, H + 2:H + 2 + Hk, :D] = SENTINEL
    assert bool((rest == SENTINEL).all())
    got = rope(c, q=q, k=k, q_out=q, k_out=k)
    assert got[0] is q and all(bool((a == b).all()) for a, b in zip(got, want))
    assert bool((fused[:, (H + Hk) * D:] == SENTINEL).all())
    major = _up(c.q, "bf16").transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((H, T, D), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert bool((rope(c, q=major, q_out=out)[0] == want[0]).all())
    one = _up(c.q, "bf16")[:, :1].expand(T, H, D)
    assert bool((rope(c, q=one)[0] == want[0][:, :1]).all())


def test_queries_alone_and_no_work():
    c = Case(9, 4, 2, 64, 32, seed=9, weights="f32")
    want = rope(c)
    got = rope(c, k=None)
    assert got[1] is None and bool((got[0] == want[0]).all())
    none = Case(0, 4, 2, 64, 32, seed=9)
    assert rope(none)[0].shape == (0, 4, 64)


def test_large_call_equals_small_ones():
    """A grid whose workgroups take several tokens, against the same tokens one by one."""
    c = Case(3001, 28, 4, 256, 32, seed=10, weights="bf16", first=100000)
    q, k = rope(c)
    pick = [0, 1, 2, 1499, 1500, 2998, 2999, 3000]
    for t in pick:
        one = Case(1, 28, 4, 256, 32, seed=10, weights="bf16")
        one.q, one.k, one.positions, one.qw, one.kw = c.q[t:t + 1], c.k[t:t + 1], c.positions[t:t + 1], c.qw, c.kw
        a, b = rope(one)
        assert bool((a[0] == q[t]).all()) and bool((b[0] == k[t]).all())
    part = slice(0, 40)
    same(_host(q)[part], *osv.turn(c.q[part], c.positions[part], c.inv_freq, False, c.qw, c.eps, c.offset), c.dtype, "large call")


# ---- appending --------------------------------------------------------------------------------


def _slots(rng, tokens, slots):
    s = rng.permutation(slots)[:tokens].astype(np.int64)
    if tokens > 3:
        s[2], s[3] = -1, slots + 7  # padding, and a slot outside
    return s


@TYPES
@pytest.mark.parametrize("weights,interleaved", [(None, False), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("head_dim,freqs", [(64, 32), (128, 16), (256, 32), (256, 128), (128, 0), (64, 8)])
def test_fp8_append_is_rope_and_store(dtype, weights, interleaved, head_dim, freqs):
    import torch

    log(f"fp8 append {dtype} w={weights} pairs={interleaved} D={head_dim} f={freqs}")
    T, Hk, slots = 37, 3, 60
    c = Case(T, 1, Hk, head_dim, freqs, dtype, seed=head_dim + freqs, weights=weights, interleaved=interleaved, offset=1.0)
    at, words = c.words()
    sm = torch.from_numpy(_slots(np.random.default_rng(1), T, slots)).to(DEV)
    ks, vs = torch.tensor([0.031], device=DEV), torch.tensor([0.011], device=DEV)
    caches = [torch.full((slots, Hk * head_dim + 16), 0x55, dtype=torch.uint8, device=DEV) for _ in range(4)]
    views = [x[:, :Hk * head_dim] for x in caches]
    nv.nvfp4_kv_fp8_append(_up(c.k, dtype), _up(c.v, dtype), *at, ks, vs, views[0], views[1], sm, k_weight=c.weight(c.kw), **words)
    turned = nv.nvfp4_qk_norm_rope(_up(c.k, dtype), None, *at, q_weight=c.weight(c.kw), **words)[0]
    nv.nvfp4_kv_fp8_store(turned.flatten(1), _up(c.v, dtype).flatten(1), ks, vs, views[2], views[3], sm)
    torch.cuda.synchronize()
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    value, size = c.turned(c.k, c.kw)
    same(_host(turned), value, size, dtype, "keys")
    # and to the oracle's codes
    host, kept = sm.cpu().numpy(), (sm.cpu().numpy() >= 0) & (sm.cpu().numpy() < slots)
    want = oracle.kv_fp8_encode(_host(turned).astype(np.float32).reshape(T, -1), np.float32(0.031))
    assert np.array_equal(views[0].cpu().numpy()[host[kept]], want[kept])


def _cache4(blocks, heads, bs, D, fill=0xEE):
    import torch

    u8 = lambda n: torch.full((blocks, heads, bs, n), fill, dtype=torch.uint8, device=DEV)  # noqa: E731
    return [u8(D // 2), u8(D // 16), u8(D // 2), u8(D // 16)]


def _rows4(cache, slots):
    """Bytes of the slots' rows: [slots, heads, n]."""
    bs = cache.shape[2]
    x = cache.cpu().numpy()
    return x[slots // bs, :, slots % bs]


@TYPES
@pytest.mark.parametrize("weights,interleaved", [(None, False), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("head_dim,freqs,block_size", [(64, 32, 16), (128, 16, 7), (256, 32, 1), (256, 128, 64), (128, 0, 16), (64, 16, 100)])
def test_fp4_append_is_rope_and_encoding(dtype, weights, interleaved, head_dim, freqs, block_size):
    import torch

    log(f"fp4 append {dtype} w={weights} pairs={interleaved} D={head_dim} f={freqs} bs={block_size}")
    T, Hk, blocks = 37, 3, -(-60 // block_size)
    slots = blocks * block_size
    c = Case(T, 1, Hk, head_dim, freqs, dtype, seed=head_dim + freqs, weights=weights, interleaved=interleaved, offset=1.0)
    at, words = c.words()
    host = _slots(np.random.default_rng(2), T, slots)
    sm = torch.from_numpy(host).to(DEV)
    kg, vg = torch.tensor([140.0], device=DEV), torch.tensor([300.0], device=DEV)
    cache = _cache4(blocks, Hk, block_size, head_dim)
    nv.nvfp4_kv_fp4_append(_up(c.k, dtype), _up(c.v, dtype), *at, kg, vg, *cache, sm, k_weight=c.weight(c.kw), **words)
    turned = nv.nvfp4_qk_norm_rope(_up(c.k, dtype), None, *at, q_weight=c.weight(c.kw), **words)[0]
    torch.cuda.synchronize()
    same(_host(turned), *c.turned(c.k, c.kw), dtype, "keys")
    kept = (host >= 0) & (host < slots)
    for x, g, codes, scales in ((_host(turned), kg, cache[0], cache[1]), (c.v, vg, cache[2], cache[3])):
        wc, ws = osv.encode4(np.asarray(x, np.float32), g.item())
        assert np.array_equal(_rows4(codes, host[kept]), wc[kept]) and np.array_equal(_rows4(scales, host[kept]), ws[kept])
        # nothing else is written
        others = np.setdiff1d(np.arange(slots), host[kept])
        assert np.all(_rows4(codes, others) == 0xEE) and np.all(_rows4(scales, others) == 0xEE)
        # the tensor encoder, whose factor may be a neighbour: the same codes wherever the scale is the same, and
        # scales next to one another where it is not
        qc, qs, _ = nv.nvfp4_quantize(torch.from_numpy(np.asarray(x, np.float32).reshape(-1, head_dim)).to(_td(dtype)).to(DEV), g)
        qc, qs = qc.cpu().numpy().reshape(wc.shape), qs.cpu().numpy().reshape(ws.shape)
        alike = np.repeat(qs == ws, 8, axis=-1)
        assert np.array_equal(qc[alike], wc[alike]) and np.abs(qs.astype(int) - ws).max() <= 1
    # and back
    for out_dtype, od in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        got = nv.nvfp4_kv_fp4_load(cache[2], cache[3], vg, sm, od)
        wc, ws = osv.encode4(c.v, vg.item())
        want = (osv.decode4(wc, ws).astype(np.float32) / np.float32(300.0)).astype(np.float32)
        want = np.where(kept[:, None, None], want if out_dtype == "f32" else to_type(want, "bf16"), 0.0)
        assert np.array_equal(_host(got), want)


def test_fp4_extreme_global_scales_and_zero_rows():
    import torch

    c = Case(8, 1, 1, 64, 0, "f32", seed=12)
    c.k[0] = 0.0
    c.k[1, 0, ::2] = -0.0
    c.k[2] *= 1e-6
    c.k[3] *= 1e-3  # under the largest scale: g / sd overflows
    c.k[3, 0, 7] = 0.0
    for g in (1e-30, 1.0, 3e5, 2.0 ** 125):
        log(f"global scale {g}")
        x = c.k if g < 1e30 else c.k * np.float32(1e-36)
        cache = _cache4(1, 1, 8, 64)
        gs = torch.tensor([g], dtype=torch.float32, device=DEV)
        nv.nvfp4_kv_fp4_append(_up(x), _up(x), None, None, gs, gs, *cache)
        wc, ws = osv.encode4(x, np.float32(g))
        for i in (0, 2):
            assert np.array_equal(_rows4(cache[i], np.arange(8)), wc) and np.array_equal(_rows4(cache[i + 1], np.arange(8)), ws)


def test_fp4_load_of_every_byte():
    """All codes under all scale bytes: bit 7 of a scale is ignored, 0x7F counts as 480."""
    import torch

    codes = np.zeros((256, 1, 2, 32), np.uint8)
    scales = np.zeros((256, 1, 2, 4), np.uint8)
    codes[:] = np.arange(64, dtype=np.uint8).reshape(1, 1, 2, 32) * 4 + np.arange(256, dtype=np.uint8).reshape(256, 1, 1, 1) % 4
    scales[:] = np.arange(256, dtype=np.uint8).reshape(256, 1, 1, 1)
    up = [torch.from_numpy(x).to(DEV) for x in (codes, scales)]
    rng = np.random.default_rng(0)
    exact = osv.decode4(codes, scales).astype(np.float32).transpose(0, 2, 1, 3).reshape(512, 1, 64)
    for g in [3.0, 1.0, 56.0, np.nextafter(np.float32(2), np.float32(1)), 2.0 ** -100, 2.0 ** 100, 1e-36, 2.0 ** 126, *np.exp2(rng.uniform(-90, 90, 40))]:
        g = np.float32(g)
        with np.errstate(over="ignore", under="ignore"):
            want = exact / g
        got = nv.nvfp4_kv_fp4_load(*up, torch.tensor([g], device=DEV)).cpu().numpy()
        assert np.array_equal(got.view(np.int32), want.view(np.int32)), g


def test_append_from_a_fused_row_without_slots_and_empty():
    import torch

    T, Hk, D = 21, 2, 128
    c = Case(T, 1, Hk, D, 32, seed=13, weights="f32")
    at, words = c.words()
    fused = torch.cat([_up(c.q, "bf16").flatten(1), _up(c.k, "bf16").flatten(1), _up(c.v, "bf16").flatten(1)], 1)
    k, v = fused[:, D:D + Hk * D].unflatten(1, (Hk, D)), fused[:, D + Hk * D:].unflatten(1, (Hk, D))
    g = torch.tensor([200.0], device=DEV)
    a, b = _cache4(2, Hk, 16, D), _cache4(2, Hk, 16, D)
    nv.nvfp4_kv_fp4_append(k, v, *at, g, g, *a, k_weight=c.weight(c.kw), **words)
    nv.nvfp4_kv_fp4_append(_up(c.k, "bf16"), _up(c.v, "bf16"), *at, g, g, *b, torch.arange(T, device=DEV), k_weight=c.weight(c.kw), **words)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    none = _cache4(2, Hk, 16, D)
    nv.nvfp4_kv_fp4_append(k[:0], v[:0], None, None, g, g, *none, torch.zeros(0, dtype=torch.int64, device=DEV))
    empty = _cache4(0, Hk, 16, D)
    nv.nvfp4_kv_fp4_append(k, v, None, None, g, g, *empty)
    # K and V side by side in one FP8 cache
    both = torch.full((T, 2 * Hk * D), 0x55, dtype=torch.uint8, device=DEV)
    nv.nvfp4_kv_fp8_append(k, v, *at, g, g, both[:, :Hk * D], both[:, Hk * D:], k_weight=c.weight(c.kw), **words)
    torch.cuda.synchronize()
    assert all(bool((x == 0xEE).all()) for x in none) and not bool((both == 0x55).all(1).any())


def test_fp4_rows_beyond_32_bits_of_bytes():
    """Slots whose codes lie 5 GB behind the first."""
    import torch

    D, Hk, bs = 256, 4, 16
    first = 5 * 2 ** 30 // (Hk * bs * D // 2)
    cache = [torch.empty((first + 1, Hk, bs, n), dtype=torch.uint8, device=DEV) for n in (D // 2, D // 16)]
    other = _cache4(1, Hk, bs, D)
    c = Case(10, 1, Hk, D, 32, seed=14)
    at, words = c.words()
    g = torch.tensor([200.0], device=DEV)
    sm = torch.arange(10, device=DEV)
    log("5 GB of codes")
    nv.nvfp4_kv_fp4_append(_up(c.k, "bf16"), _up(c.v, "bf16"), *at, g, g, *other, sm, **words)
    small = [torch.zeros((first + 1, Hk, bs, n), dtype=torch.uint8, device=DEV) for n in (D // 2, D // 16)]
    nv.nvfp4_kv_fp4_append(_up(c.k, "bf16"), _up(c.v, "bf16"), *at, g, g, *cache, *small, sm + first * bs, **words)
    torch.cuda.synchronize()
    assert torch.equal(cache[0][first, :, :10], other[0][0, :, :10]) and torch.equal(small[1][first, :, :10], other[3][0, :, :10])
    a = nv.nvfp4_kv_fp4_load(*cache, g, sm + first * bs)
    b = nv.nvfp4_kv_fp4_load(other[0], other[1], g, sm)
    assert torch.equal(a, b)


def test_side_stream_and_captured_graphs():
    """Captured and replayed with other inputs and eager work between the replays."""
    import torch

    c = Case(70, 6, 2, 128, 64, seed=15, weights="bf16")
    at, words = c.words()
    g = torch.tensor([200.0], device=DEV)
    q, k, v = (_up(x, "bf16") for x in (c.q, c.k, c.v))
    qw, kw = c.weight(c.qw), c.weight(c.kw)
    qo, ko, a = torch.empty_like(q), torch.empty_like(k), _cache4(5, 2, 16, 128)

    def step(q_out, k_out, cache):
        nv.nvfp4_qk_norm_rope(q, k, *at, q_weight=qw, k_weight=kw, q_out=q_out, k_out=k_out, **words)
        nv.nvfp4_kv_fp4_append(k, v, *at, g, g, *cache, k_weight=kw, **words)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(qo, ko, a)
    side.synchronize()
    same(_host(qo), *c.turned(c.q, c.qw), "bf16", "side stream")
    log("graph")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qo, ko, a)
    for r in range(4):
        q.mul_(-1.0)
        k.copy_(v if r % 2 else k * 0.5)
        at[0].add_(13)
        for x in (qo, ko):
            x.fill_(SENTINEL)
        for x in a:
            x.fill_(0xEE)
        graph.replay()
        b, q2, k2 = _cache4(5, 2, 16, 128), torch.empty_like(q), torch.empty_like(k)
        step(q2, k2, b)
        torch.cuda.synchronize()
        assert torch.equal(qo, q2) and torch.equal(ko, k2) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_numbers_of_other_types_are_taken():
    """numpy's scalars for the numbers and the flag give what Python's give."""
    import torch

    c = Case(5, 4, 2, 64, 16, weights="f32", interleaved=True, eps=0.125, offset=0.5)
    d = dict(positions=torch.from_numpy(c.positions).to(torch.int32).to(DEV), inv_freq=_up(c.inv_freq), q_weight=_up(c.qw), k_weight=_up(c.kw))
    q, k = _up(c.q, c.dtype), _up(c.k, c.dtype)
    log("numpy scalars")
    want = nv.nvfp4_qk_norm_rope(q, k, **d, eps=0.125, weight_offset=0.5, interleaved=True)
    got = nv.nvfp4_qk_norm_rope(q, k, **d, eps=np.float32(0.125), weight_offset=np.float64(0.5), interleaved=np.True_)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g", [56.0, 448.0, 200.0, 140.0, 300.0, 3.0])
def test_fp4_scales_at_the_middles_between_codes(g, dtype):
    """The scale by its definition where the choice between two codes turns; and, where the encoder's factor g / 6 is the
    same number as the cache's g fl(1/6) (140, 300, 3), the tensor encoder's codes and scales to the last bit."""
    import torch

    maxima = np.unique(_values(middle_maxima(g), dtype))
    rng = np.random.default_rng(16)
    rows = -(-len(maxima) // 4)
    x = rng.uniform(-1.0, 1.0, (rows * 4, 16)).astype(np.float32)
    peak = np.resize(maxima, rows * 4).astype(np.float32)
    x = _values(x * peak[:, None], dtype)
    x[np.arange(rows * 4), rng.integers(0, 16, rows * 4)] = peak * rng.choice([-1.0, 1.0], rows * 4).astype(np.float32)
    x = x.reshape(rows, 1, 64)
    log(f"middles g={g} {dtype}")
    gs = torch.tensor([g], device=DEV)
    cache = _cache4(1, 1, rows, 64)
    nv.nvfp4_kv_fp4_append(_up(x, dtype), _up(-x, dtype), None, None, gs, gs, *cache)
    codes, scales, back, same_scales = (_rows4(t, np.arange(rows)) for t in cache)
    want = np.array([scale_code(a, g) for a in np.abs(x).reshape(-1, 16).max(1)]).reshape(rows, 1, 4)
    assert np.array_equal(scales, want) and np.array_equal(same_scales, want)
    assert np.array_equal(codes, osv.encode4(x, g)[0]) and np.array_equal(back, osv.encode4(-x, g)[0])
    if np.float32(g) / np.float32(6) == np.float32(g) * (np.float32(1) / np.float32(6)):
        qc, qs, _ = nv.nvfp4_quantize(_up(x.reshape(rows, 64), dtype), gs)
        assert np.array_equal(qc.cpu().numpy().reshape(codes.shape), codes) and np.array_equal(qs.cpu().numpy().reshape(scales.shape), scales)

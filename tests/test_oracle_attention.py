"""CPU pins of the attention oracle (oracle/attention.py): closed forms, torch's softmax in binary64, and
the host arithmetic that the kernels rely on (quotients by a multiplication, LDS column scrambles)."""

import numpy as np
import pytest

from oracle import attention as oa

from .attention_util import Problem, pack, tree_mask, unpack


def test_block_tables_worked_example():
    # request 0: 3 cached of block size 4 (one block), 2 new: one more block; request 1: 8 cached, 1 new
    table = np.array([[7, -1, -1], [5, 6, -1]])
    slots, pos, start, lens, used, out = oa.block_tables([3, 8], [2, 1], [9, 2], table, 4, 5)
    assert slots.tolist() == [31, 36, 8, -1, -1]
    assert pos.tolist() == [3, 4, 8, 0, 0]
    assert start.tolist() == [0, 2, 3] and lens.tolist() == [5, 9] and used == 2
    assert out.tolist() == [[7, 9, -1], [5, 6, 2]]


def test_block_tables_exhausted_and_beyond_the_table():
    table = np.full((1, 2), -1)
    slots, _, _, lens, used, out = oa.block_tables([0], [12], [3], table, 4, 12)
    assert slots.tolist() == [12, 13, 14, 15] + [-1] * 8 and used == 2 and lens.tolist() == [12]
    assert out.tolist() == [[3, -1]]


def test_attention_of_equal_scores_is_the_mean():
    p = Problem([(5, 3)], 2, 1, 64, seed=1)
    p.q[:] = 0
    out, _ = p.oracle()
    slot = oa.slots_of(p.table[0], 8, p.block_size, p.num_slots)
    v = oa._decode(p.vc[slot], p.vs)
    for i in range(3):
        assert np.allclose(out[i, 0], v[:6 + i].mean(0), rtol=1e-12)


@pytest.mark.parametrize("tree", [False, True])
def test_attention_against_torch(tree):
    import torch

    p = Problem([(9, 6)], 4, 2, 64, seed=2, q_std=2.0)
    p.options["softcap"] = 8.0
    p.options["slopes"] = np.array([0.5, 0.1, 0.0, 1.0], np.float32)
    if tree:
        p.options["tree_mask"] = tree_mask(p.rng, [6])
        p.options["positions"] = 9 + p.rng.integers(0, 3, 6)
    else:
        p.options["doc_start"] = np.array([0, 0, 4, 4, 14, 14])
        p.options["prefix_lens"] = np.array([13])
    out, _ = p.oracle()
    slot = oa.slots_of(p.table[0], 15, p.block_size, p.num_slots)
    j, i = torch.arange(15), torch.arange(6)
    if tree:
        at = torch.from_numpy(p.options["positions"])
        kat = torch.cat([torch.arange(9), at])
        see = (j < 9)[None, :].repeat(6, 1)
        see[:, 9:] |= torch.from_numpy(unpack(p.options["tree_mask"])[:, :6])
    else:
        at, kat = 9 + i, j
        see = (j[None] <= at[:, None]) | (j < 13)
        see &= j[None] >= torch.from_numpy(p.options["doc_start"])[:, None]
    for h in range(4):
        cols = slice((h // 2) * 64, (h // 2) * 64 + 64)
        k, v = (torch.from_numpy(oa._decode(c[slot][:, cols], s)) for c, s in ((p.kc, p.ks), (p.vc, p.vs)))
        x = 8.0 * torch.tanh(torch.from_numpy(p.q[:, h].astype(np.float64)) @ k.t() * p.scale / 8.0)
        x = x + float(p.options["slopes"][h]) * (kat[None] - at[:, None]).double()
        w = torch.softmax(x.masked_fill(~see, -np.inf), -1)
        want = torch.where(see.any(-1, keepdim=True), w, 0.0) @ v  # a row that sees nothing: zeros
        assert np.allclose(out[:, h], want.numpy(), rtol=1e-10, atol=1e-12)


def test_tree_masks_hold_ancestors():
    rng = np.random.default_rng(3)
    bits = unpack(tree_mask(rng, [70]))
    assert bits.shape == (70, 128)
    for i in range(70):
        assert bits[i, i] and not bits[i, i + 1:].any()
        for a in np.flatnonzero(bits[i]):
            assert not (bits[a] & ~bits[i]).any()
    assert np.array_equal(unpack(pack(bits)), bits)


def test_tolerance_covers_the_roundings_it_counts():
    """The oracle's own formula in FP32 with exponentials rounded to FP16 and the result to bfloat16 stays
    within the tolerance; a key left out, or one mask bit wrong, does not."""
    import torch

    p = Problem([(200, 2)], 2, 1, 64, seed=4)
    want, tol = p.oracle()
    slot = oa.slots_of(p.table[0], 202, p.block_size, p.num_slots)
    k, v = (torch.from_numpy(oa._decode(c[slot], s)).float() for c, s in ((p.kc, p.ks), (p.vc, p.vs)))
    for h in range(2):
        for i in range(2):
            n = 201 + i
            x = (k[:n] @ torch.from_numpy(p.q[i, h])) * p.scale
            e = torch.exp(x - x.max())

            def out(w):
                return ((w.half().float() @ v[:n]) / w.sum()).to(torch.bfloat16).double().numpy()

            assert np.all(np.abs(out(e) - want[i, h]) <= tol[i, h])
            less = e.clone()
            less[e.argmax()] = 0
            assert np.any(np.abs(out(less) - want[i, h]) > tol[i, h])


def test_quotient_by_multiplication():
    """The launch constant of a division by d: exact for every dividend below 2^31."""
    def const(d):
        l = 0
        while (1 << l) < d:
            l += 1
        return -(-(1 << (31 + l)) // d), 31 + l

    rng = np.random.default_rng(5)
    for d in [1, 2, 3, 5, 7, 16, 48, 100, 641, 1000, 4095, 65535, (1 << 24) - 1, 1 << 24] + rng.integers(1, 1 << 24, 200).tolist():
        mul, shift = const(d)
        assert mul < 1 << 32
        n = np.concatenate([rng.integers(0, 1 << 31, 200), np.arange(0, 50), [(1 << 31) - 1],
                            (rng.integers(1, (1 << 31) // d + 1, 100) * d - 1), rng.integers(0, (1 << 31) // d + 1, 100) * d])
        for x in n[(n >= 0) & (n < 1 << 31)].tolist():
            assert (x * mul) >> shift == x // d


@pytest.mark.parametrize("D", [64, 128, 256])
def test_lds_layouts_of_the_tiled_kernel(D):
    """The scrambled column maps: every granule of a tile has a place of its own, what a lane reads for
    operand e of key or dim 32 n + r is what was stored there, and the lanes served together touch 16
    different columns."""
    keys = 8192 // D

    def bits(x):
        return [(x >> i) & 1 for i in range(5)]

    def k_at(key, gr):
        k0, k1, k2, k3, _ = bits(key)
        if D == 64:
            return ((key >> 1) << 8) + ((((k0 << 3) | gr) ^ ((k1 << 2) | (k2 << 1) | k3)) << 4)
        return key * 2 * D + ((gr ^ ((k0 << 3) | (k1 << 2) | (k2 << 1) | k3)) << 4)

    def v_at(dim, gr):
        d0, d1, d2, d3, d4 = bits(dim)
        if D == 256:
            return ((dim >> 2) << 8) + ((((d1 << 3) | (d0 << 2) | gr) ^ ((d4 << 3) | (d3 << 2) | (d2 << 1) | d3)) << 4)
        if D == 128:
            return ((dim >> 1) << 8) + ((((d0 << 3) | gr) ^ ((d4 << 3) | (d2 << 2) | ((d1 ^ d3) << 1) | d3)) << 4)
        return (dim << 8) + ((gr ^ (((d0 ^ d4) << 3) | ((d1 ^ d3) << 2) | (d2 << 1) | d3)) << 4)

    for at, rows, granules in ((k_at, keys, D // 8), (v_at, D, keys // 8)):
        places = {at(r, g) for r in range(rows) for g in range(granules)}
        assert len(places) == 1024 and min(places) == 0 and max(places) == 16384 - 16
        for g in range(granules):
            for b in range(0, 32, 16):
                assert len({(at(b + x, g) >> 4) % 16 for x in range(16)}) == 16
        for b in range(0, 32, 8):
            assert len({(at(b + x, h) >> 4) % 16 for x in range(8) for h in (0, 1)}) == 16
    for r in range(32):
        for h in (0, 1):
            for n in range(keys // 32):
                for e in range(D // 16):
                    assert (k_at(r, h) ^ ((e & 7) << 5)) + n * 64 * D + (e >> 3) * 256 == k_at(32 * n + r, 2 * e + h)
            for n in range(D // 32):
                for e in range(keys // 16):
                    assert (v_at(r, h) ^ (e << 5)) + n * 64 * keys == v_at(32 * n + r, 2 * e + h)

"""GPU parity of what becomes of a score in the attentions over the paged FP8 cache, at the ends of its range, against
the binary64 oracle under its derived tolerance: caps from the smallest number to the largest."""

import numpy as np
import pytest

from .attention_util import Problem, compare, tree_mask
from .gpu_util import log

pytestmark = pytest.mark.gpu

#: new tokens of 4 heads a KV head: tiles of 16, 32 and (shared: 256, else 32) rows; the last, of 2 heads a KV head and
#: more items than short sequences may have: tiles of 256 in both divisions
NEW = [1, 9, 40]
WITH_TILES = NEW + [130]


def check(p, what, **kw):
    log(f"attention scores {what}")
    want, tol = p.oracle()
    got = p.run(**kw)
    compare(got, want, tol, what)
    return got


def problem(new, head_dim, dtype="bf16", seed=0, tree=False, slopes=False, positions=False, q_std=2.0):
    lens = [(700 if new < 130 else 90, new), (33, max(1, new // 2)), (0, new), (300 if new < 130 else 60, new)]
    heads, kv_heads = (8, 2) if new < 130 else (16, 8)
    p = Problem(lens, heads, kv_heads, head_dim, dtype=dtype, seed=100 + new + seed, q_std=q_std)
    counts = [n for _, n in lens]
    if tree:
        p.options["tree_mask"] = tree_mask(p.rng, counts)
    if slopes:
        p.options["slopes"] = np.linspace(0.01, 0.7, heads).astype(np.float32)
    if positions:
        p.options["positions"] = np.concatenate([c + p.rng.integers(0, 4, n) for c, n in lens])
    return p


def hints(new, split):
    """Bounds under which the longest sequence is shared among workgroups and joined, or not."""
    return dict(max_query_len=new, max_seq_len=100000 if split else (1000 if new < 40 else 100 if new < 130 else 256))


@pytest.mark.parametrize("cap", [1e-45, 1e-38, 1e-8, 1e-3, 128.0, 129.0, 1e3, 1e5, 1e6, 1e9, 3e38])
@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_caps_of_every_size(cap, new, head_dim):
    p = problem(new, head_dim)
    p.q[::7] = 0  # scores of exactly 0
    p.options["softcap"] = float(np.float32(cap))
    check(p, f"cap={cap} new={new} D={head_dim}", **hints(new, False))


@pytest.mark.parametrize("cap", [129.0, 250.0])
@pytest.mark.parametrize("new", NEW)
def test_scores_that_reach_a_wide_cap(cap, new):
    p = problem(new, 64, dtype="f16")
    p.scale = 4.0  # scores of about +- 100
    p.options["softcap"] = cap
    check(p, f"reached cap={cap} new={new}", **hints(new, False))


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("new", WITH_TILES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_kernel_with_a_wide_cap(dtype, head_dim, new, split):
    for tree, slopes in ((False, False), (False, True), (True, True)):
        p = problem(new, head_dim, dtype, seed=7, tree=tree, slopes=slopes, positions=tree)
        p.options["softcap"] = 1e5
        check(p, f"wide cap {dtype} D={head_dim} new={new} split={split} tree={tree}", **hints(new, split))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_a_wide_cap_where_row_tiles_are_searched(dtype, head_dim):
    lens = [((i * 7) % 40, i % 3 % 2) for i in range(60)]
    lens[20] = (11, 300)
    p = Problem(lens, 4, 2, head_dim, dtype=dtype, seed=3, pad_tokens=3)
    p.options["softcap"] = 1e5
    check(p, f"wide cap searched {dtype} D={head_dim}", max_query_len=300, max_seq_len=256)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_small_weights_of_many_keys_beside_a_large_one(dtype, head_dim, new):
    """One key with a value of 0 weighs 2^25.3 times as much as each of 3000 others with values of +-448: the output
    is theirs, and none of them may be lost."""
    from oracle import attention as oa

    ctx = 3000
    p = Problem([(ctx, new)], 8, 2, head_dim, dtype=dtype, seed=61)
    slots = oa.slots_of(p.table[0], ctx + new, p.block_size, p.num_slots)
    p.q[:] = 1
    row = 2 * head_dim
    p.kc[slots, :row] = 0
    p.vc[slots, :row] = np.where(np.arange(row) % 3 == 0, 0xFE, 0x7E)  # -448, 448
    top = slots[ctx - 1]  # the last position that every row sees
    p.kc[top, :row] = 0x38  # 1.0
    p.vc[top, :row] = 0
    p.vs = np.float32(1.0)
    p.scale = float(np.float32(25.3 * np.log(2.0) / (head_dim * float(p.ks))))
    got = check(p, f"small weights {dtype} D={head_dim} new={new}", max_query_len=new, max_seq_len=1000)
    assert np.all(got != 0)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("new", WITH_TILES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("factor", [-1.0, 0.0])
def test_negative_and_zero_scales(factor, head_dim, new, split):
    """scale < 0 turns the order of the scores round, scale = 0 makes them all 0: masks, caps and biases stay."""
    for dtype, cap, slopes, tree in (("bf16", 0.0, False, False), ("f16", 6.0, True, True), ("bf16", 1e4, False, True),
                                     ("f16", 0.0, True, False)):
        p = problem(new, head_dim, dtype, seed=13, tree=tree, slopes=slopes, positions=tree and slopes)
        p.scale *= factor
        if cap:
            p.options["softcap"] = cap
        if not tree:
            p.options["doc_start"] = np.concatenate([np.maximum(np.arange(c, c + n) - 50, 0) for c, n in p.lens])
        check(p, f"scale {factor} {dtype} D={head_dim} new={new} split={split} cap={cap} slopes={slopes} tree={tree}",
              **hints(new, split))


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("new", WITH_TILES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_moved_drafted_keys_without_a_cap(dtype, head_dim, new, split):
    """Positions of drafted tokens in the distance bias of scores that are not capped, also under a negative scale."""
    for factor in (1.0, -0.5):
        p = problem(new, head_dim, dtype, seed=17, tree=True, slopes=True, positions=True)
        p.scale *= factor
        check(p, f"moved keys {dtype} D={head_dim} new={new} split={split} factor={factor}", **hints(new, split))


@pytest.mark.parametrize("new", WITH_TILES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_queries_that_are_no_numbers_under_a_scale_of_zero(dtype, head_dim, new):
    """0 times an infinite or undefined score is undefined: those rows are NaN, the others the mean of the values."""
    p = problem(new, head_dim, dtype, seed=19)
    p.scale = 0.0
    rows = [(0, 1, np.inf), (1, 6, np.nan), (p.tokens - 1, 0, -np.inf)]
    for t, h, x in rows:
        p.q[t, h, head_dim - 3] = 0.0
    want, tol = p.oracle()
    for t, h, x in rows:
        p.q[t, h, head_dim - 3] = x
    log(f"no numbers, scale 0, {dtype} D={head_dim} new={new}")
    got = p.run(**hints(new, False))
    for t, h, _ in rows:
        assert np.isnan(got[t, h]).all(), (t, h)
        want[t, h], tol[t, h], got[t, h] = 0.0, 0.0, 0.0
    compare(got, want, tol, "other rows")

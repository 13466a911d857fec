"""GPU parity of the attentions over the 4-bit cache (nvfp4_kv_fp4_attention, nvfp4_kv_fp4_tree_attention) against the
binary64 oracle, under the tolerance derived in oracle/attention.py (codes are decoded exactly, as those of the FP8
cache are).

Slots that no request owns hold the largest bytes there are, rows of no request a sentinel, in every case."""

import numpy as np
import pytest

from .attention_util import SENTINEL, compare, pack, tree_mask
from .fp4_attention_util import Problem4
from .gpu_util import DEV, log

pytestmark = pytest.mark.gpu

DIMS = pytest.mark.parametrize("head_dim", [64, 128, 256])


def check(p, what, **kw):
    log(f"fp4 attention {what}")
    want, tol = p.oracle()
    got = p.run(**kw)
    compare(got, want, tol, what)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@DIMS
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (16, 1), (5, 5)])
def test_types_and_head_layouts(dtype, head_dim, heads, kv_heads):
    p = Problem4([(45, 7), (0, 1), (130, 1)], heads, kv_heads, head_dim, dtype=dtype, seed=heads + head_dim)
    check(p, f"{dtype} D={head_dim} H={heads}/{kv_heads}")


@pytest.mark.parametrize("ctx", [0, 1, 31, 32, 33, 127, 128, 129, 256, 513])
@pytest.mark.parametrize("new", [1, 3])
def test_lengths_around_the_steps(ctx, new):
    p = Problem4([(ctx, new)], 8, 2, 128, seed=ctx * 5 + new)
    check(p, f"ctx={ctx} new={new}")


@pytest.mark.parametrize("new", [2, 17, 64, 65, 150, 300])
@DIMS
def test_prompts(new, head_dim):
    p = Problem4([(0, new), (19, max(1, new // 2))], 4, 2, head_dim, seed=new)
    check(p, f"prompt {new} D={head_dim}")


@pytest.mark.parametrize("new,heads,kv_heads", [(11, 3, 1), (12, 8, 2), (48, 2, 2), (13, 10, 2), (24, 4, 1), (33, 4, 2), (9, 14, 2)])
@pytest.mark.parametrize("head_dim,dtype", [(64, "bf16"), (128, "f16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("ctx", [40, 1500])
def test_between_the_row_tiles(new, heads, kv_heads, head_dim, dtype, ctx):
    """33 to 48 rows in one tile and 65 to 96 in two (of 48, by the bound of the lengths, and of 32 without it); the
    second request fills a tile in part, the third has no token."""
    lens = [(ctx, new), (ctx // 3, new // 2), (ctx, 0), (0, new)]
    p = Problem4(lens, heads, kv_heads, head_dim, dtype=dtype, seed=new + ctx)
    check(p, f"{new} x {heads}/{kv_heads} D={head_dim} ctx={ctx}")
    check(p, f"{new} x {heads}/{kv_heads} D={head_dim} ctx={ctx}, long", max_seq_len=5000)
    if head_dim == 128 and dtype == "bf16":
        p.options["softcap"] = 20.0
        p.options["slopes"] = np.linspace(0.0, 0.3, heads, dtype=np.float32)
        check(p, f"{new} x {heads}/{kv_heads} with a cap and a bias, ctx={ctx}", max_seq_len=5000)
        p.options["softcap"] = 200.0
        check(p, f"{new} x {heads}/{kv_heads} with a wide cap and a bias, ctx={ctx}", max_seq_len=5000)
        del p.options["softcap"], p.options["slopes"]
    if head_dim <= 128:
        p.options["tree_mask"] = tree_mask(p.rng, [n for _, n in lens])
        check(p, f"{new} x {heads}/{kv_heads} trees, ctx={ctx}", max_seq_len=5000)


@pytest.mark.parametrize("new,head_dim", [(9, 64), (9, 128), (4, 64), (4, 256), (8, 128), (1, 128)])
@pytest.mark.parametrize("max_seq_len", [None, 5000])
def test_more_items_than_compute_units(new, head_dim, max_seq_len):
    """1040 items of up to 36 rows: a workgroup of four wavefronts for each, whatever the bound of the lengths."""
    p = Problem4([(3 + r % 150, max(1, new - r % 3)) for r in range(130)], 32, 8, head_dim, seed=5)
    check(p, f"130 requests, {4 * new} rows", max_seq_len=max_seq_len)


@pytest.mark.parametrize("new,head_dim", [(1, 64), (1, 128), (1, 256), (4, 256), (8, 64), (8, 128), (8, 256)])
@pytest.mark.parametrize("longest", [127, 128, 129, 255, 256, 257, 511, 513, 1024])
def test_few_items_of_few_steps(new, head_dim, longest):
    """Around the steps of a workgroup of eight wavefronts (256 positions), with requests that end in its first ones and one
    without a token."""
    p = Problem4([(longest - new, new), (5, new), (longest // 2, new), (100, 0)], 8, 2, head_dim, seed=longest)
    check(p, f"{new} tokens over {longest}", max_seq_len=longest)


@pytest.mark.parametrize("block_size", [1, 3, 16, 48, 64, 1000])
def test_block_sizes_and_ragged_batch(block_size):
    lens = [(0, 0), (77, 5), (0, 31), (500, 1), (0, 0), (200, 12), (3, 0)]
    p = Problem4(lens, 6, 3, 64, block_size=block_size, seed=block_size, pad_tokens=4)
    got = check(p, f"block_size={block_size}")
    assert np.all(got[p.real:] == SENTINEL)


@pytest.mark.parametrize("head_dim,scale_code", [(d, c) for d in (64, 128, 256) for c in (0x00, 0x01, 0x07, 0x08, 0x38, 0x7E)])
def test_every_code_under_small_and_large_scales(head_dim, scale_code):
    """All sixteen E2M1 codes in every place, under subnormal, zero and largest block scales, beside an ordinary
    head."""
    p = Problem4([(40, 2)], 4, 2, head_dim, seed=scale_code)
    lane = np.arange(head_dim // 2)
    for j in range(42):
        b, o = p.place(0, j)
        p.kc[b, 0, o] = ((lane + j) % 16) | (((lane * 3 + j) % 16) << 4)
        p.vc[b, 0, o] = ((lane * 5 + j) % 16) | (((lane + 7 * j) % 16) << 4)
        p.kcs[b, 0, o] = p.vcs[b, 0, o] = scale_code
        p.vcs[b, 0, o, j % (head_dim // 16)] = 0x3A  # and one block under another scale
    p.kg = np.float32({0x7E: 4000.0, 0x38: 30.0}.get(scale_code, 1.0))
    for new in (2, 600):  # the streaming kernels, and the tiled one by its bound
        check(p, f"codes under 0x{scale_code:02x}, D={head_dim}", max_query_len=new)


@pytest.mark.parametrize("softcap,bias,docs,prefix", [(5.0, False, False, False), (500.0, True, False, False),
                                                      (0.0, True, False, False), (0.0, False, True, False),
                                                      (0.0, False, False, True), (30.0, True, True, True)])
@pytest.mark.parametrize("lens", [[(0, 90), (33, 20)], [(700, 4), (300, 1)], [(300, 130), (0, 140)]])
@pytest.mark.parametrize("head_dim", [64, 256])
def test_caps_biases_and_masks(softcap, bias, docs, prefix, lens, head_dim):
    p = Problem4(lens, 4, 2, head_dim, seed=11, q_std=3.0)
    if softcap:
        p.options["softcap"] = softcap
    if bias:
        p.options["slopes"] = np.array([0.5, 0.03, 0.0, 2.0], np.float32)
    if docs:
        p.options["doc_start"] = np.concatenate([np.arange(c, c + n) // 37 * 37 for c, n in p.lens])
    if prefix:
        p.options["prefix_lens"] = np.array([c + n // 2 for c, n in p.lens])
    check(p, f"cap={softcap} bias={bias} docs={docs} prefix={prefix}")


@pytest.mark.parametrize("new", [5, 200])
def test_rows_that_see_nothing_are_zero(new):
    p = Problem4([(40, new), (0, new)], 4, 2, 128, seed=12)
    start = np.zeros(p.tokens, np.int64)
    start[::2] = 10 ** 6  # beyond every key
    start[1] = -5  # below 0: nothing hidden
    p.options["doc_start"] = start
    got = check(p, "empty rows")
    assert np.all(got[::2] == 0)


def test_more_query_rows_than_positions():
    p = Problem4([(0, 20), (0, 6)], 4, 2, 64, seed=13)
    p.seq_lens[:] = [12, 0]
    got = check(p, "short seq_lens")
    assert np.all(got[:8] == 0) and np.all(got[20:26] == 0)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new", [6, 130])
@DIMS
def test_positions_outside_the_cache_are_not_seen(tree, new, head_dim):
    p = Problem4([(100, new), (64, new), (20, new)], 4, 2, head_dim, seed=14)
    p.table[0, 2] = -3
    p.table[0, 4] = p.blocks  # the first one outside
    p.table[1, 0] = 2 ** 31 - 1
    p.table[2, :] = -1  # nothing there at all
    if tree:
        p.options["tree_mask"] = tree_mask(p.rng, [new] * 3)
    got = check(p, "bad blocks")
    assert np.all(got[2 * new:] == 0)


def test_positions_beyond_the_table():
    p = Problem4([(100, 3)], 4, 2, 64, seed=15)
    p.table = p.table[:, :4].copy()  # 64 positions
    check(p, "narrow table")
    p.table = np.zeros((1, 0), np.int64)
    got = check(p, "table of width 0")
    assert np.all(got == 0)


@pytest.mark.parametrize("new,head_dim", [(6, 64), (6, 256), (90, 128), (140, 256)])
def test_bytes_of_unseen_positions_change_nothing(new, head_dim):
    """The last positions hold other bytes, NaN scale codes among them: rows before them keep their bits."""
    p = Problem4([(20, new)], 4, 2, head_dim, seed=16)
    a = p.run()
    for j in range(20 + new - 3, 20 + new):
        b, o = p.place(0, j)
        p.kc[b, :, o] = p.vc[b, :, o] = 0xF7
        p.kcs[b, :, o] = 0x7F
        p.vcs[b, :, o] = 0xFF
    got = check(p, "other bytes behind")
    assert np.array_equal(got[: new - 3], a[: new - 3]) and not np.array_equal(got[new - 1], a[new - 1])


def test_infinite_and_nan_queries_stay_in_their_rows():
    for new in (4, 150):
        p = Problem4([(50, new)], 4, 2, 64, seed=18)
        p.q[1, 2, 3] = np.inf
        p.q[2, 1, 0] = np.nan
        log("infinite queries")
        clean = Problem4([(50, new)], 4, 2, 64, seed=18)
        want, tol = clean.oracle()
        got = p.run()
        keep = np.ones((new, 4), bool)
        keep[1, 2] = keep[2, 1] = False
        compare(got[keep], want[keep], tol[keep], "other rows")
        assert np.isnan(got[2, 1]).all() and not np.isfinite(got[1, 2]).any()


@pytest.mark.parametrize("dtype,head_dim,heads,kv_heads", [("bf16", 64, 8, 8), ("f16", 128, 8, 2), ("bf16", 256, 6, 1)])
@pytest.mark.parametrize("counts", [[1], [5, 12, 1], [64, 17], [130, 3]])
def test_trees(dtype, head_dim, heads, kv_heads, counts):
    lens = [(int(40 * (i + 1) ** 2), n) for i, n in enumerate(counts)]
    p = Problem4(lens, heads, kv_heads, head_dim, dtype=dtype, seed=sum(counts))
    p.options["tree_mask"] = tree_mask(p.rng, counts)
    check(p, f"tree {counts}")


def test_tree_without_context_and_with_empty_rows():
    p = Problem4([(0, 7), (50, 7)], 4, 2, 64, seed=20)
    m = tree_mask(p.rng, [7, 7])
    m[2] = 0
    m[9] = 0
    p.options["tree_mask"] = m
    got = check(p, "tree with empty rows")
    assert np.all(got[2] == 0) and np.any(got[9] != 0)


@pytest.mark.parametrize("with_positions", [False, True])
@pytest.mark.parametrize("new", [9, 80])
def test_tree_cap_and_bias(with_positions, new):
    p = Problem4([(90, new), (300, 4)], 4, 2, 128, seed=23, q_std=2.0)
    p.options["tree_mask"] = tree_mask(p.rng, [new, 4])
    p.options["softcap"] = 20.0
    p.options["slopes"] = np.array([0.4, 0.01, 1.0, 0.2], np.float32)
    if with_positions:
        p.options["positions"] = np.concatenate([90 + p.rng.integers(0, 5, new), 300 + p.rng.integers(0, 3, 4)])
    check(p, f"tree bias positions={with_positions}")


def test_causal_chain_as_a_tree_equals_the_prompt_form():
    p = Problem4([(200, 8), (31, 3)], 8, 2, 128, seed=24)
    a = p.run()
    bits = np.zeros((11, 64), bool)
    bits[:8, :8] = np.tril(np.ones((8, 8), bool))
    bits[8:, :3] = np.tril(np.ones((3, 3), bool))
    p.options["tree_mask"] = pack(bits)
    assert np.array_equal(a, p.run())


@pytest.mark.parametrize("max_query_len,max_seq_len", [(1, 1), (1, 10 ** 9), (10 ** 6, 1), (10 ** 6, 10 ** 9), (30, 2000)])
def test_bounds_only_divide_the_work(max_query_len, max_seq_len):
    p = Problem4([(900, 30), (5, 2), (0, 0), (64, 1)], 8, 2, 128, seed=25)
    check(p, f"bounds {max_query_len} {max_seq_len}", max_query_len=max_query_len, max_seq_len=max_seq_len)


@pytest.mark.parametrize("lens", [[(3000, 1)], [(2500, 20), (900, 3)], [(0, 700)], [(1500, 300), (10, 40)]])
@DIMS
def test_longer_contexts(lens, head_dim):
    p = Problem4(lens, 4, 1, head_dim, seed=26, block_size=48)
    check(p, f"{lens} D={head_dim}")


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("mods", [False, True])
@pytest.mark.parametrize("new", [1, 9, 40])
@DIMS
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_kernel_and_division(dtype, head_dim, new, mods, split):
    """4 heads a KV head: 4, 36 and 160 rows, so tiles of 16, 32 and 256; a workgroup per item, and shared
    among workers and joined; plain scores, and capped and biased ones; prompts and trees."""
    lens = [(700, new), (33, max(1, new // 2)), (0, new), (300, new)]
    for tree in (False, True):
        p = Problem4(lens, 8, 2, head_dim, dtype=dtype, seed=50 + new, q_std=2.0)
        if mods:
            p.options["softcap"] = 12.0
            p.options["slopes"] = np.linspace(0.01, 0.7, 8).astype(np.float32)
        if tree:
            counts = [n for _, n in lens]
            p.options["tree_mask"] = tree_mask(p.rng, counts)
            if mods:
                p.options["positions"] = np.concatenate([c + p.rng.integers(0, 4, n) for c, n in lens])
        hint = 100000 if split else (1000 if new < 40 else 100)
        check(p, f"{dtype} D={head_dim} new={new} mods={mods} split={split} tree={tree}", max_query_len=new,
              max_seq_len=hint)


@pytest.mark.parametrize("requests,longest", [(60, 300), (200, 290)])
@DIMS
def test_one_prompt_among_single_tokens(requests, longest, head_dim):
    for place in (0, requests // 2, requests - 1):
        lens = [((i * 7) % 40, i % 3 % 2) for i in range(requests)]
        lens[place] = (11, longest)
        p = Problem4(lens, 4, 2, head_dim, seed=place + longest, pad_tokens=3)
        check(p, f"{requests} requests, one of {longest} at {place}, D={head_dim}", max_query_len=300, max_seq_len=256)


@pytest.mark.parametrize("scale", [0.0, -0.2])
@pytest.mark.parametrize("new", [3, 150])
def test_scales_that_are_zero_or_negative(scale, new):
    p = Problem4([(60, new)], 4, 2, 128, seed=37)
    p.scale = float(np.float32(scale))
    check(p, f"scale {scale}")


def test_strided_query_and_output():
    """q as the first columns of a fused qkv row, out as a window, in place, and head-major storage."""
    import torch

    p = Problem4([(50, 9), (0, 33)], 4, 2, 64, seed=28)
    want, tol = p.oracle()
    d = p.device()
    T, H, D = d["q"].shape
    fused = torch.full((T, (H + 4) * D), 3.0, dtype=d["q"].dtype, device=DEV)
    fused[:, : H * D] = d["q"].reshape(T, H * D)
    q = fused[:, : H * D].unflatten(1, (H, D))
    wide = torch.full((T, H + 2, D + 8), SENTINEL, dtype=d["q"].dtype, device=DEV)
    log("strided q and out")
    compare(p.run(q=q, out=wide[:, 1:H + 1, :D]), want, tol, "window")
    untouched = wide.clone()
    untouched[:, 1:H + 1, :D] = SENTINEL
    assert bool((untouched == SENTINEL).all())
    qh = d["q"].transpose(0, 1).contiguous().transpose(0, 1)
    oh = torch.full((H, T, D), SENTINEL, dtype=d["q"].dtype, device=DEV).transpose(0, 1)
    compare(p.run(q=qh, out=oh), want, tol, "head-major")
    compare(p.run(q=q, out=q), want, tol, "in place")
    assert bool((fused[:, H * D:] == 3.0).all())


def test_rows_beyond_32_bits_of_bytes():
    """A cache whose last blocks lie 5 GB of codes after its first."""
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    p = Problem4([(60, 3)], 8, 4, 256, seed=31)
    want, tol = p.oracle()
    d = p.device()
    first = 5 * 2 ** 30 // (4 * 16 * 128)
    log("5 GB of codes")
    for name in ("key_codes", "key_scales", "value_codes", "value_scales"):
        big = torch.empty((first + p.blocks, *d[name].shape[1:]), dtype=torch.uint8, device=DEV)
        big[first:] = d[name]
        d[name] = big
    d["block_table"] = torch.where(d["block_table"] >= 0, d["block_table"] + first, d["block_table"])
    for new in (3, 600):
        out = nv.nvfp4_kv_fp4_attention(**{**d, "max_query_len": new})
        torch.cuda.synchronize()
        compare(out.double().cpu().numpy(), want, tol, "5 GB of codes")


def test_results_repeat_bit_for_bit():
    p = Problem4([(1800, 5), (40, 1), (900, 64)], 8, 2, 128, seed=30)
    a = p.run(max_query_len=5)
    for _ in range(3):
        assert np.array_equal(a, p.run(max_query_len=5))


def test_empty_calls():
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    p = Problem4([(20, 2)], 2, 1, 64, seed=32)
    d = p.device()
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    none = {**d, "q": d["q"][:0], "out": d["out"][:0], "query_start": i32(2)}
    assert nv.nvfp4_kv_fp4_attention(**none).shape[0] == 0
    nobody = {**d, "query_start": i32(1), "seq_lens": i32(0), "block_table": d["block_table"][:0]}
    out = nv.nvfp4_kv_fp4_attention(**nobody)
    torch.cuda.synchronize()
    assert bool((out == SENTINEL).all())


def test_another_stream_and_captured_graphs():
    """On a side stream; captured (two graphs, each with its own workspace) and replayed with eager work between the
    replays, on inputs that change in place."""
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    p = Problem4([(1500, 2), (700, 2)], 8, 2, 128, seed=33)
    t = Problem4([(1500, 2), (700, 2)], 8, 2, 128, seed=33)
    t.options["tree_mask"] = tree_mask(t.rng, [2, 2])
    want, tol = p.oracle()
    twant, ttol = t.oracle()
    log("side stream")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        d, td = p.device(), t.device()
        out = nv.nvfp4_kv_fp4_attention(**d)
    side.synchronize()
    compare(out.double().cpu().numpy(), want, tol, "side stream")
    log("graphs")
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(ga):
        nv.nvfp4_kv_fp4_attention(**d)
    with torch.cuda.graph(gb):
        nv.nvfp4_kv_fp4_tree_attention(**td)
    q0 = d["q"].clone()
    for k in range(4):
        d["out"].fill_(SENTINEL)
        td["out"].fill_(SENTINEL)
        d["q"].copy_(q0 if k % 2 == 0 else -q0)
        ga.replay()
        gb.replay()
        eager = nv.nvfp4_kv_fp4_attention(**{**d, "out": None})
        torch.cuda.synchronize()
        assert bool((d["out"] == eager).all())
        compare(td["out"].double().cpu().numpy(), twant, ttol, f"tree replay {k}")
        if k % 2 == 0:
            compare(d["out"].double().cpu().numpy(), want, tol, f"replay {k}")


def test_two_streams_at_once():
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    ps = [Problem4([(1200 + 300 * k, 3)], 8, 2, 128, seed=40 + k) for k in range(2)]
    ds = [p.device() for p in ps]
    refs = [p.oracle() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    log("two streams")
    outs = [[] for _ in ps]
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[k].append(nv.nvfp4_kv_fp4_attention(**{**ds[k], "out": None}))
    torch.cuda.synchronize()
    for k, (want, tol) in enumerate(refs):
        for o in outs[k]:
            assert bool((o == outs[k][0]).all())
        compare(outs[k][0].double().cpu().numpy(), want, tol, f"stream {k}")


@pytest.mark.parametrize("head_dim", [64, 256])
@pytest.mark.parametrize("max_query_len,new", [(1, 6), (3, 9), (None, 40)])
def test_more_pieces_than_a_wavefront_joins(max_query_len, new, head_dim):
    """Two long requests over all workgroups: more than 16 pieces an item, and more rows than the bound said."""
    p = Problem4([(9000, new), (5000, 1)], 8, 2, head_dim, seed=31)
    check(p, f"{new} tokens said to be {max_query_len}", max_query_len=max_query_len)

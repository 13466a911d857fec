"""GPU parity of the attentions over the paged FP8 cache (nvfp4_kv_fp8_attention,
nvfp4_kv_fp8_tree_attention) against the binary64 oracle, under its derived tolerance.

Slots that no request owns hold NaN codes, rows of no request a sentinel, in every case."""

import numpy as np
import pytest

from .attention_util import SENTINEL, Problem, compare, pack, tree_mask
from .gpu_util import DEV, log

pytestmark = pytest.mark.gpu


def check(p, what, **kw):
    log(f"attention {what}")
    want, tol = p.oracle()
    got = p.run(**kw)
    compare(got, want, tol, what)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (16, 1), (5, 5)])
def test_types_and_head_layouts(dtype, head_dim, heads, kv_heads):
    p = Problem([(45, 7), (0, 1), (130, 1)], heads, kv_heads, head_dim, dtype=dtype, seed=heads + head_dim)
    check(p, f"{dtype} D={head_dim} H={heads}/{kv_heads}")


@pytest.mark.parametrize("ctx", [0, 1, 30, 31, 32, 33, 127, 128, 129, 255, 256, 300, 513])
@pytest.mark.parametrize("new", [1, 3])
def test_lengths_around_the_steps(ctx, new):
    p = Problem([(ctx, new)], 8, 2, 128, seed=ctx * 5 + new)
    check(p, f"ctx={ctx} new={new}")


@pytest.mark.parametrize("new", [2, 9, 17, 40, 64, 65, 150, 300])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_prompts(new, head_dim):
    p = Problem([(0, new), (19, max(1, new // 2))], 4, 2, head_dim, seed=new)
    check(p, f"prompt {new} D={head_dim}")


@pytest.mark.parametrize("block_size", [1, 3, 16, 48, 64, 1000])
def test_block_sizes_and_ragged_batch(block_size):
    lens = [(0, 0), (77, 5), (0, 31), (500, 1), (0, 0), (200, 12), (3, 0)]
    p = Problem(lens, 6, 3, 64, block_size=block_size, seed=block_size, pad_tokens=4)
    got = check(p, f"block_size={block_size}")
    assert np.all(got[p.real:] == SENTINEL)


def test_many_requests_of_mixed_lengths():
    rng = np.random.default_rng(3)
    lens = [(int(rng.integers(0, 400)) if i % 3 else 0, int(rng.integers(0, 4))) for i in range(300)]
    p = Problem(lens, 2, 1, 64, seed=4)
    check(p, "300 requests")


@pytest.mark.parametrize("softcap,bias,docs,prefix", [(5.0, False, False, False), (0.0, True, False, False),
                                                      (0.0, False, True, False), (0.0, False, False, True),
                                                      (30.0, True, True, True)])
@pytest.mark.parametrize("lens", [[(0, 90), (33, 20)], [(700, 4), (300, 1)]])
@pytest.mark.parametrize("head_dim", [64, 256])
def test_caps_biases_and_masks(softcap, bias, docs, prefix, lens, head_dim):
    p = Problem(lens, 4, 2, head_dim, seed=11, q_std=3.0)
    if softcap:
        p.options["softcap"] = softcap
    if bias:
        p.options["slopes"] = np.array([0.5, 0.03, 0.0, 2.0], np.float32)
    if docs:
        start = []
        for c, n in p.lens:
            pos = np.arange(c, c + n)
            start.append(pos // 37 * 37)
        p.options["doc_start"] = np.concatenate(start)
    if prefix:
        p.options["prefix_lens"] = np.array([c + n // 2 for c, n in p.lens])
    check(p, f"cap={softcap} bias={bias} docs={docs} prefix={prefix}")


@pytest.mark.parametrize("new", [5, 200])
def test_rows_that_see_nothing_are_zero(new):
    p = Problem([(40, new), (0, new)], 4, 2, 128, seed=12)
    start = np.zeros(p.tokens, np.int64)
    start[::2] = 10 ** 6  # beyond every key
    start[1] = -5  # below 0: nothing hidden
    p.options["doc_start"] = start
    got = check(p, "empty rows")
    assert np.all(got[::2] == 0)


def test_more_query_rows_than_positions():
    """seq_lens below the number of query rows: the rows before position 0 see nothing."""
    p = Problem([(0, 20), (0, 6)], 4, 2, 64, seed=13)
    p.seq_lens[:] = [12, 0]
    got = check(p, "short seq_lens")
    assert np.all(got[:8] == 0) and np.all(got[20:26] == 0)


@pytest.mark.parametrize("tree", [False, True])
def test_positions_outside_the_cache_are_not_seen(tree):
    p = Problem([(100, 6), (64, 6), (20, 6)], 4, 2, 64, seed=14)
    p.table[0, 2] = -3
    p.table[0, 4] = p.num_slots  # far outside
    p.table[1, 0] = 2 ** 31 - 1
    p.table[2, :] = -1  # nothing there at all
    if tree:
        p.options["tree_mask"] = tree_mask(p.rng, [6, 6, 6])
    got = check(p, "bad blocks")
    assert np.all(got[12:18] == 0)


def test_positions_beyond_the_table():
    p = Problem([(100, 3)], 4, 2, 64, seed=15)
    p.table = p.table[:, :4].copy()  # 64 positions
    check(p, "narrow table")
    p.table = np.zeros((1, 0), np.int64)
    got = check(p, "table of width 0")
    assert np.all(got == 0)


@pytest.mark.parametrize("new,head_dim", [(6, 64), (6, 256), (90, 128)])
def test_nan_codes_reach_only_the_rows_that_see_them(new, head_dim):
    p = Problem([(20, new)], 4, 2, head_dim, seed=16)
    from oracle import attention as oa

    s = oa.slots_of(p.table[0], 20 + new, p.block_size, p.num_slots)
    p.vc[s[20 + new - 2], 5] = 0xFF  # the last position but one: only the last two rows see it
    p.vc[s[20 + new - 1], head_dim + 3] = 0x7F  # the last position, the other KV head
    p.kc[s[20 + new - 1], 2] = 0x7F  # and a key
    got = check(p, "NaN codes")
    assert np.isnan(got).any() and not np.isnan(got[: new - 2]).any()


def test_nan_codes_in_drafted_trees():
    p = Problem([(33, 5)], 2, 1, 128, seed=17)
    from oracle import attention as oa

    bits = np.zeros((5, 64), bool)
    for i, row in enumerate([[0], [0, 1], [0, 2], [0, 1, 3], []]):
        bits[i, row] = True
    p.options["tree_mask"] = pack(bits)
    s = oa.slots_of(p.table[0], 38, p.block_size, p.num_slots)
    p.vc[s[33 + 1], :] = 0x7F  # drafted token 1: seen by rows 1 and 3
    got = check(p, "NaN in a tree")
    assert np.isnan(got[[1, 3]]).all() and not np.isnan(got[[0, 2, 4]]).any()


def test_infinite_and_nan_queries_stay_in_their_rows():
    p = Problem([(50, 4)], 4, 2, 64, seed=18)
    p.q[1, 2, 3] = np.inf
    p.q[2, 1, 0] = np.nan
    log("infinite queries")
    clean = Problem([(50, 4)], 4, 2, 64, seed=18)
    want, tol = clean.oracle()
    got = p.run()
    keep = np.ones((4, 4), bool)
    keep[1, 2] = keep[2, 1] = False
    compare(got[keep], want[keep], tol[keep], "other rows")
    assert np.isnan(got[2, 1]).all() and not np.isfinite(got[1, 2]).any()


@pytest.mark.parametrize("dtype,head_dim,heads,kv_heads", [("bf16", 64, 8, 8), ("f16", 128, 8, 2), ("bf16", 256, 6, 1)])
@pytest.mark.parametrize("counts", [[1], [5, 12, 1], [64, 17], [130, 3]])
def test_trees(dtype, head_dim, heads, kv_heads, counts):
    lens = [(int(40 * (i + 1) ** 2), n) for i, n in enumerate(counts)]
    p = Problem(lens, heads, kv_heads, head_dim, dtype=dtype, seed=sum(counts))
    p.options["tree_mask"] = tree_mask(p.rng, counts)
    check(p, f"tree {counts}")


def test_tree_without_context_and_with_empty_rows():
    p = Problem([(0, 7), (50, 7)], 4, 2, 64, seed=20)
    m = tree_mask(p.rng, [7, 7])
    m[2] = 0
    m[9] = 0
    p.options["tree_mask"] = m
    got = check(p, "tree with empty rows")
    assert np.all(got[2] == 0) and np.any(got[9] != 0)


def test_tree_bits_beyond_the_words_and_beyond_the_tokens():
    p = Problem([(10, 80)], 2, 1, 64, seed=21)
    bits = p.rng.random((80, 64)) < 0.5  # one word: drafted tokens 64 .. 79 are seen by nobody
    p.options["tree_mask"] = pack(bits)
    check(p, "one word for 80 tokens")
    p = Problem([(10, 5)], 2, 1, 64, seed=22)
    p.options["tree_mask"] = np.full((5, 3), -1, np.int64)  # every bit set
    check(p, "all bits set")


@pytest.mark.parametrize("with_positions", [False, True])
def test_tree_cap_and_bias(with_positions):
    p = Problem([(90, 9), (300, 4)], 4, 2, 128, seed=23, q_std=2.0)
    p.options["tree_mask"] = tree_mask(p.rng, [9, 4])
    p.options["softcap"] = 20.0
    p.options["slopes"] = np.array([0.4, 0.01, 1.0, 0.2], np.float32)
    if with_positions:
        p.options["positions"] = np.concatenate([90 + p.rng.integers(0, 5, 9), 300 + p.rng.integers(0, 3, 4)])
    check(p, f"tree bias positions={with_positions}")


def test_causal_chain_as_a_tree_equals_the_prompt_form():
    lens = [(200, 8), (31, 3)]
    p = Problem(lens, 8, 2, 128, seed=24)
    a = p.run()
    bits = np.zeros((11, 64), bool)
    bits[:8, :8] = np.tril(np.ones((8, 8), bool))
    bits[8:, :3] = np.tril(np.ones((3, 3), bool))
    p.options["tree_mask"] = pack(bits)
    want, tol = p.oracle()
    b = p.run()
    compare(b, want, tol, "chain")
    assert np.array_equal(a, b)


@pytest.mark.parametrize("max_query_len,max_seq_len", [(1, 1), (1, 10 ** 9), (10 ** 6, 1), (10 ** 6, 10 ** 9), (30, 2000)])
def test_bounds_only_divide_the_work(max_query_len, max_seq_len):
    p = Problem([(900, 30), (5, 2), (0, 0), (64, 1)], 8, 2, 128, seed=25)
    check(p, f"bounds {max_query_len} {max_seq_len}", max_query_len=max_query_len, max_seq_len=max_seq_len)


@pytest.mark.parametrize("lens", [[(3000, 1)], [(2500, 20), (900, 3)], [(0, 700)], [(1500, 300), (10, 40)]])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_longer_contexts(lens, head_dim):
    p = Problem(lens, 4, 1, head_dim, seed=26, block_size=48)
    check(p, f"{lens} D={head_dim}")


def test_growing_scores_move_the_reference():
    """Keys whose scores rise along the sequence: the running reference is raised again and again, and
    early contributions vanish."""
    p = Problem([(600, 2)], 2, 1, 64, seed=27, q_std=1.0)
    from oracle import attention as oa

    s = oa.slots_of(p.table[0], 602, p.block_size, p.num_slots)
    ramp = np.linspace(-1, 1, 602)[:, None] * np.sign(p.q[1, 0])[None, :] * 60
    from .attention_util import _encode

    p.kc[s, :64] = _encode(ramp)
    check(p, "rising scores")
    p.kc[s, :64] = _encode(ramp[::-1].copy())
    check(p, "falling scores")


def test_strided_query_and_output():
    """q as the first columns of a fused qkv row, out as a window, and head-major storage of both."""
    import torch

    p = Problem([(50, 9), (0, 33)], 4, 2, 64, seed=28)
    want, tol = p.oracle()
    d = p.device()
    T, H, D = d["q"].shape
    fused = torch.full((T, (H + 4) * D), 3.0, dtype=d["q"].dtype, device=DEV)
    fused[:, : H * D] = d["q"].reshape(T, H * D)
    wide = torch.full((T, H + 2, D + 8), SENTINEL, dtype=d["q"].dtype, device=DEV)
    log("strided q and out")
    got = p.run(q=fused[:, : H * D].unflatten(1, (H, D)), out=wide[:, 1:H + 1, :D])
    compare(got, want, tol, "window")
    untouched = wide.clone()
    untouched[:, 1:H + 1, :D] = SENTINEL
    assert bool((untouched == SENTINEL).all())
    qh = d["q"].transpose(0, 1).contiguous().transpose(0, 1)
    oh = torch.full((H, T, D), SENTINEL, dtype=d["q"].dtype, device=DEV).transpose(0, 1)
    compare(p.run(q=qh, out=oh), want, tol, "head-major")
    one = d["q"][:, :1].expand(T, H, D)  # one head's query for all heads: stride 0
    same = Problem([(50, 9), (0, 33)], 4, 2, 64, seed=28)
    same.q = np.repeat(p.q[:, :1], H, axis=1)
    want, tol = same.oracle()
    compare(p.run(q=one), want, tol, "broadcast query")


def test_wide_cache_rows():
    p = Problem([(70, 4)], 4, 2, 64, seed=29, cache_pad=48)
    check(p, "padded cache rows")


def test_results_repeat_bit_for_bit():
    p = Problem([(1800, 5), (40, 1), (900, 64)], 8, 2, 128, seed=30)
    a = p.run(max_query_len=5)
    for _ in range(3):
        assert np.array_equal(a, p.run(max_query_len=5))


def test_offsets_beyond_32_bits():
    """A cache whose last rows lie 5 GB after its first."""
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    p = Problem([(60, 3)], 2, 1, 64, seed=31)
    want, tol = p.oracle()
    d = p.device()
    pitch, bs = 65536, p.block_size
    slots = 80000 // bs * bs  # 5.2 GB a tensor
    first = slots // bs - p.num_slots // bs
    log("5 GB cache")
    for name in ("key_cache", "value_cache"):
        big = torch.empty((slots, pitch), dtype=torch.uint8, device=DEV)
        big[first * bs:, :64] = d[name]
        d[name] = big[:, :64]
    d["block_table"] = torch.where(d["block_table"] >= 0, d["block_table"] + first, d["block_table"])
    out = nv.nvfp4_kv_fp8_attention(**d)
    torch.cuda.synchronize()
    compare(out.double().cpu().numpy(), want, tol, "5 GB cache")


def test_empty_calls():
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    p = Problem([(20, 2)], 2, 1, 64, seed=32)
    d = p.device()
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    none = {**d, "q": d["q"][:0], "out": d["out"][:0], "query_start": i32(2)}
    assert nv.nvfp4_kv_fp8_attention(**none).shape[0] == 0
    nobody = {**d, "query_start": i32(1), "seq_lens": i32(0), "block_table": d["block_table"][:0]}
    out = nv.nvfp4_kv_fp8_attention(**nobody)
    torch.cuda.synchronize()
    assert bool((out == SENTINEL).all())


def test_another_stream_and_captured_graphs():
    """On a side stream; captured (two graphs, each with its own workspace) and replayed with eager
    work between the replays, on inputs that change in place."""
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    p = Problem([(1500, 2), (700, 2)], 8, 2, 128, seed=33)
    t = Problem([(1500, 2), (700, 2)], 8, 2, 128, seed=33)
    t.options["tree_mask"] = tree_mask(t.rng, [2, 2])
    want, tol = p.oracle()
    twant, ttol = t.oracle()
    log("side stream")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        d, td = p.device(), t.device()
        out = nv.nvfp4_kv_fp8_attention(**d)
    side.synchronize()
    compare(out.double().cpu().numpy(), want, tol, "side stream")
    log("graphs")
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(ga):
        nv.nvfp4_kv_fp8_attention(**d)
    with torch.cuda.graph(gb):
        nv.nvfp4_kv_fp8_tree_attention(**td)
    q0 = d["q"].clone()
    for k in range(4):
        d["out"].fill_(SENTINEL)
        td["out"].fill_(SENTINEL)
        d["q"].copy_(q0 if k % 2 == 0 else -q0)
        ga.replay()
        gb.replay()
        eager = nv.nvfp4_kv_fp8_attention(**{**d, "out": None})
        torch.cuda.synchronize()
        assert bool((d["out"] == eager).all())
        compare(td["out"].double().cpu().numpy(), twant, ttol, f"tree replay {k}")
        if k % 2 == 0:
            compare(d["out"].double().cpu().numpy(), want, tol, f"replay {k}")


def test_two_streams_at_once():
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    ps = [Problem([(1200 + 300 * k, 3)], 8, 2, 128, seed=40 + k) for k in range(2)]
    ds = [p.device() for p in ps]
    refs = [p.oracle() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    log("two streams")
    outs = [[] for _ in ps]
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[k].append(nv.nvfp4_kv_fp8_attention(**{**ds[k], "out": None}))
    torch.cuda.synchronize()
    for k, (want, tol) in enumerate(refs):
        for o in outs[k]:
            assert bool((o == outs[k][0]).all())
        compare(outs[k][0].double().cpu().numpy(), want, tol, f"stream {k}")


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("mods", [False, True])
@pytest.mark.parametrize("new", [1, 9, 40])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_kernel_and_division(dtype, head_dim, new, mods, split):
    """4 heads a KV head: 4, 36 and 160 rows, so tiles of 16, 32 and 256; a workgroup per item, and shared
    among workers and joined; plain scores, and capped and biased ones; prompts and trees."""
    lens = [(700, new), (33, max(1, new // 2)), (0, new), (300, new)]
    for tree in (False, True):
        p = Problem(lens, 8, 2, head_dim, dtype=dtype, seed=50 + new, q_std=2.0)
        if mods:
            p.options["softcap"] = 12.0
            p.options["slopes"] = np.linspace(0.01, 0.7, 8).astype(np.float32)
        if tree:
            counts = [n for _, n in lens]
            p.options["tree_mask"] = tree_mask(p.rng, counts)
            if mods:
                p.options["positions"] = np.concatenate([c + p.rng.integers(0, 4, n) for c, n in lens])
        # a row tile of 256 is shared where the context is most of the work
        hint = 100000 if split else (1000 if new < 40 else 100)
        check(p, f"{dtype} D={head_dim} new={new} mods={mods} split={split} tree={tree}", max_query_len=new,
              max_seq_len=hint)


@pytest.mark.parametrize("requests,new", [(300, 2), (700, 1), (600, 60)])
def test_more_requests_than_threads_share_the_work(requests, new):
    rng = np.random.default_rng(requests)
    lens = [(int(rng.integers(0, 60)), int(rng.integers(0, new + 1))) for _ in range(requests)]
    lens[requests // 2] = (2000, new)
    p = Problem(lens, 2, 1, 64, seed=5)
    check(p, f"{requests} requests shared", max_query_len=new, max_seq_len=10 ** 6)


def test_lengths_beyond_the_table_end_in_time():
    """seq_lens far beyond what the table holds (left over from another batch): the keys that the table
    has are used, positions count from the length given."""
    p = Problem([(60, 2), (40, 30)], 4, 2, 64, seed=34)
    p.table = p.table[:, :3].copy()
    want, tol = p.oracle()
    huge = p.seq_lens.copy()
    huge[0] = 2 ** 31 - 1  # every key of the table lies below both rows
    p.seq_lens = np.array([48 + 2, huge[1]])  # the oracle's loops: the same 48 keys, all of them seen
    want, tol = p.oracle()
    d = p.device()
    import torch

    d["seq_lens"] = torch.tensor([2 ** 31 - 1, int(huge[1])], dtype=torch.int32, device=DEV)
    for hint in (64, 10 ** 6):
        log(f"huge length hint={hint}")
        d["out"].fill_(SENTINEL)
        compare(p.run(**{**d, "max_seq_len": hint}), want, tol, f"hint {hint}")


def test_padding_without_requests():
    p = Problem([(5, 0), (9, 0)], 4, 2, 64, seed=35, pad_tokens=6)
    for hint in (64, 10 ** 6):
        got = check(p, "no tokens", max_seq_len=hint)
        assert np.all(got == SENTINEL)


def test_rows_before_the_first_request_and_default_bounds():
    """query_start that begins above 0, and no bounds given."""
    p = Problem([(30, 1)] * 40, 8, 2, 128, seed=36, pad_tokens=3)
    p.query_start = p.query_start + 2
    got = check(p, "offset rows")
    assert np.all(got[:2] == SENTINEL) and np.all(got[42:] == SENTINEL)


@pytest.mark.parametrize("requests,longest,hint", [(60, 300, 300), (700, 300, 300), (60, 700, 300), (200, 290, 100000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("mods", [False, True])
def test_one_prompt_among_single_tokens(requests, longest, hint, dtype, head_dim, mods):
    """Few of the row tiles that the longest request's bound allows exist: workgroups find theirs from
    the lengths.  First, in the middle and last; bounds below and above the truth."""
    for place in (0, requests // 2, requests - 1):
        lens = [((i * 7) % 40, i % 3 % 2) for i in range(requests)]
        lens[place] = (11, longest)
        p = Problem(lens, 4, 2, head_dim, dtype=dtype, seed=place + longest, pad_tokens=3)
        if mods:
            p.options["softcap"] = 20.0
        check(p, f"{requests} requests, one of {longest} at {place}, D={head_dim}", max_query_len=hint, max_seq_len=256)


@pytest.mark.parametrize("new,hint", [(1, 64), (1, 2 ** 31 - 1), (200, 64), (200, 2 ** 31 - 1)])
def test_positions_near_31_bits(new, hint):
    """All table columns name one block of 2^20 slots; the documents begin close below the last position
    that is looked at, 2047 * 2^20, and the request is longer still."""
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    log(f"positions near 2^31, new={new} hint={hint}")
    bs, D, heads = 1 << 20, 64, 2
    g = torch.Generator().manual_seed(new)
    end = 2047 * bs
    tail = 300  # the slots of the positions before `end` are the block's last ones
    codes = torch.randint(0, 0x78, (2, tail, D), generator=g, dtype=torch.uint8)
    kc = torch.full((bs, D), 0x7F, dtype=torch.uint8, device=DEV)  # NaN codes elsewhere
    vc = torch.full((bs, D), 0x7F, dtype=torch.uint8, device=DEV)
    kc[-tail:], vc[-tail:] = codes[0].to(DEV), codes[1].to(DEV)
    q = torch.randn(new, heads, D, generator=g).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    one = torch.tensor([0.01], device=DEV)
    first = end - 1 - torch.arange(new) % (tail - 10)
    out = nv.nvfp4_kv_fp8_attention(
        q.to(DEV), kc, vc, one, one, torch.zeros(1, 2048, **i32), torch.tensor([0, new], **i32),
        torch.tensor([2 ** 31 - 1], **i32), block_size=bs, num_kv_heads=1, doc_start=first.to(**i32),
        max_seq_len=hint)
    value = codes.view(torch.float8_e4m3fn).double() * torch.tensor([0.01]).double()
    x = (q.double().reshape(new * heads, D) @ value[0].t().contiguous()) * D ** -0.5
    hidden = torch.arange(end - tail, end)[None, :] < first.repeat_interleave(heads)[:, None]
    p = torch.softmax(x.masked_fill(hidden, float("-inf")), dim=1)
    want = (p @ value[1]).reshape(new, heads, D)
    mean = (p @ value[1].abs()).reshape(new, heads, D)
    # bf16 half step of the result and FP16 half step of each weight; the scores' FP32 sums of 64 products
    # (|x| <= 64 * |q| * 4.5 / 8 < 150, off by at most 64 * 2^-24 * 150 < 2^-10) twice
    tol = want.abs() * 2 ** -8 + mean * (2 ** -11 + 2 ** -9) + 2 ** -20
    assert bool(((out.cpu().double() - want).abs() <= tol).all())

"""GPU parity of nvfp4_kv_block_tables with the oracle (every output exactly), and the serving steps
that use it: tables, store, prompt attention, then drafted trees, over one cache."""

import numpy as np
import pytest

import oracle
from oracle import attention as oa

from .attention_util import EPS, compare, to_type, tree_mask, unpack
from .gpu_util import DEV, log, scalar

pytestmark = pytest.mark.gpu


def _run(ctx, new, free, table, bs, max_tokens, start=None):
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).to(DEV)  # noqa: E731
    t = i32(table)
    got = nv.nvfp4_kv_block_tables(i32(ctx), i32(new), i32(free), t, bs, max_tokens,
                                   None if start is None else i32([start]))
    torch.cuda.synchronize()
    return [g.cpu().numpy() for g in got] + [t.cpu().numpy()]


def _check(ctx, new, free, table, bs, max_tokens, start=None):
    got = _run(ctx, new, free, table, bs, max_tokens, start)
    want = oa.block_tables(ctx, new, free, table, bs, max_tokens, start or 0)
    names = ("slot_mapping", "positions", "query_start", "seq_lens", "blocks_needed", "block_table")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(np.asarray(g).reshape(-1), np.asarray(w).reshape(-1)), name


def _case(rng, R, ctx_max, new_max, bs, spare=5):
    ctx = rng.integers(0, ctx_max + 1, R)
    new = rng.integers(0, new_max + 1, R)
    need = -(-(ctx + new) // bs)
    have = -(-ctx // bs)
    width = int(need.max(initial=0)) + 1
    ids = rng.permutation(int(need.sum()) + spare)
    table = np.full((R, width), -1, np.int64)
    at = 0
    for r in range(R):
        table[r, : have[r]] = ids[at: at + have[r]]
        at += have[r]
    return ctx, new, ids[at:], table


@pytest.mark.parametrize("R", [0, 1, 2, 63, 64, 65, 511, 512, 513, 1500])
@pytest.mark.parametrize("bs", [1, 16, 48])
def test_against_the_oracle(R, bs):
    rng = np.random.default_rng(R * 3 + bs)
    ctx, new, free, table = _case(rng, R, 200, 9, bs)
    log(f"tables R={R} bs={bs}")
    _check(ctx, new, free, table, bs, int(new.sum()) + 13)


def test_largest_number_of_requests():
    rng = np.random.default_rng(5)
    ctx, new, free, table = _case(rng, 8192, 50, 3, 16)
    log("tables 8192 requests")
    _check(ctx, new, free, table, 16, int(new.sum()) + 1)


def test_long_prompts():
    rng = np.random.default_rng(6)
    ctx, new, free, table = _case(rng, 5, 40000, 30000, 16)
    log("tables long prompts")
    _check(ctx, new, free, table, 16, int(new.sum()))


def test_exhausted_free_list_narrow_table_and_dropped_tokens():
    rng = np.random.default_rng(7)
    ctx, new, free, table = _case(rng, 20, 100, 60, 16)
    log("tables exhausted")
    _check(ctx, new, free[:7], table, 16, int(new.sum()))
    _check(ctx, new, free[:0], table, 16, int(new.sum()))
    _check(ctx, new, free, table[:, :3].copy(), 16, int(new.sum()))
    _check(ctx, new, free, np.zeros((20, 0), np.int64), 16, int(new.sum()))
    _check(ctx, new, free, table, 16, int(new.sum()) // 2)
    _check(ctx, new, free, table, 16, 0)


def test_free_start_and_negative_lengths():
    rng = np.random.default_rng(8)
    ctx, new, free, table = _case(rng, 9, 60, 40, 8)
    log("tables free_start")
    _check(ctx, new, np.concatenate([free, free + 1000]), table, 8, int(new.sum()), start=4)
    _check(ctx, new, free, table, 8, int(new.sum()), start=-2)  # the first two have no block
    ctx[2], new[3] = -7, -4
    table[2] = -1
    _check(ctx, new, np.arange(500), table, 8, 400)


def test_lengths_near_31_bits():
    ctx = np.array([2 ** 31 - 1, 2 ** 31 - 20, 5])
    new = np.array([10, 7, 3])
    table = np.full((3, 4), 9, np.int64)
    import torch  # noqa: F401

    log("tables near 2^31")
    got = _run(ctx, new, np.arange(10), table, 16, 20)
    assert got[3].tolist() == [2 ** 31 - 1, 2 ** 31 - 13, 8]
    assert got[2].tolist() == [0, 10, 17, 20]
    assert np.all(got[0][:17] == -1)  # beyond a table of 4 blocks
    assert got[0][17:20].tolist() == [9 * 16 + 5, 9 * 16 + 6, 9 * 16 + 7]
    assert got[4].tolist() == [0] and np.all(got[5] == 9)


def test_buffers_in_place_repeat_and_graph():
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    rng = np.random.default_rng(9)
    ctx, new, free, table = _case(rng, 40, 300, 20, 16)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).to(DEV)  # noqa: E731
    T = int(new.sum()) + 5
    kept = dict(slot_mapping=torch.empty(T, dtype=torch.int64, device=DEV), positions=i32(np.zeros(T)),
                query_start=i32(np.zeros(41)), seq_lens=i32(np.zeros(40)), blocks_needed=i32([0]))
    wide = torch.full((40, table.shape[1] + 3), 77, dtype=torch.int32, device=DEV)
    wide[:, : table.shape[1]] = i32(table)
    args = (i32(ctx), i32(new), i32(free), wide[:, : table.shape[1]], 16)
    want = oa.block_tables(ctx, new, free, table, 16, T)
    log("tables graph")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = nv.nvfp4_kv_block_tables(*args, **kept)
    for _ in range(3):
        for b in kept.values():
            b.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        assert np.array_equal(wide[:, : table.shape[1]].cpu().numpy(), want[5])
        assert bool((wide[:, table.shape[1]:] == 77).all())
    assert got[0] is kept["slot_mapping"]


def test_a_serving_run():
    """Prompts, then a drafted tree, then a decode step: tables built on the GPU, keys and values
    stored through their slot map, attention through their block table."""
    import torch

    import bit_block_scaled_nvfp4_amd as nv

    rng = np.random.default_rng(10)
    H, Hk, D, bs, R = 6, 2, 128, 16, 3
    blocks = 40
    kc = torch.full((blocks * bs, Hk * D), 0x7F, dtype=torch.uint8, device=DEV)
    vc = torch.full((blocks * bs, Hk * D), 0xFF, dtype=torch.uint8, device=DEV)
    ks, vs = np.float32(0.02), np.float32(0.015)
    free = torch.from_numpy(rng.permutation(blocks)).to(torch.int32).to(DEV)
    taken = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.full((R, 12), -1, dtype=torch.int32, device=DEV)
    ctx = torch.zeros(R, dtype=torch.int32, device=DEV)
    keys = [np.zeros((0, Hk * D), np.uint8) for _ in range(R)]
    vals = [np.zeros((0, Hk * D), np.uint8) for _ in range(R)]
    for step, counts in enumerate([[50, 7, 90], [5, 9, 3], [1, 1, 1]]):
        T = sum(counts) + 4  # padded batch
        new = torch.tensor(counts, dtype=torch.int32, device=DEV)
        slots, pos, start, lens, need = nv.nvfp4_kv_block_tables(ctx, new, free, table, bs, T, free_start=taken)
        k = to_type(rng.standard_normal((T, Hk * D)) * 3, "bf16")
        v = to_type(rng.standard_normal((T, Hk * D)), "bf16")
        q = to_type(rng.standard_normal((T, H, D)), "bf16")
        dev = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(DEV)  # noqa: E731
        nv.nvfp4_kv_fp8_store(dev(k), dev(v), scalar(ks), scalar(vs), kc, vc, slots)
        args = (dev(q), kc, vc, scalar(ks), scalar(vs), table, start, lens)
        kw = dict(block_size=bs, num_kv_heads=Hk, out=torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV))
        mask = None
        if step == 1:
            mask = np.concatenate([tree_mask(rng, counts), np.zeros((4, 1), np.int64)])
            out = nv.nvfp4_kv_fp8_tree_attention(*args, torch.from_numpy(mask).to(DEV), **kw)
        else:
            out = nv.nvfp4_kv_fp8_attention(*args, **kw)
        taken += need
        ctx = lens
        torch.cuda.synchronize()
        log(f"serving step {step}")
        at = 0
        for r, n in enumerate(counts):
            keys[r] = np.concatenate([keys[r], oracle.kv_fp8_encode(k[at:at + n], ks)])
            vals[r] = np.concatenate([vals[r], oracle.kv_fp8_encode(v[at:at + n], vs)])
            L = len(keys[r])
            own = dict(tree=unpack(mask)[at:at + n]) if mask is not None else {}
            want, tol = oa.attention(q[at:at + n], keys[r], vals[r], ks, vs, np.arange(1)[None], [0, n], [L], L, Hk,
                                     D ** -0.5, out_eps=EPS["bf16"], **own)
            compare(out[at:at + n].double().cpu().numpy(), want, tol, f"step {step} request {r}")
            at += n
        assert bool((out[at:] == 0).all())

"""GPU parity of the attention over tiles of 256 query rows with a workgroup per item (the form that long prompts
take) at sizes that the oracle can follow: every type and head size with every mask, bad blocks, NaN codes
and rows that see nothing.  That these sizes lead there is tested in test_attention_plan.py."""

import numpy as np
import pytest

from oracle import attention as oa

from .attention_util import SENTINEL, Problem, compare, pack
from .gpu_util import log
from .test_gpu_attention_scores import hints, problem

pytestmark = pytest.mark.gpu

NEW = 130
TYPES = pytest.mark.parametrize("dtype", ["bf16", "f16"])
DIMS = pytest.mark.parametrize("head_dim", [64, 128, 256])


def check(p, what):
    log(f"tiles {what}")
    want, tol = p.oracle()
    got = p.run(**hints(NEW, False))
    compare(got, want, tol, what)
    return got


@TYPES
@DIMS
@pytest.mark.parametrize("masks", ["none", "documents", "prefix", "both"])
def test_prompts(dtype, head_dim, masks):
    for cap, slopes in ((0.0, False), (20.0, True)):
        p = problem(NEW, head_dim, dtype, seed=23, slopes=slopes)
        if masks in ("documents", "both"):
            p.options["doc_start"] = np.concatenate([np.arange(c, c + n) // 37 * 37 for c, n in p.lens])
        if masks in ("prefix", "both"):
            p.options["prefix_lens"] = np.array([c + n // 2 for c, n in p.lens])
        if cap:
            p.options["softcap"] = cap
        check(p, f"{dtype} D={head_dim} masks={masks} cap={cap} slopes={slopes}")


@TYPES
@DIMS
def test_trees_of_three_words(dtype, head_dim):
    p = problem(NEW, head_dim, dtype, seed=29, tree=True)
    assert p.options["tree_mask"].shape[1] == 3
    p.options["tree_mask"][[0, 7, 200]] = 0
    got = check(p, f"tree {dtype} D={head_dim}")
    assert np.any(got[0] != 0)  # 90 positions of context


@DIMS
def test_rows_that_see_nothing_and_blocks_outside_the_cache(head_dim):
    p = problem(NEW, head_dim, seed=31)
    start = np.zeros(p.tokens, np.int64)
    start[::3] = 10 ** 6
    p.options["doc_start"] = start
    p.table[0, 3] = -7
    p.table[0, 5] = p.num_slots
    p.table[1, 0] = 2 ** 31 - 1
    p.table[3, :] = -1
    got = check(p, f"empty rows D={head_dim}")
    assert np.all(got[::3] == 0) and np.all(got[-NEW:] == 0)


@TYPES
@DIMS
@pytest.mark.parametrize("tree", [False, True])
def test_nan_codes_reach_only_the_rows_that_see_them(dtype, head_dim, tree):
    p = problem(NEW, head_dim, dtype, seed=37)
    c, n = p.lens[0]
    if tree:
        bits = np.zeros((p.tokens, 192), bool)
        bits[np.arange(p.tokens), np.concatenate([np.arange(m) for _, m in p.lens])] = True  # itself alone
        bits[:n:5, n - 4] = True
        p.options["tree_mask"] = pack(bits)
    s = oa.slots_of(p.table[0], c + n, p.block_size, p.num_slots)
    p.vc[s[c + n - 4], 5] = 0xFF
    p.vc[s[c + n - 4], 7 * head_dim + 1] = 0x7F
    p.kc[s[c + n - 2], 2] = 0x7F
    got = check(p, f"NaN codes {dtype} D={head_dim} tree={tree}")
    assert np.isnan(got[: n]).any() and not np.isnan(got[1 if tree else 0]).any() and not np.isnan(got[n:]).any()


def test_rows_of_no_request_and_strided_outputs():
    import torch

    lens = [(90, NEW), (33, 65), (0, NEW), (60, NEW)]
    p = Problem(lens, 16, 8, 64, seed=41, pad_tokens=5)
    want, tol = p.oracle()
    d = p.device()
    wide = torch.full((p.tokens, 18, 72), SENTINEL, dtype=d["out"].dtype, device=d["out"].device)
    log("strided tiles")
    got = p.run(out=wide[:, 1:17, :64], **hints(NEW, False))
    compare(got, want, tol, "window")
    assert np.all(got[p.real:] == SENTINEL)
    untouched = wide.clone()
    untouched[: p.real, 1:17, :64] = SENTINEL
    assert bool((untouched == SENTINEL).all())

"""Which positions a token sees under a document mask, a prefix mask, and both: the sets themselves, read off the
attention's output (queries of zeros, so that every visible position weighs the same, and the value of position
j is 1 in dim j alone)."""

import numpy as np
import pytest

from .attention_util import Problem

D = 64


def seen(p, t, docs, prefix):
    """The definition: doc_start <= j and (j <= p or j < prefix)."""
    first = docs[t] if docs is not None else 0
    return {j for j in range(len(p.docs_of)) if first <= j and (j <= t or j < prefix)}


def problem(starts, n, docs, prefix):
    """One request of n fresh tokens whose documents begin at ``starts``."""
    p = Problem([(0, n)], 4, 2, D, seed=1)
    from oracle import attention as oa

    slots = oa.slots_of(p.table[0], n, p.block_size, p.num_slots)
    p.q[:] = 0
    p.vc[slots] = 0
    for j in range(n):
        p.vc[slots[j], [j, D + j]] = 0x38  # 1.0
    p.vs = np.float32(1.0)
    p.docs_of = np.array(starts)[np.searchsorted(starts, np.arange(n), side="right") - 1]
    if docs:
        p.options["doc_start"] = p.docs_of
    if prefix:
        p.options["prefix_lens"] = np.array([prefix])
    return p


def check(p, out, docs, prefix):
    for t in range(p.tokens):
        want = seen(p, t, p.docs_of if docs else None, prefix)
        for h in range(4):
            assert set(np.flatnonzero(out[t, h]).tolist()) == want, (t, h)
            if want:  # equal weights; the sum of the rounded quotients: half a bf16 step each
                assert np.allclose(out[t, h][sorted(want)], 1.0 / len(want), rtol=2.0 ** -8 + 2.0 ** -20)


CASES = [(docs, prefix) for docs in (False, True) for prefix in (0, 3, 5, 7, 12, 40)]
STARTS, N = [0, 5, 9], 12


@pytest.mark.parametrize("docs,prefix", CASES)
def test_the_oracle_sees_these_sets(docs, prefix):
    p = problem(STARTS, N, docs, prefix)
    check(p, p.oracle()[0], docs, prefix)


def test_documents_bound_the_prefix():
    """Both masks: a prefix within the first document stays with that document, whose tokens see all of it; one that
    reaches further shows a document's tokens the beginning of the next one."""
    p = problem(STARTS, N, True, 3)
    assert [seen(p, t, p.docs_of, 3) for t in (0, 4, 5, 8, 9)] == [{0, 1, 2}, {0, 1, 2, 3, 4}, {5}, {5, 6, 7, 8}, {9}]
    assert [seen(p, t, p.docs_of, 7) for t in (0, 4, 5, 8, 9)] == [
        {0, 1, 2, 3, 4, 5, 6}, {0, 1, 2, 3, 4, 5, 6}, {5, 6}, {5, 6, 7, 8}, {9}]


@pytest.mark.gpu
@pytest.mark.parametrize("docs,prefix", CASES)
@pytest.mark.parametrize("longest", [1, 12, 60])  # tiles of 16, 32 and 256 rows
def test_the_kernels_see_these_sets(docs, prefix, longest):
    from .gpu_util import log

    log(f"masks docs={docs} prefix={prefix} longest={longest}")
    p = problem([0, 5, 9, 30], 60, docs, prefix)
    check(p, p.run(max_query_len=longest, max_seq_len=2000 if longest == 60 else 60), docs, prefix)

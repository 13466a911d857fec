"""GPU: the attention's output written over its query (the same tensor), in every kernel and division, and into the
columns of the fused row that the query is a window of."""

import numpy as np
import pytest

from .attention_util import SENTINEL, compare
from .gpu_util import log
from .test_gpu_attention_scores import hints, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("new", [1, 9, 40, 130])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_output_over_the_query(head_dim, new, split, tree):
    p = problem(new, head_dim, seed=43, tree=tree)
    want, tol = p.oracle()
    d = p.device()
    log(f"in place D={head_dim} new={new} split={split} tree={tree}")
    got = p.run(q=d["q"], out=d["q"], **hints(new, split))
    compare(got, want, tol, "in place")
    assert np.array_equal(got, d["q"].double().cpu().numpy())


@pytest.mark.parametrize("new", [1, 40])
def test_output_beside_the_query_in_a_fused_row(new):
    import torch

    p = problem(new, 64, seed=47)
    want, tol = p.oracle()
    q = p.device()["q"]
    T, H, D = q.shape
    fused = torch.full((T, 3 * H, D), SENTINEL, dtype=q.dtype, device=q.device)
    fused[:, H:2 * H] = q
    log(f"fused row new={new}")
    got = p.run(q=fused[:, H:2 * H], out=fused[:, :H], **hints(new, True))
    compare(got, want, tol, "fused row")
    assert bool((fused[:, H:2 * H] == q).all()) and bool((fused[:, 2 * H:] == SENTINEL).all())

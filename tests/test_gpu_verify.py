"""GPU parity of nvfp4_verify_drafted against the oracle in exact rationals: every number has to be equal.  Probabilities of
ordinary distributions (sums in binary64 decide them alike but within 2^-45 of a border, which seeded numbers do not
come near), and dyadic ones, whose sums are exact in binary64, with random numbers on the borders themselves."""

import numpy as np
import pytest

import bit_block_scaled_nvfp4_amd as nv
from oracle import serving as osv

from .gpu_util import DEV, log

pytestmark = pytest.mark.gpu


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Batch:
    def __init__(self, counts, vocab, seed=0, near=0.4, certain=False, pad=0):
        rng = np.random.default_rng(seed)
        start = np.concatenate([[0], np.cumsum([n + 1 if n >= 0 else 0 for n in counts])])
        rows = int(start[-1]) + pad
        logits = rng.standard_normal((rows, vocab)) * 2.0
        self.p = _softmax(logits)
        self.q = None if certain else _softmax(logits + near * rng.standard_normal((rows, vocab)))
        draw = self.p if certain else self.q
        self.tokens = np.array([rng.choice(vocab, p=x.astype(np.float64) / x.astype(np.float64).sum()) for x in np.roll(draw, 1, 0)], np.int64).reshape(rows)
        self.start, self.rows, self.vocab = start.astype(np.int64), rows, vocab
        self.u, self.w = rng.random(rows).astype(np.float32), rng.random(len(counts)).astype(np.float32)

    def device(self):
        import torch

        i32 = lambda x: torch.from_numpy(np.asarray(x)).to(torch.int32).to(DEV)  # noqa: E731
        f32 = lambda x: None if x is None else torch.from_numpy(np.asarray(x, np.float32)).to(DEV)  # noqa: E731
        return dict(target_probs=f32(self.p), draft_probs=f32(self.q), tokens=i32(self.tokens), query_start=i32(self.start),
                    accept_u=f32(self.u), sample_u=f32(self.w))

    def want(self):
        return osv.verify(self.p, self.q, self.tokens, self.start, self.u, self.w, np.full(self.rows, -7))


def check(b, what, **kw):
    import torch

    log(f"verify {what}")
    want = b.want()
    out = torch.full((b.rows,), -7, dtype=torch.int32, device=DEV)
    got = nv.nvfp4_verify_drafted(**{**b.device(), "out": out, **kw})
    torch.cuda.synchronize()
    got = [x.cpu().numpy() for x in got]
    assert np.array_equal(got[0], want[0]), (what, got[0], want[0])
    assert np.array_equal(got[1], want[1]), (what, np.argwhere(got[1] != want[1]).tolist(), got[1], want[1])
    return got


@pytest.mark.parametrize("vocab", [1, 2, 63, 257, 4095, 4096, 4097, 9001])
@pytest.mark.parametrize("certain", [False, True])
def test_vocabularies(vocab, certain):
    for seed in range(4):
        check(Batch([3, 0, 1, 5, 2], vocab, seed=seed, certain=certain), f"V={vocab} certain={certain}")


@pytest.mark.parametrize("counts", [[0], [1], [64], [65, 63, 200], [-1, 3, -1, -1, 0, 7], [0] * 300 + [4]])
def test_counts_of_drafts(counts):
    """More drafts than lanes, requests without rows, many requests; drafts that agree mostly."""
    got = check(Batch(counts, 70, seed=len(counts), near=0.05, pad=3), f"counts {counts[:8]}")
    assert np.all(got[1][-3:] == -7)


def test_everything_accepted_and_nothing_accepted():
    b = Batch([5, 9, 70], 500, seed=1)
    b.u[:] = 0.0
    got = check(b, "all accepted")
    assert got[0].tolist() == [5, 9, 70]
    b.p[np.arange(b.rows - 1), b.tokens[1:]] = 0.0
    got = check(b, "none accepted")
    assert got[0].tolist() == [0, 0, 0]


def test_equal_distributions_accept_everything():
    b = Batch([6] * 20, 300, seed=2)
    b.q = b.p.copy()
    got = check(b, "equal distributions")
    assert np.all(got[0] == 6)


def test_borders_of_the_sampling():
    """Dyadic probabilities: the sums are exact, and a random number on a border belongs to the next token."""
    V = 16
    p = np.tile(np.float32(1.0 / 16), (17, V))
    for start_of in (0, 3, 9):
        b = Batch([0] * 17, V, seed=3)
        b.p, b.q = p.copy(), None
        b.p[:, start_of] = 0.0
        b.p[:, (start_of + 5) % V] += np.float32(1.0 / 16)
        b.w = (np.arange(17) / 16.0).astype(np.float32)  # 1.0 among them: the last token with a weight
        check(b, f"borders, token {start_of} without weight")


@pytest.mark.parametrize("vocab", [4096 * 3, 4096 * 2 + 5])
def test_borders_between_chunks(vocab):
    """Weights at the ends of chunks alone; random numbers on the border between them."""
    places = [4095, 4096, 8191, vocab - 1]
    b = Batch([0] * 9, vocab, seed=4)
    b.q = None
    b.p[:] = 0.0
    b.p[:, places] = np.float32(0.25)
    b.w = np.array([0.0, 0.2, 0.25, 0.4, 0.5, 0.7, 0.75, 0.99, 1.0 - 2.0 ** -24], np.float32)
    got = check(b, f"chunk borders V={vocab}")
    assert got[1].tolist() == [4095, 4095, 4096, 4096, 8191, 8191, vocab - 1, vocab - 1, vocab - 1]


def test_borders_of_the_acceptance():
    """u q = p is not accepted; products are not rounded."""
    b = Batch([1, 1, 1], 8, seed=5)
    b.q[:] = np.float32(0.5)
    b.p[:] = np.float32(0.125)
    b.u[[0, 2, 4]] = [0.25, np.nextafter(np.float32(0.25), np.float32(0)), np.nextafter(np.float32(0.25), np.float32(1))]
    assert check(b, "u q = p")[0].tolist() == [0, 1, 0]


def test_zero_weights():
    """No weight left (the target below the draft everywhere): the target's row; an empty row: -1; NaN counts as 0."""
    b = Batch([2, 2, 2, 1], 100, seed=6)
    b.q[0] = b.p[0] + np.float32(0.25)  # every w is 0
    b.u[0] = 0.999999
    b.p[3] = 0.0
    got = check(b, "no weights")
    assert got[0][1] == 0 and got[1][3] == -1
    b.p[6, 10:20] = np.nan
    b.q[6, 40:50] = np.nan
    import torch

    d = b.device()
    clean = Batch([2, 2, 2, 1], 100, seed=6)
    clean.q, clean.p = b.q.copy(), b.p.copy()
    clean.p[6, 10:20] = 0.0
    clean.p[6, 40:50] = 0.0  # p > q is false there
    clean.q[6, 40:50] = 0.0
    clean.tokens[7] = b.tokens[7] = 45  # a NaN draft probability is not accepted
    clean.q[6, 45] = 1.0
    d["tokens"] = torch.from_numpy(b.tokens).to(torch.int32).to(DEV)
    got = [x.cpu().numpy() for x in nv.nvfp4_verify_drafted(**d)]
    want = osv.verify(clean.p, clean.q, clean.tokens, clean.start, clean.u, clean.w, np.full(b.rows, -1))
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_tokens_outside_the_vocabulary_are_not_accepted():
    for certain in (False, True):
        b = Batch([3, 3], 50, seed=7, certain=certain)
        b.u[:] = 0.0
        b.tokens[2], b.tokens[5] = 50, -3
        assert check(b, "outside")[0].tolist() == [1, 0]


def test_random_numbers_outside_their_range():
    b = Batch([2, 2, 2, 2], 60, seed=8)
    b.w[:] = [1.0, 5.0, np.nan, -1.0]
    import torch

    got = [x.cpu().numpy() for x in nv.nvfp4_verify_drafted(**b.device())]
    c = Batch([2, 2, 2, 2], 60, seed=8)
    c.w[:] = [1.0, 1.0, 1.0, 0.0]
    want = c.want()
    torch.cuda.synchronize()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_strided_rows_and_starts_outside():
    import torch

    b = Batch([3, 4, 2], 77, seed=9, pad=2)
    want = b.want()
    d = b.device()
    wide = torch.full((b.rows, 200), 9.0, device=DEV)
    wide[:, 1:78] = d["target_probs"]
    wide[:, 100:177] = d["draft_probs"]
    got = nv.nvfp4_verify_drafted(**{**d, "target_probs": wide[:, 1:78], "draft_probs": wide[:, 100:177]})
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy()[:-2], want[1][:-2])
    b.start = np.array([-4, 3, 2, 10 ** 6])  # clamped; a start that falls is a request without rows
    check(b, "starts outside")


def test_no_work():
    import torch

    b = Batch([2], 30, seed=10)
    d = b.device()
    none = {**d, "query_start": torch.zeros(1, dtype=torch.int32, device=DEV), "sample_u": d["sample_u"][:0]}
    got = nv.nvfp4_verify_drafted(**none)
    assert got[0].shape == (0,) and bool((got[1] == -1).all())
    empty = {k: (None if v is None else v[:0]) for k, v in d.items()}
    empty.update(query_start=torch.zeros(3, dtype=torch.int32, device=DEV), sample_u=torch.rand(2, device=DEV))
    assert nv.nvfp4_verify_drafted(**empty)[0].tolist() == [0, 0]


def test_large_vocabulary_and_many_requests():
    """Against the same definition in binary64 (the exact one would take minutes)."""
    import torch

    log("verify V=131077, 40 requests")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    n, R, V = 4, 40, 131077
    logits = torch.randn((R * (n + 1), V), generator=g, device=DEV)
    p, q = torch.softmax(logits, 1), torch.softmax(logits + 0.4 * torch.randn(logits.shape, generator=g, device=DEV), 1)
    tokens = torch.multinomial(q, 1, generator=g).flatten().roll(1).to(torch.int32)
    start = torch.arange(0, R * (n + 1) + 1, n + 1, dtype=torch.int32, device=DEV)
    u, w = torch.rand(R * (n + 1), generator=g, device=DEV), torch.rand(R, generator=g, device=DEV)
    acc, out = nv.nvfp4_verify_drafted(p, q, tokens, start, u, w)
    for r in range(R):
        row, last = r * (n + 1), r * (n + 1) + n
        while row < last and u[row].item() * q[row, tokens[row + 1].item()].item() < p[row, tokens[row + 1].item()].item():
            row += 1
        assert acc[r].item() == row - r * (n + 1)
        left = (p[row].double() - q[row].double()).clamp(min=0) if row < last else p[row].double()
        upto = left.cumsum(0).cpu()
        assert out[row].item() == int(torch.searchsorted(upto, upto[-1:] * w[r].item(), right=True))
        assert out[r * (n + 1):row].tolist() == tokens[r * (n + 1) + 1:row + 1].tolist() and out[row + 1:last + 1].tolist() == [-1] * (last - row)


def test_side_stream_graphs_and_two_at_once():
    import torch

    b = Batch([3, 7, 0, 5], 9001, seed=11)
    want = b.want()
    d = b.device()
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s in side:
            with torch.cuda.stream(s):
                outs.append(nv.nvfp4_verify_drafted(**d))
    torch.cuda.synchronize()
    for a, o in outs:
        assert np.array_equal(a.cpu().numpy(), want[0]) and np.array_equal(o.cpu().numpy(), want[1])
    log("graphs")
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            kept.append(nv.nvfp4_verify_drafted(**d))
    for k in range(4):
        d["sample_u"].copy_(torch.rand(4, device=DEV))
        d["accept_u"].mul_(0.7)
        for a, o in kept:
            a.fill_(-9)
        for graph in graphs:
            graph.replay()
        a, o = nv.nvfp4_verify_drafted(**d)
        torch.cuda.synchronize()
        for x, y in kept:
            assert torch.equal(x, a) and torch.equal(y, o)


@pytest.mark.parametrize("start", [[0, 6, 2, 9, 0, 4, 4, 12, -3, 1], [0, 3, 7, 12, 0, 0, 0], [0, 12, 0, 12, 0, 12], [5, 12, 4, 8, 3, 6, 0, 1]])
def test_starts_that_fall_leave_a_rows_last_request(start):
    """Rows of several requests: the last one's tokens, whatever order the workgroups run in."""
    b = Batch([0] * (len(start) - 1), 9001, seed=12, pad=12 - (len(start) - 1))
    b.start = np.array(start)
    for k in range(8):
        b.u = np.roll(b.u, 1)
        check(b, f"starts {start}, {k}")


def test_starts_that_fall_among_many_requests():
    b = Batch([0] * 700, 40, seed=13)
    rng = np.random.default_rng(14)
    b.start = np.cumsum(rng.integers(-3, 5, 701))  # falls now and then, by less than it rises
    b.start[300:310] = b.start[300]
    check(b, "700 requests whose starts fall")


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("vocab", [4097, 32000])
def test_numbers_of_one_and_more_take_the_last_token_with_a_weight(vocab, certain):
    """Wide rows whose second half weighs less than a sum's rounding: running sums reach the total before its end, and
    pass it where they are added in another order."""
    rng = np.random.default_rng(15)
    n = 40
    b = Batch([1] * n, 2, seed=15, certain=certain)
    logits = rng.standard_normal((b.rows, vocab)) * 3.0
    logits[:, vocab // 2:] -= 50.0
    b.p, b.vocab = _softmax(logits), vocab
    b.q = None if certain else _softmax(logits + 0.4 * rng.standard_normal(logits.shape))
    b.tokens = np.zeros(b.rows, np.int64)
    b.u[:] = 1.0  # (half of the first rows are refused where drafts are not certain)
    for w in (1.0, 1.5, np.inf, np.nan):
        b.w[:] = w
        got = [x.cpu().numpy() for x in nv.nvfp4_verify_drafted(**b.device())]
        for r in range(n):
            row = 2 * r + got[0][r]
            left = b.p[row].astype(np.float64)
            if got[0][r] == 0 and certain:
                left[0] = 0.0
            elif got[0][r] == 0:
                left = left - b.q[row]
            assert got[1][row] == np.flatnonzero(left > 0)[-1], (w, r)


def test_starts_that_fall_and_rows_without_a_weight():
    """A request that finds no token to sample leaves a later one's rows alone too."""
    b = Batch([0] * 4, 5000, seed=17, pad=8)
    b.start = np.array([0, 7, 3, 10, 6])
    b.u[:] = 1e9  # nothing is accepted
    b.p[0] = 0.0
    got = check(b, "an empty first row")
    assert got[0].tolist() == [0, 0, 0, 0] and got[1][0] == -1 and got[1][3] >= 0


def test_a_batch_padded_with_requests_at_row_zero():
    """Starts of zero behind the last request: none of its rows, or of the others', is theirs."""
    b = Batch([3, 0, 5, 2] + [0] * 400, 300, seed=18)
    b.start[5:] = 0
    got = check(b, "starts of zero behind the last request")
    assert np.all(got[1][:14] >= -1) and np.all(got[1][14:] == -7)

"""The serving operators together, as a step runs them: block tables, norm and rotation, append, attention over either
cache, verification of drafted tokens; several steps on one cache, and a step captured into a graph."""

import numpy as np
import pytest

import bit_block_scaled_nvfp4_amd as nv
import oracle
from oracle import attention as oa
from oracle import serving as osv

from .attention_util import EPS, compare, to_type
from .gpu_util import DEV, log

pytestmark = pytest.mark.gpu

H, HK, D, BS, V, LAST = 6, 2, 64, 16, 600, 4  # heads, KV heads, dims, block size, vocabulary, most drafts


class Serving:
    """A layer's weights, a cache of either format, and what a loop keeps from step to step."""

    def __init__(self, cache, requests=3, seed=0):
        import torch

        rng = np.random.default_rng(seed)
        self.rng, self.cache, self.R = rng, cache, requests
        self.qw, self.kw = (to_type(rng.standard_normal(D) * 0.3, "bf16") for _ in range(2))
        self.freq = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
        f32 = lambda x: torch.tensor(np.atleast_1d(np.asarray(x, np.float32)), device=DEV)  # noqa: E731
        self.scales = (0.02, 0.009) if cache == "fp8" else (300.0, 700.0)
        self.dev = dict(qw=f32(self.qw).bfloat16(), kw=f32(self.kw).bfloat16(), freq=f32(self.freq), ks=f32(self.scales[0]), vs=f32(self.scales[1]))
        blocks, u8 = 24, dict(dtype=torch.uint8, device=DEV)
        if cache == "fp8":
            self.kv = [torch.full((blocks * BS, HK * D), 0x7F, **u8) for _ in range(2)]
        else:
            self.kv = [torch.full((blocks, HK, BS, n), 0x7F, **u8) for n in (D // 2, D // 16, D // 2, D // 16)]
        self.table = torch.full((requests, 8), -1, dtype=torch.int32, device=DEV)
        self.free = torch.from_numpy(rng.permutation(blocks)).to(torch.int32).to(DEV)
        self.free_start = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.context = np.zeros(requests, np.int64)

    def inputs(self, new):
        """Rows of a fused projection for the new tokens, with two rows of padding."""
        import torch

        T = int(np.sum(new)) + 2
        row = to_type(self.rng.standard_normal((T, (H + 2 * HK) * D)), "bf16")
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).to(DEV)  # noqa: E731
        return row, torch.from_numpy(row).bfloat16().to(DEV), i32(self.context), i32(np.asarray(new))

    def step(self, fused, context, new, q_out, out):
        """One step's launches; everything they write is the caller's or returned."""
        T = fused.shape[0]
        q = fused[:, :H * D].unflatten(1, (H, D))
        k = fused[:, H * D:(H + HK) * D].unflatten(1, (HK, D))
        v = fused[:, (H + HK) * D:].unflatten(1, (HK, D))
        d = self.dev
        slots, pos, start, lens, used = nv.nvfp4_kv_block_tables(context, new, self.free, self.table, BS, T, free_start=self.free_start)
        nv.nvfp4_qk_norm_rope(q, None, pos, d["freq"], q_weight=d["qw"], weight_offset=1.0, q_out=q_out)
        words = dict(k_weight=d["kw"], weight_offset=1.0)
        bounds = dict(max_query_len=T, max_seq_len=128, out=out)
        if self.cache == "fp8":
            nv.nvfp4_kv_fp8_append(k, v, pos, d["freq"], d["ks"], d["vs"], *self.kv, slots, **words)
            nv.nvfp4_kv_fp8_attention(q_out, *self.kv, d["ks"], d["vs"], self.table, start, lens, block_size=BS, num_kv_heads=HK, **bounds)
        else:
            nv.nvfp4_kv_fp4_append(k, v, pos, d["freq"], d["ks"], d["vs"], *self.kv, slots, **words)
            nv.nvfp4_kv_fp4_attention(q_out, *self.kv, d["ks"], d["vs"], self.table, start, lens, **bounds)
        return slots, pos, start, lens, used

    def rows(self):
        """Exact values of the cache's rows by slot, keys and values, less their global scale."""
        if self.cache == "fp8":
            return [oa._decode(x.cpu().numpy(), 1.0) for x in self.kv]
        c = [x.cpu().numpy() for x in self.kv]
        return [osv.decode4(c[i], c[i + 1]).transpose(0, 2, 1, 3).reshape(-1, HK * D) for i in (0, 2)]

    def check(self, row, new, got, q_out, out):
        """The step's results against the oracle's, from the step's inputs."""
        slots, pos, start, lens, _ = (x.cpu().numpy().astype(np.int64) for x in got)
        T = len(row)
        q, k, v = row[:, :H * D].reshape(T, H, D), row[:, H * D:(H + HK) * D].reshape(T, HK, D), row[:, (H + HK) * D:].reshape(T, HK, D)
        assert np.array_equal(pos[:start[-1]], np.concatenate([np.arange(c, c + n) for c, n in zip(self.context, new)]))
        assert np.all(slots[start[-1]:] == -1) and np.all(slots[:start[-1]] >= 0)
        turned = [osv.round_to(osv.turn(x, pos, self.freq, weight=w, eps=1e-6, offset=1.0)[0], "bf16").astype(np.float64) for x, w in ((q, self.qw), (k, self.kw))]
        mine = slice(0, start[-1])
        assert np.array_equal(q_out.double().cpu().numpy(), turned[0])
        rows = self.rows()
        for x, value, scale in zip(rows, (turned[1], v), self.scales):
            x = x[slots[mine]].reshape(-1, HK, D)
            value = value[mine].astype(np.float32)
            want = oa._decode(oracle.kv_fp8_encode(value, np.float32(scale)), 1.0) if self.cache == "fp8" else osv.decode4(*osv.encode4(value, scale))
            assert np.array_equal(x, want)
        by = self.scales if self.cache == "fp8" else tuple(1.0 / np.float64(np.float32(s)) for s in self.scales)
        want, tol = oa.attention(turned[0], rows[0], rows[1], np.float64(np.float32(by[0])) if self.cache == "fp8" else by[0],
                                 np.float64(np.float32(by[1])) if self.cache == "fp8" else by[1], self.table.cpu().numpy(), start, lens, BS, HK,
                                 D ** -0.5, out=np.full((T, H, D), 7.5), out_eps=EPS["bf16"], decode=lambda x, s: x * s)
        compare(out.double().cpu().numpy(), want, tol, f"attention over {self.cache}")

    def buffers(self, T):
        import torch

        return torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV), torch.full((T, H, D), 7.5, dtype=torch.bfloat16, device=DEV)


def _probabilities(rng, rows):
    import torch

    x = torch.from_numpy(rng.standard_normal((rows, V)) * 1.5)
    y = x + 0.3 * torch.from_numpy(rng.standard_normal((rows, V)))
    return torch.softmax(x, 1).float().to(DEV), torch.softmax(y, 1).float().to(DEV)


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
def test_prompts_then_steps_of_drafted_tokens(cache):
    import torch

    s = Serving(cache)
    new = np.array([5, 37, 1])
    log(f"prompts, {cache}")
    row, fused, context, lens = s.inputs(new)
    q_out, out = s.buffers(len(row))
    got = s.step(fused, context, lens, q_out, out)
    s.check(row, new, got, q_out, out)
    s.context += new
    s.free_start += got[4]
    for k in range(4):
        # the last token and up to four drafted ones; those that are rejected are written over by the next step
        new = 1 + s.rng.integers(0, LAST + 1, s.R)
        log(f"step {k}, {cache}: contexts {s.context.tolist()}, {new.tolist()} tokens")
        row, fused, context, lens = s.inputs(new)
        q_out, out = s.buffers(len(row))
        got = s.step(fused, context, lens, q_out, out)
        s.check(row, new, got, q_out, out)
        rows = len(row)
        p, q = _probabilities(s.rng, rows)
        tokens = torch.multinomial(q.cpu(), 1).flatten().roll(1).to(torch.int32).to(DEV)
        u, w = torch.rand(rows, device=DEV), torch.rand(s.R, device=DEV)
        emitted = torch.full((rows,), -7, dtype=torch.int32, device=DEV)
        accepted, emitted = nv.nvfp4_verify_drafted(p, q, tokens, got[2], u, w, out=emitted)
        want = osv.verify(*(x.cpu().numpy() for x in (p, q, tokens, got[2], u, w)), np.full(rows, -7))
        assert np.array_equal(accepted.cpu().numpy(), want[0]) and np.array_equal(emitted.cpu().numpy(), want[1])
        assert emitted[-2:].tolist() == [-7, -7]
        # blocks that the rejected tokens took stay with their request: the next step needs them, or finds them held
        held = -(-(s.context + new) // BS)
        s.context += 1 + want[0]
        assert np.all(-(-s.context // BS) <= held)
        s.table[torch.arange(8, device=DEV)[None, :] >= torch.from_numpy(-(-s.context // BS)).to(DEV)[:, None]] = -1
        s.free_start += got[4]
        if int(s.free_start) > 16:
            break


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
def test_a_step_in_a_graph(cache):
    """Captured once and replayed with other tokens, against the same step run eagerly on a second cache."""
    import torch

    a, b = Serving(cache, seed=5), Serving(cache, seed=5)
    new = np.array([9, 2, 20])
    row, fused, context, lens = a.inputs(new)
    q_out, out = a.buffers(len(row))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(fused, context, lens, q_out, out)
    side.synchronize()
    log(f"graph over {cache}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(fused, context, lens, q_out, out)
    for k in range(4):
        fused.mul_(-0.75)
        q_out.fill_(3.0)
        out.fill_(7.5)
        graph.replay()
        q2, o2 = b.buffers(len(row))
        b.step(fused, context, lens, q2, o2)
        torch.cuda.synchronize()
        assert torch.equal(q_out, q2) and torch.equal(out, o2) and all(torch.equal(x, y) for x, y in zip(a.kv, b.kv))

"""Shared by the tests of the cache's attention operators: seeded paged problems, and their comparison
with the oracle (oracle/attention.py) under its derived tolerance."""

from __future__ import annotations

import numpy as np

from oracle import attention as oa

#: relative step of the output types: half of it is the last rounding's error
EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}
SENTINEL = 7.5  # rows that must stay as they were


class Problem:
    """A ragged batch over a paged cache of random codes (numpy, host).

    ``lens``: (context, new) of every request.  Blocks are handed out in shuffled order; ``spare``
    blocks and every slot no request owns hold NaN codes, so that a read of one shows."""

    def __init__(self, lens, heads=4, kv_heads=2, head_dim=64, block_size=16, dtype="bf16", seed=0,
                 pad_tokens=0, spare=3, q_std=1.0, cache_pad=0):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kv_heads, self.head_dim = list(lens), heads, kv_heads, head_dim
        self.block_size, self.dtype, self.rng = block_size, dtype, rng
        self.requests = len(self.lens)
        self.seq_lens = np.array([c + n for c, n in self.lens], np.int64)
        self.query_start = np.concatenate([[0], np.cumsum([n for _, n in self.lens])]).astype(np.int64)
        self.real = int(self.query_start[-1])
        self.tokens = self.real + pad_tokens
        need = -(-self.seq_lens // block_size)
        self.width = int(need.max(initial=0)) + 2
        blocks = rng.permutation(int(need.sum()) + spare)
        self.num_slots = len(blocks) * block_size
        self.table = np.full((self.requests, self.width), -1, np.int64)
        row = kv_heads * head_dim
        self.cache_ld = row + cache_pad
        self.kc = np.full((self.num_slots, self.cache_ld), 0x7F, np.uint8)
        self.vc = np.full((self.num_slots, self.cache_ld), 0xFF, np.uint8)
        at = 0
        for r in range(self.requests):
            self.table[r, : need[r]] = blocks[at: at + need[r]]
            at += need[r]
            slots = oa.slots_of(self.table[r], int(self.seq_lens[r]), block_size, self.num_slots)
            for c in (self.kc, self.vc):
                x = rng.standard_normal((len(slots), row)) * 2.0
                c[slots, :row] = _encode(x)
        self.ks, self.vs = np.float32(0.37), np.float32(0.021)
        self.scale = float(np.float32(head_dim ** -0.5))
        q = rng.standard_normal((self.tokens, heads, head_dim)) * q_std
        self.q = to_type(q, dtype)
        self.options = {}

    def oracle(self):
        kw = dict(self.options)
        tree = kw.pop("tree_mask", None)
        if tree is not None:
            kw["tree"] = unpack(tree)
        out0 = np.full((self.tokens, self.heads, self.head_dim), SENTINEL)
        return oa.attention(self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.query_start,
                            self.seq_lens, self.block_size, self.kv_heads, self.scale, out=out0,
                            out_eps=EPS[self.dtype], **kw)

    def device(self):
        """Keyword arguments of the binding, on the GPU; ``out`` is full of the sentinel."""
        import torch

        from .gpu_util import DEV

        td = {"bf16": torch.bfloat16, "f16": torch.float16}[self.dtype]
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).to(DEV)  # noqa: E731
        row = self.kv_heads * self.head_dim
        d = dict(q=torch.from_numpy(self.q).to(td).to(DEV), key_cache=torch.from_numpy(self.kc).to(DEV)[:, :row],
                 value_cache=torch.from_numpy(self.vc).to(DEV)[:, :row],
                 key_scale=torch.tensor([self.ks], device=DEV), value_scale=torch.tensor([self.vs], device=DEV),
                 block_table=i32(self.table), query_start=i32(self.query_start), seq_lens=i32(self.seq_lens),
                 block_size=self.block_size, num_kv_heads=self.kv_heads, scale=self.scale,
                 out=torch.full((self.tokens, self.heads, self.head_dim), SENTINEL, dtype=td, device=DEV))
        for k, v in self.options.items():
            if k == "softcap":
                d[k] = v
            elif k == "slopes":
                d[k] = torch.from_numpy(np.asarray(v, np.float32)).to(DEV)
            elif k == "tree_mask":
                d[k] = torch.from_numpy(v).to(DEV)
            else:
                d[k] = i32(v)
        return d

    def run(self, **kw):
        """The product's result as float64 numpy."""
        import torch

        import bit_block_scaled_nvfp4_amd as nv

        d = {**self.device(), **kw}
        fn = nv.nvfp4_kv_fp8_tree_attention if "tree_mask" in d else nv.nvfp4_kv_fp8_attention
        out = fn(**d)
        torch.cuda.synchronize()
        return out.double().cpu().numpy()


def _encode(x):
    """E4M3 codes of x, rounding toward zero in magnitude classes: any finite codes do for a cache."""
    import torch

    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def to_type(x, dtype):
    import torch

    td = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    return torch.from_numpy(np.asarray(x, np.float32)).to(td).to(torch.float32).numpy()


def unpack(mask):
    """Words of drafted-token bits as bool [tokens, 64 * words]."""
    m = np.asarray(mask).astype(np.int64).view(np.uint64)
    return ((m[:, :, None] >> np.arange(64, dtype=np.uint64)) & np.uint64(1)).astype(bool).reshape(len(m), -1)


def pack(bits):
    """Bool [tokens, drafted] as int64 words."""
    t, d = bits.shape
    words = max(1, -(-d // 64))
    full = np.zeros((t, 64 * words), np.uint64)
    full[:, :d] = bits
    return (full.reshape(t, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)


def tree_mask(rng, counts, words=None):
    """Random trees: each drafted token's ancestors and itself, one row of words a token."""
    most = max(list(counts) + [1])
    words = words or max(1, -(-most // 64))
    bits = np.zeros((int(sum(counts)), 64 * words), bool)
    t = 0
    for n in counts:
        for i in range(n):
            parent = int(rng.integers(-1, i)) if i else -1
            if parent >= 0:
                bits[t + i] = bits[t + parent]
            bits[t + i, i] = True
        t += n
    return pack(bits)


def compare(got, want, tol, what):
    assert got.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), (
        f"{what}: NaN in {int(np.isnan(got).sum())} elements, expected in {int(nan.sum())}; "
        f"first difference at {np.argwhere(np.isnan(got) != nan)[0].tolist()}")
    err = np.abs(np.where(nan, 0, got - want))
    lim = np.where(nan, 0, tol)
    bad = np.argwhere(err > lim)
    assert bad.size == 0, (f"{what}: {len(bad)} of {err.size} elements out of tolerance, first {bad[0].tolist()}: "
                           f"got {got[tuple(bad[0])]!r}, expected {want[tuple(bad[0])]!r} +- {lim[tuple(bad[0])]!r}")

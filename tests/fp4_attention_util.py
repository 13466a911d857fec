"""Seeded paged problems over the 4-bit cache, for the tests of its attentions: as ``attention_util.Problem``, with the
cache in blocks of codes and scales."""

from __future__ import annotations

import numpy as np

from oracle import attention as oa
from oracle import serving as osv

from .attention_util import EPS, SENTINEL, Problem, unpack


class Problem4(Problem):
    """Slots that no request owns hold the largest codes and scale bytes that there are (0x7F, or 0xFF: sign and
    all), so that a read of one shows."""

    def __init__(self, lens, heads=4, kv_heads=2, head_dim=64, block_size=16, **kw):
        super().__init__(lens, heads, kv_heads, head_dim, block_size, **kw)
        self.blocks = self.num_slots // block_size
        shape = (self.blocks, kv_heads, block_size)
        self.kc, self.vc = np.full((*shape, head_dim // 2), 0x77, np.uint8), np.full((*shape, head_dim // 2), 0xFF, np.uint8)
        self.kcs, self.vcs = np.full((*shape, head_dim // 16), 0x7F, np.uint8), np.full((*shape, head_dim // 16), 0xFF, np.uint8)
        self.kg, self.vg = np.float32(130.0), np.float32(410.0)
        for r in range(self.requests):
            s = oa.slots_of(self.table[r], int(self.seq_lens[r]), block_size, self.num_slots)
            b, o = s // block_size, s % block_size
            for codes, scales, g in ((self.kc, self.kcs, self.kg), (self.vc, self.vcs, self.vg)):
                x = self.rng.standard_normal((len(s), kv_heads, head_dim)) * 2.0
                c, sc = osv.encode4(x, g)
                codes[b, :, o], scales[b, :, o] = c, sc

    def place(self, request, position):
        """(block, place in it) of a position."""
        return int(self.table[request, position // self.block_size]), position % self.block_size

    def oracle(self):
        kw = dict(self.options)
        tree = kw.pop("tree_mask", None)
        if tree is not None:
            kw["tree"] = unpack(tree)
        rows = lambda c, s: osv.decode4(c, s).transpose(0, 2, 1, 3).reshape(self.num_slots, -1)  # noqa: E731
        out0 = np.full((self.tokens, self.heads, self.head_dim), SENTINEL)
        return oa.attention(self.q, rows(self.kc, self.kcs), rows(self.vc, self.vcs), 1.0 / float(self.kg), 1.0 / float(self.vg),
                            self.table, self.query_start, self.seq_lens, self.block_size, self.kv_heads, self.scale,
                            out=out0, out_eps=EPS[self.dtype], decode=lambda x, s: x * s, **kw)

    def device(self):
        import torch

        from .gpu_util import DEV

        td = {"bf16": torch.bfloat16, "f16": torch.float16}[self.dtype]
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).to(DEV)  # noqa: E731
        d = dict(q=torch.from_numpy(self.q).to(td).to(DEV), block_table=i32(self.table), query_start=i32(self.query_start),
                 seq_lens=i32(self.seq_lens), scale=self.scale,
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
        up = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
        d.update(key_codes=up(self.kc), key_scales=up(self.kcs), value_codes=up(self.vc), value_scales=up(self.vcs),
                 key_gscale=torch.tensor([self.kg], device=DEV), value_gscale=torch.tensor([self.vg], device=DEV))
        return d

    def run(self, **kw):
        import torch

        import bit_block_scaled_nvfp4_amd as nv

        d = {**self.device(), **kw}
        fn = nv.nvfp4_kv_fp4_tree_attention if "tree_mask" in d else nv.nvfp4_kv_fp4_attention
        out = fn(**d)
        torch.cuda.synchronize()
        return out.double().cpu().numpy()

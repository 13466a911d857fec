"""Measured calls of the operators of a serving step around the caches: norms and position rotation of
queries and keys, appending keys and values to the paged caches (FP8, or NVFP4: 4-bit codes with a scale for
each 16), attention over the 4-bit cache, and verification of drafted tokens.

``run`` computes them in plain torch operations, or, where ``own`` is true, through this
repository's entry points.  ``exact`` computes the definitions again in binary64.

A step runs them in this order: queries and keys are normed and rotated, keys and values appended, the
queries attend to the cache, and the drafted tokens that took part are verified against what came out.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    """Twelve cases.  24 heads over 4 KV heads of 256 dims, a quarter of them rotated, is the attention
    layer of this repository's KV workload (width 1024); the other layouts and the vocabularies are generic."""
    return [
        # one decode step of one request: the smallest call (latency)
        _rope("rope_decode_1", tokens=1, heads=24, kv_heads=4, head_dim=256, rotated=64, norm=True),
        # a whole prompt
        _rope("rope_prompt_8192", tokens=8192, heads=24, kv_heads=4, head_dim=256, rotated=64, norm=True),
        # a chunk of a long context, all dims rotated in neighbouring pairs, no norm, odd length
        _rope("rope_chunk_f16_pairs", tokens=3001, heads=32, kv_heads=8, head_dim=128, rotated=128, interleaved=True, dtype="f16", first=190000),
        # the new tokens of a decode batch, into the 4-bit cache and read back
        _append("append_fp4_decode_64", "fp4", tokens=64, kv_heads=4, head_dim=256, rotated=64, norm=True),
        # a long prompt into the 4-bit cache and read back: the largest append
        _append("append_fp4_prompt_16384", "fp4", tokens=16384, kv_heads=4, head_dim=256, rotated=64, norm=True),
        # a chunk into the FP8 cache, odd length, neighbouring pairs, no norm
        _append("append_fp8_chunk", "fp8", tokens=2047, kv_heads=8, head_dim=128, rotated=128, interleaved=True, dtype="f16", first=30000),
        # one chat request, one token, short context: the smallest attention call
        _attend("attend_one", requests=1, context=500, new=1, spread=0.0, heads=24, kv_heads=4, head_dim=256),
        # an ordinary decode batch of single tokens with ragged contexts
        _attend("attend_batch_64", requests=64, context=8000, new=1, spread=0.9, heads=24, kv_heads=4, head_dim=256),
        # a small drafted tree per request, half types, scores capped
        _attend("attend_tree_batch_16", requests=16, context=6001, new=12, spread=0.6, heads=32, kv_heads=8, head_dim=128, dtype="f16", cap=30.0, tree=True),
        # one chunk of a long prompt whose earlier chunks are in the cache: the largest call
        _attend("attend_chunk_2048", requests=1, context=30011, new=2048, spread=0.0, heads=24, kv_heads=4, head_dim=256),
        # one request with a few drafted tokens (latency)
        _verify("verify_1", requests=1, drafts=4, vocab=32000),
        # a batch with ragged drafts over a large vocabulary of odd size
        _verify("verify_batch_64", requests=64, drafts=8, vocab=131077),
    ]


def _rope(name, **kw):
    return {"name": name, "op": "rope", "dtype": "bf16", "norm": False, "interleaved": False, "first": 0, **kw}


def _append(name, cache, **kw):
    return {"name": name, "op": "append", "cache": cache, "dtype": "bf16", "norm": False, "interleaved": False, "first": 0, "block_size": 16, **kw}


def _attend(name, **kw):
    return {"name": name, "op": "attend", "dtype": "bf16", "cap": 0.0, "bias": False, "tree": False, "docs": False, "block_size": 16, "lens": 2, **kw}


def _verify(name, **kw):
    return {"name": name, "op": "verify", "sharp": 1.0, "lens": 3, **kw}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


HEADS = ((20, 4), (32, 8), (8, 8), (16, 1), (40, 8), (7, 1))


def draw(rng):
    """One more case: each operator equally often, sizes spread over their logarithm."""
    op = rng.choice(("rope", "append", "attend", "verify"))
    heads, kv_heads = rng.choice(HEADS)
    head_dim, dtype = rng.choice((64, 128, 256)), rng.choice(("bf16", "f16"))
    if op in ("rope", "append"):
        if op == "rope":
            head_dim, dtype = rng.choice((64, 80, 128, 192, 256)), rng.choice(("bf16", "bf16", "f16", "f32"))
        turned = {"norm": rng.random() < 0.6, "interleaved": rng.random() < 0.4, "first": rng.choice((0, 0, _log_int(rng, 1, 1000000))), "dtype": dtype}
        width = (heads + kv_heads if op == "rope" else 2 * kv_heads) * head_dim * (2 if dtype == "f32" else 1)
        tokens = _log_int(rng, 1, min(20000, (8192 * 28 * 256 if op == "rope" else 16384 * 2048) // width))
        if op == "rope":
            rotated = rng.choice((head_dim, head_dim, head_dim // 32 * 16))
            return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotated": rotated, **turned}
        return {"op": op, "cache": rng.choice(("fp4", "fp4", "fp8")), "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "rotated": rng.choice((head_dim, head_dim, head_dim // 2)),
                "block_size": rng.choice((8, 16, 48, 64, 256)), **turned}
    lens, spread = rng.randrange(1, 1 << 20), round(rng.uniform(0.0, 1.0), 3)
    if op == "verify":
        requests = _log_int(rng, 1, 96)
        vocab = _log_int(rng, 1000, min(160000, 64 * 9 * 131077 // (10 * requests)))
        return {"op": op, "requests": requests, "drafts": _log_int(rng, 1, max(1, min(24, 64 * 9 * 131077 // (requests * vocab) - 1))), "vocab": vocab, "sharp": round(rng.uniform(0.3, 4.0), 2), "lens": lens}
    case = {"op": op, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "block_size": rng.choice((8, 16, 48, 64, 256)),
            "lens": lens, "spread": spread, "cap": rng.choice((0.0, 0.0, 30.0)), "bias": rng.random() < 0.3, "tree": rng.random() < 0.3, "docs": False}
    kind, row = rng.choice(("decode", "decode", "prompt")), heads * head_dim
    if kind == "decode":
        requests, new = _log_int(rng, 1, 96), rng.choice((1, 1, _log_int(rng, 1, 32)))
        # at most the keys of the decode batch listed above and a quarter of the largest call's products
        most = min(480000 // requests, 2048 * 30011 * 24 * 64 // (requests * new * row), 60000)
        return {**case, "requests": requests, "new": new, "context": _log_int(rng, 1, max(1, most))}
    # padded to the longest request, at most a quarter of the largest call's products and scores
    requests, new = _log_int(rng, 1, 6), _log_int(rng, 33, 3000)
    while True:
        most = 2048 * 30011 * 24 // (4 * requests * new * max(heads, row // 256)) - new
        if most >= 0 or requests == 1:
            break
        requests = max(1, requests // 2)
    context = 0 if rng.random() < 0.4 or most < 1 else _log_int(rng, 1, min(most, 30000))
    return {**case, "requests": requests, "new": new, "context": context, "tree": False, "docs": rng.random() < 0.3}


def _lengths(case):
    """(context, new) of every request, from the case alone: between (1 - spread) of the named
    length and the length itself; the first request has both lengths in full."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for r in range(case["requests"]):
        a, b = (0.0, 0.0) if r == 0 else (rng.random(), rng.random())
        ctx.append(int(round(case["context"] * (1.0 - case["spread"] * a))))
        new.append(max(1, int(round(case["new"] * (1.0 - case["spread"] * b)))))
    return np.array(ctx, np.int64), np.array(new, np.int64)


def _doc_starts(case, ctx, new):
    """First position of the document that each new token belongs to: every request is cut into
    documents of 64 to 2048 tokens."""
    rng = random.Random(case["lens"] + 1)
    out = []
    for c, n in zip(ctx.tolist(), new.tolist()):
        cuts = [0]
        while cuts[-1] < c + n:
            cuts.append(cuts[-1] + _log_int(rng, 64, 2048))
        cuts = np.array(cuts)
        out.append(cuts[np.searchsorted(cuts, np.arange(c, c + n), side="right") - 1])
    return np.concatenate(out)


def _tree_bits(case, new):
    """Ancestor bits of each drafted token (itself among them) as int64, and its depth."""
    rng = random.Random(case["lens"] + 2)
    bits, depth = [], []
    for n in new.tolist():
        b, d = [], []
        for i in range(n):
            p = -1 if i == 0 else rng.randrange(max(0, i - 4), i)
            b.append((b[p] if p >= 0 else 0) | 1 << i)
            d.append(d[p] + 1 if p >= 0 else 0)
        bits += [x - (1 << 64) if x >> 63 else x for x in b]
        depth += d
    return np.array(bits, np.int64), np.array(depth, np.int64)


def _draft_counts(case):
    rng = random.Random(case["lens"])
    return [case["drafts"]] + [rng.randrange(0, case["drafts"] + 1) for _ in range(case["requests"] - 1)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": dict(case)}
    return {"rope": _prepare_rope, "append": _prepare_append, "attend": _prepare_attend, "verify": _prepare_verify}[case["op"]](case, s, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _prepare_turn(case, s, gen):
    """Positions, frequencies and a norm's weights, as a layer keeps them."""
    T, D = case["tokens"], case["head_dim"]
    s["positions"] = case["first"] + torch.arange(T, dtype=torch.int32, device=DEV)
    if T > 1:  # some requests' tokens begin anew
        s["positions"][T // 2:] = torch.arange(T - T // 2, dtype=torch.int32, device=DEV)
    n = case["rotated"] // 2
    s["inv_freq"] = (10000.0 ** (-torch.arange(n, device=DEV, dtype=torch.float64) / n)).float()
    s["q_weight"], s["k_weight"] = (0.2 * _randn(gen, D) if case["norm"] else None for _ in range(2))
    s["offset"], s["eps"] = 1.0, 1e-6


def _prepare_rope(case, s, gen):
    T, H, Hk, D, dt = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
    _prepare_turn(case, s, gen)
    # one fused row a token, as the projection leaves it: queries, keys, values
    row = (2.0 * _randn(gen, T, (H + 2 * Hk) * D)).to(dt)
    s["q"] = row[:, :H * D].unflatten(1, (H, D))
    s["k"] = row[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    s["q_out"], s["k_out"] = (torch.empty((T, n, D), dtype=dt, device=DEV) for n in (H, Hk))
    return s


def _prepare_append(case, s, gen):
    T, Hk, D, bs, dt = case["tokens"], case["kv_heads"], case["head_dim"], case["block_size"], TYPES[case["dtype"]]
    _prepare_turn(case, s, gen)
    k = _randn(gen, T, Hk * D)
    k[:, torch.randperm(Hk * D, generator=gen, device=DEV)[: Hk * D // 50 + 1]] *= 8.0  # a few hot key channels
    v = _randn(gen, T, Hk * D)
    row = torch.cat([k, v], 1).to(dt)
    s["key"], s["value"] = row[:, :Hk * D].unflatten(1, (Hk, D)), row[:, Hk * D:].unflatten(1, (Hk, D))
    blocks = -(-T // bs) + 5
    order = torch.randperm(blocks, generator=gen, device=DEV)
    t = torch.arange(T, device=DEV)
    s["slots"] = order[t // bs] * bs + t % bs
    s["slots"][1::97] = -1  # padding tokens
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=DEV)  # noqa: E731
    one = lambda x: torch.full((1,), x, dtype=torch.float32, device=DEV)  # noqa: E731
    if case["cache"] == "fp8":
        s["kc"], s["vc"] = u8(blocks * bs, Hk * D), u8(blocks * bs, Hk * D)
        s["ks"], s["vs"] = one(48.0 / 448.0), one(6.0 / 448.0)  # calibrated: amax / 448
    else:
        s["kc"], s["vc"] = u8(blocks, Hk, bs, D // 2), u8(blocks, Hk, bs, D // 2)
        s["kcs"], s["vcs"] = u8(blocks, Hk, bs, D // 16), u8(blocks, Hk, bs, D // 16)
        s["ks"], s["vs"] = one(2688.0 / 48.0), one(2688.0 / 6.0)  # calibrated: 2688 / amax
        s["k_read"], s["v_read"] = (torch.empty((T, Hk, D), dtype=torch.float32, device=DEV) for _ in range(2))
    return s


def _prepare_attend(case, s, gen):
    ctx, new = _lengths(case)
    R, bs = len(ctx), case["block_size"]
    total = ctx + new
    need = -(-total // bs)
    width = int(need.max()) + 2
    dev32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(device=DEV, dtype=torch.int32)  # noqa: E731
    H, Hk, D, dt = case["heads"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
    blocks = int(need.sum()) + 37
    shuffled = torch.randperm(blocks, generator=gen, device=DEV, dtype=torch.int64).to(torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    table[dev32(np.arange(width)[None, :] < need[:, None]).bool()] = shuffled[: int(need.sum())]
    # N(0, 1) keys and values with a few hot key channels, held as the cache holds them; head by head, for
    # the room that their encoding takes
    s["kc"], s["vc"] = (torch.empty((blocks, Hk, bs, D // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    s["kcs"], s["vcs"] = (torch.empty((blocks, Hk, bs, D // 16), dtype=torch.uint8, device=DEV) for _ in range(2))
    s["kg"], s["vg"] = (torch.full((1,), 2688.0 / amax, dtype=torch.float32, device=DEV) for amax in (48.0, 6.0))
    for h in range(Hk):
        k = _randn(gen, blocks, bs, D)
        k[..., torch.randperm(D, generator=gen, device=DEV)[: D // 50 + 1]] *= 8.0
        s["kc"][:, h], s["kcs"][:, h] = _encode4(k, s["kg"])
        s["vc"][:, h], s["vcs"][:, h] = _encode4(_randn(gen, blocks, bs, D), s["vg"])
    T = int(new.sum())
    s.update(
        R=R, T=T, q=_randn(gen, T, H, D).to(dt), block_table=table,
        query_start=dev32(np.concatenate([[0], np.cumsum(new)])), seq_lens=dev32(total), scale=D ** -0.5, cap=case["cap"],
        max_query_len=int(new.max()), max_seq_len=int(total.max()),
        slopes=(2.0 ** (-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)) if case["bias"] else None)
    if case["tree"]:
        bits, depth = _tree_bits(case, new)
        s["tree_mask"] = torch.from_numpy(bits).to(DEV).reshape(-1, 1)
        s["tree_positions"] = dev32(np.repeat(ctx, new) + depth)
    s["doc_start"] = dev32(_doc_starts(case, ctx, new)) if case["docs"] else None
    return s


def _prepare_verify(case, s, gen):
    counts = np.array(_draft_counts(case), np.int64)
    rows, R, V = int(counts.sum()) + len(counts), len(counts), case["vocab"]
    # the target's distribution, and a draft's that is like it: they agree about as often as a good draft does
    logits = case["sharp"] * _randn(gen, rows, V) + 6.0 * (_randn(gen, rows, V) > 3.0)
    s["target"] = torch.softmax(logits, 1)
    s["draft"] = torch.softmax(logits + 0.5 * _randn(gen, rows, V), 1)
    start = np.concatenate([[0], np.cumsum(counts + 1)])
    s["query_start"] = torch.from_numpy(start).to(device=DEV, dtype=torch.int32)
    # token i + 1 of a request was drawn from the draft's row i
    s["tokens"] = torch.multinomial(s["draft"], 1, generator=gen).reshape(-1).roll(1).to(torch.int32)
    s["accept_u"] = torch.rand(rows, generator=gen, device=DEV)
    s["sample_u"] = torch.rand(R, generator=gen, device=DEV)
    s["accepted"] = torch.empty(R, dtype=torch.int32, device=DEV)
    s["out"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "verify": _own_verify}[op](s)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}[op](s)


def _turn_words(s):
    return {"eps": s["eps"], "weight_offset": s["offset"], "interleaved": s["case"]["interleaved"]}


def _own_rope(s):
    import bit_block_scaled_nvfp4_amd as nv

    return nv.nvfp4_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], q_out=s["q_out"], k_out=s["k_out"], **_turn_words(s))


def _own_append(s):
    import bit_block_scaled_nvfp4_amd as nv

    kw = {"k_weight": s["k_weight"], **_turn_words(s)}
    if s["case"]["cache"] == "fp8":
        nv.nvfp4_kv_fp8_append(s["key"], s["value"], s["positions"], s["inv_freq"], s["ks"], s["vs"], s["kc"], s["vc"], s["slots"], **kw)
        return [s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn)]
    nv.nvfp4_kv_fp4_append(s["key"], s["value"], s["positions"], s["inv_freq"], s["ks"], s["vs"], s["kc"], s["kcs"], s["vc"], s["vcs"], s["slots"], **kw)
    return [nv.nvfp4_kv_fp4_load(s["kc"], s["kcs"], s["ks"], s["slots"], out=s["k_read"]), nv.nvfp4_kv_fp4_load(s["vc"], s["vcs"], s["vs"], s["slots"], out=s["v_read"])]


def _own_attend(s):
    import bit_block_scaled_nvfp4_amd as nv

    args = (s["q"], s["kc"], s["kcs"], s["vc"], s["vcs"], s["kg"], s["vg"], s["block_table"], s["query_start"], s["seq_lens"])
    kw = {"scale": s["scale"], "softcap": s["cap"], "slopes": s["slopes"], "max_query_len": s["max_query_len"], "max_seq_len": s["max_seq_len"]}
    if s["case"]["tree"]:
        return nv.nvfp4_kv_fp4_tree_attention(*args, s["tree_mask"], positions=s["tree_positions"], **kw)
    return nv.nvfp4_kv_fp4_attention(*args, doc_start=s["doc_start"], **kw)


def _own_verify(s):
    import bit_block_scaled_nvfp4_amd as nv

    return nv.nvfp4_verify_drafted(s["target"], s["draft"], s["tokens"], s["query_start"], s["accept_u"], s["sample_u"], accepted=s["accepted"], out=s["out"])


# ---- plain forms ------------------------------------------------------------------------------


def _turned(x, weight, s, wide):
    """Heads ``x [tokens, heads, head_dim]`` normed and rotated, in 32 or 64 bits (angles always in 64)."""
    x = x.to(wide)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * (s["offset"] + weight.to(wide))
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().to(wide)[:, None], angle.sin().to(wide)[:, None]
    n = s["inv_freq"].numel()
    if s["case"]["interleaved"]:
        a, b = x[..., :2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _plain_rope(s):
    return [_turned(s[n], s[n + "_weight"], s, torch.float32).to(s[n].dtype) for n in ("q", "k")]


def _once(x, dtype):
    """64 bits to ``dtype`` in one rounding: cut to 32 bits with the last bit set where anything is lost,
    which leaves the next rounding to nearest what it has to know."""
    f = x.float()
    back = f.double()
    bits = f.view(torch.int32) - (back.abs() > x.abs()).int()
    return (bits | (back != x).int()).view(torch.float32).to(dtype)


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode4(x, g):
    """NVFP4 codes (two a byte, the even element low) and scales of ``x [..., 16 n]``: the block's largest
    magnitude times g / 6 as E4M3, elements times g over that as E2M1, ties to the even code."""
    v = x.float().unflatten(-1, (-1, 16))
    s = (v.abs().amax(-1) * (g / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sd = s.float()
    r = torch.where(sd > 0, (g.double() / sd.double()).float(), 0.0)
    y = (v.abs() * r[..., None])
    c = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for middle, low in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        c += y > middle if low else y >= middle
    c += 8 * torch.signbit(v)
    c = c.flatten(-2)
    return c[..., 0::2] | c[..., 1::2] << 4, s.view(torch.uint8)


def _values4(codes, scales):
    """What codes and scales stand for, but for the global scale."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), device=codes.device)
    pairs = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    return grid[pairs] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _plain_append(s):
    # in 64 bits and rounded once to the keys' type: what follows are steps, and a value next to one falls on a side
    key = _once(_turned(s["key"], s["k_weight"], s, torch.float64), s["key"].dtype)
    kept = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][kept]
    if s["case"]["cache"] == "fp8":
        for x, cache, scale in ((key, s["kc"], s["ks"]), (s["value"], s["vc"], s["vs"])):
            codes = (x[kept].flatten(1).float() * (1.0 / scale.double()).float()).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            cache[slot] = codes.view(torch.uint8)
        return [s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn)]
    bs, got = s["case"]["block_size"], []
    for x, cache, scales, g in ((key, s["kc"], s["kcs"], s["ks"]), (s["value"], s["vc"], s["vcs"], s["vs"])):
        cache[slot // bs, :, slot % bs], scales[slot // bs, :, slot % bs] = _encode4(x[kept], g)
        back = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        back[kept] = (_values4(cache[slot // bs, :, slot % bs], scales[slot // bs, :, slot % bs]).double() / g.double()).float()
        got.append(back)
    return got


def _plain_attend(s):
    q, bs, dev = s["q"], s["case"]["block_size"], s["q"].device
    T, H, D = q.shape
    Hk = s["kc"].shape[1]
    R, G, n, L = s["R"], H // Hk, s["max_query_len"], s["max_seq_len"]
    start, lens = s["query_start"].long(), s["seq_lens"].long()
    count = start[1:] - start[:-1]
    ctx = lens - count
    j = torch.arange(L, device=dev)
    i = torch.arange(n, device=dev)
    block, off = s["block_table"].long()[:, j // bs], (j % bs).expand(R, L)
    there = j[None, :] < lens[:, None]
    block = torch.where(there & (block >= 0), block, 0)
    k = (_values4(s["kc"][block, :, off], s["kcs"][block, :, off]) / s["kg"]).permute(0, 2, 3, 1).contiguous()
    v = (_values4(s["vc"][block, :, off], s["vcs"][block, :, off]) / s["vg"]).permute(0, 2, 1, 3).contiguous()
    token = (start[:-1, None] + i).clamp(max=T - 1)  # [R, n]
    qq = q.float()[token].reshape(R, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hk, G * n, D).contiguous()
    x = torch.matmul(qq, k).reshape(R, H, n, L) * s["scale"]
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    drafted = j[None, :] - ctx[:, None]  # [R, L]: number of the drafted token at a key, or below 0
    if s["case"]["tree"]:
        bit = (s["tree_mask"][token][..., :1] >> drafted.clamp(0, 63)[:, None, :]) & 1
        see = there[:, None, :] & ((drafted < 0)[:, None, :] | (bit == 1))
        at = s["tree_positions"].long()[token]  # [R, n]
        kat = torch.where(drafted < 0, j[None, :], at.gather(1, drafted.clamp(0, n - 1)))
    else:
        at = ctx[:, None] + i
        kat = j[None, :].expand(R, L)
        see = (j[None, None, :] <= at[:, :, None]) & there[:, None, :]
        if s["doc_start"] is not None:
            see = see & (j[None, None, :] >= s["doc_start"].long()[token][:, :, None])
    if s["slopes"] is not None:
        x = x + s["slopes"][None, :, None, None] * (kat[:, None, :] - at[:, :, None]).float()[:, None]
    x = torch.where(see[:, None], x, -math.inf)
    top = x.max(-1, keepdim=True).values
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(R, Hk, G * n, L), v).reshape(R, H, n, D) / torch.where(total == 0, 1.0, total)
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(start, t, right=True) - 1
    return o[r, :, t - start[r]].to(q.dtype)


def _plain_verify(s):
    p, q, start, dev = s["target"], s["draft"], s["query_start"].long(), s["target"].device
    rows, R = p.shape[0], start.numel() - 1
    t = torch.arange(rows, device=dev)
    r = torch.searchsorted(start, t, right=True) - 1
    # the drafted token behind row t is the request's next input token; the last row has none
    follows = t + 1 < start[r + 1]
    token = s["tokens"].long().roll(-1)
    at = token[:, None].clamp(0, p.shape[1] - 1)
    # products of 32-bit numbers, whole in 64
    yes = follows & (s["accept_u"].double() * q.gather(1, at)[:, 0].double() < p.gather(1, at)[:, 0].double())
    stop = torch.where(yes, rows, t)
    end = torch.full((R,), rows, dtype=torch.int64, device=dev).scatter_reduce(0, r, stop, "amin")  # first row that goes no further
    pe = p[end].double()
    left = torch.where(follows[end][:, None], (pe - q[end].double()).clamp(min=0.0), pe)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, pe)
    upto = left.cumsum(1)
    pick = (upto > s["sample_u"].double()[:, None] * upto[:, -1:]).to(torch.uint8).argmax(1)
    out = torch.where(t < end[r], token, -1)
    out[end] = pick
    return [(end - start[:-1]).int(), out.int()]


# ---- work and exact values --------------------------------------------------------------------


def _visible(case):
    """Number of (query token, key) pairs that are attended, and of keys that any token attends."""
    ctx, new = _lengths(case)
    total = ctx + new
    if case["tree"]:
        bits, _ = _tree_bits(case, new)
        return int((ctx * new).sum()) + sum(bin(b & (1 << 64) - 1).count("1") for b in bits.tolist()), int(total.sum())
    end = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx.tolist(), new.tolist())]) + 1
    first = _doc_starts(case, ctx, new) if case["docs"] else np.zeros_like(end)
    at = np.concatenate([[0], np.cumsum(new)[:-1]])
    return int((end - first).clip(0).sum()), int((total - np.minimum.reduceat(first, at)).sum())


def work(case):
    if case["op"] == "rope":
        T, n = case["tokens"], (case["heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": T * (2 * n * (4 if case["dtype"] == "f32" else 2) + 4), "flops": 0}
    if case["op"] == "append":
        T, n = case["tokens"], case["kv_heads"] * case["head_dim"]
        # keys and values in, codes out; in 4 bits with their scales, and read again as 32-bit numbers
        return {"bytes": T * (2 * n * 2 + 12 + (2 * n if case["cache"] == "fp8" else 2 * n * 9 // 16 * 2 + 2 * n * 4)), "flops": 0}
    if case["op"] == "verify":
        counts = _draft_counts(case)
        # a request that takes all its drafts reads one row, the others two: most stop before the end
        return {"bytes": sum(4 * case["vocab"] * (2 if n else 1) + 20 * n + 16 for n in counts), "flops": 0}
    ctx, new = _lengths(case)
    pairs, keys = _visible(case)
    T, H, Hk, D = int(new.sum()), case["heads"], case["kv_heads"], case["head_dim"]
    return {"bytes": 2 * T * H * D * 2 + keys * Hk * D * 2 * 9 // 16 + 4 * (keys // case["block_size"] + 2 * len(ctx)) + (12 * T if case["tree"] else 0), "flops": 4 * pairs * H * D}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](s)


def _exact_turned(x, weight, s):
    """Pairs as complex numbers times exp(i angle)."""
    x = x.double().clone()
    if weight is not None:
        x *= ((s["offset"] + weight.double()) / (x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt())
    n = s["inv_freq"].numel()
    pairs = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
    if not s["case"]["interleaved"]:
        pairs = slice(0, n), slice(n, 2 * n)
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    z = torch.complex(x[..., pairs[0]].contiguous(), x[..., pairs[1]].contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
    return x


def _exact_rope(s):
    return [_exact_turned(s[n], s[n + "_weight"], s) for n in ("q", "k")]


def _nearest(x, grid):
    """Index of the grid's value nearest to each ``x >= 0``, ties to the even index (values 0 to 6 or 448 and
    beyond: the last); ``grid`` rises."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(x, middle), torch.bucketize(x, middle, right=True)
    return torch.where(below % 2 == 0, below, above)


E4M3 = tuple(m * 2.0 ** -9 for m in range(8)) + tuple((8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7))


def _rounded(x, dtype):
    """``x`` in 64 bits to the nearest number of ``dtype``, ties to even, in 64 bits."""
    low, high = {torch.bfloat16: (-126, 7), torch.float16: (-14, 10)}[dtype]
    e = torch.frexp(torch.where(x == 0, 1.0, x))[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=low) - high)
    return (x / step).round() * step


def _exact_append(s):
    case = s["case"]
    key = _rounded(_exact_turned(s["key"], s["k_weight"], s), s["key"].dtype)
    T, Hk, D = key.shape
    table = torch.tensor(E4M3, dtype=torch.float64, device=DEV)
    kept = s["slots"] >= 0
    got = []
    for x, scale, cache in ((key, s["ks"], s["kc"]), (s["value"].double(), s["vs"], s["vc"])):
        if case["cache"] == "fp8":
            y = (x.float() * (1.0 / scale.double()).float()).double().flatten(1)
            whole = torch.zeros(cache.shape, dtype=torch.float64, device=DEV)
            whole[s["slots"][kept]] = (table[_nearest(y.abs(), E4M3)] * y.sign())[kept]
            got.append(whole)
            continue
        v = x.float().reshape(T, Hk, D // 16, 16)
        sd = table[_nearest((v.abs().max(-1).values * (scale / 6.0)).double(), E4M3)]
        r = torch.where(sd > 0, scale.double() / torch.where(sd > 0, sd, 1.0), 0.0).float()
        y = (v.abs() * r[..., None]).double()
        y = torch.tensor(GRID, dtype=torch.float64, device=DEV)[_nearest(y, GRID)] * v.sign() * sd[..., None] / scale.double()
        got.append(torch.where(kept[:, None, None], y.reshape(T, Hk, D), 0.0))
    return got


def _exact_attend(s):
    """Request by request and head by head, blocks of 1024 query tokens, in binary64."""
    case = s["case"]
    ctx, new = _lengths(case)
    H, Hk, D, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    byte = torch.arange(256, device=DEV)
    grid = torch.tensor(GRID, dtype=torch.float64, device=DEV)
    both = torch.stack([grid[byte % 8] * torch.where(byte % 16 < 8, 1.0, -1.0), grid[byte // 16 % 8] * torch.where(byte < 128, 1.0, -1.0)], 1)
    step = torch.tensor(E4M3, dtype=torch.float64, device=DEV)
    out = torch.zeros((s["T"], H, D), dtype=torch.float64, device=DEV)
    bits, depth = _tree_bits(case, new) if case["tree"] else (None, None)
    docs = _doc_starts(case, ctx, new) if case["docs"] else None
    t0 = 0
    for r in range(len(ctx)):
        c, n = int(ctx[r]), int(new[r])
        key = torch.arange(c + n, device=DEV)
        block, off = s["block_table"][r].long().repeat_interleave(bs)[: c + n], key % bs
        kat = key.clone()
        if bits is not None:
            kat[c:] = c + torch.from_numpy(depth[t0:t0 + n]).to(DEV)
        for b in range(0, n, 1024):
            i = torch.arange(b, min(n, b + 1024), device=DEV)
            if bits is not None:
                see = torch.ones((len(i), c + n), dtype=torch.bool, device=DEV)
                word = torch.from_numpy(bits[t0 + b:t0 + b + len(i)]).to(DEV)
                see[:, c:] = (word[:, None] >> torch.arange(n, device=DEV)) & 1 == 1
            else:
                see = key <= c + i[:, None]
                if docs is not None:
                    see &= key >= torch.from_numpy(docs[t0 + b:t0 + b + len(i)]).to(DEV)[:, None]
            far = (kat - kat[c + i][:, None]).double()
            for h in range(H):
                g = h // (H // Hk)
                if h % (H // Hk) == 0:
                    kk, vv = ((both[codes[block, g, off].long()].flatten(1).reshape(c + n, D // 16, 16) * step[scales[block, g, off].long()][..., None]).reshape(c + n, D) / by.double()
                              for codes, scales, by in ((s["kc"], s["kcs"], s["kg"]), (s["vc"], s["vcs"], s["vg"])))
                x = s["q"][t0 + i, h].double() @ kk.t().contiguous() * s["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if s["slopes"] is not None:
                    x += s["slopes"][h].double() * far
                x[~see] = -math.inf
                out[t0 + i, h] = torch.nan_to_num(torch.softmax(x, -1)) @ vv
        t0 += n
    return out


def _exact_verify(s):
    """Request by request, token by token, on the host."""
    start, tokens, u, w = (s[n].tolist() for n in ("query_start", "tokens", "accept_u", "sample_u"))
    accepted, out = [], [-1] * start[-1]
    for r in range(len(start) - 1):
        row, last = start[r], start[r + 1] - 1
        while row < last and u[row] * s["draft"][row, tokens[row + 1]].item() < s["target"][row, tokens[row + 1]].item():
            out[row] = tokens[row + 1]
            row += 1
        accepted.append(row - start[r])
        p = s["target"][row].cpu().numpy().astype(np.float64)
        left = np.maximum(p - s["draft"][row].cpu().numpy(), 0.0) if row < last else p
        upto = np.cumsum(left if left.any() else p)
        out[row] = int(np.searchsorted(upto, w[r] * upto[-1], side="right"))
    return [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (accepted, out)]

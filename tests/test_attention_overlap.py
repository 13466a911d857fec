"""Results that share memory with inputs or with one another: in nvfp4_kv_block_tables workgroups read the lengths while
others write results, in the attentions rows are read and written in any order, so the binding refuses
such calls (CPU: the library call is replaced by a recorder; the tensors have memory, and claim to
live on the GPU)."""

import os

import pytest

import bit_block_scaled_nvfp4_amd as nv
from bit_block_scaled_nvfp4_amd import attention as at

from .test_attention_abi import _Dev, _gpu_visible

pytestmark = [
    pytest.mark.skipif(not os.path.exists(nv.LIB_PATH), reason="libnvfp4.so not built"),
    pytest.mark.skipif(_gpu_visible(), reason="host-only checks"),
]

R, W, T, F = 6, 4, 40, 30
OUTPUTS = {"slot_mapping": T, "positions": T, "query_start": R + 1, "seq_lens": R, "blocks_needed": 1}


@pytest.fixture
def call(monkeypatch):
    import torch

    seen = []
    monkeypatch.setattr(at, "_call", lambda device, fn, *args: seen.append(args))

    def make(**kw):
        z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt)  # noqa: E731
        a = dict(context_lens=z(R), query_lens=z(R), free_blocks=z(F), block_table=z((R, W)), block_size=16, max_tokens=T,
                 free_start=z(1))
        a.update(kw)
        a["context_lens"] = _Dev(a["context_lens"])
        n = len(seen)
        out = nv.nvfp4_kv_block_tables(**a)
        assert len(seen) == n + 1
        return out

    make.seen = seen
    return make


def _buffer(n):
    import torch

    return torch.zeros(n, dtype=torch.int32)


@pytest.mark.parametrize("given", ["context_lens", "query_lens", "free_blocks", "free_start"])
@pytest.mark.parametrize("result", ["positions", "query_start", "seq_lens", "blocks_needed"])
@pytest.mark.parametrize("whole", [True, False])
def test_a_result_that_shares_memory_with_an_input_is_refused(call, given, result, whole):
    """The same tensor, or the last element of one and the first of the other."""
    size = {"context_lens": R, "query_lens": R, "free_blocks": F, "free_start": 1}[given]
    n = OUTPUTS[result]
    buf = _buffer(size + n)
    first, second = buf[:size], (buf[:n] if whole else buf[size - 1:size - 1 + n])
    with pytest.raises(ValueError, match=result):
        call(**{given: first, result: second})
    assert not call.seen
    call(**{given: first, result: buf[size:size + n]})  # next to each other


@pytest.mark.parametrize("result", ["query_start", "seq_lens", "blocks_needed"])
def test_results_that_share_memory_with_one_another_are_refused(call, result):
    import torch

    n = OUTPUTS[result]
    buf = _buffer(T + n)
    with pytest.raises(ValueError, match="positions"):
        call(positions=buf[:T], **{result: buf[T - 1:T - 1 + n]})
    slots = torch.zeros(T, dtype=torch.int64)
    with pytest.raises(ValueError, match="slot_mapping"):
        call(slot_mapping=slots, **{result: slots.view(torch.int32)[2 * T - n:]})
    assert not call.seen
    call(positions=buf[:T], slot_mapping=slots, **{result: buf[T:]})


def test_the_lengths_of_the_last_step_are_not_updated_in_place(call):
    lens = _buffer(R)
    with pytest.raises(ValueError, match="seq_lens"):
        call(context_lens=lens, seq_lens=lens)
    taken = _buffer(1)
    with pytest.raises(ValueError, match="blocks_needed"):
        call(free_start=taken, blocks_needed=taken)


def test_a_table_that_shares_memory_is_refused(call):
    buf = _buffer(R * (W + 3) + R)
    table = buf[: R * (W + 3)].view(R, W + 3)[:, :W]
    for kw in (dict(context_lens=buf[:R]), dict(free_blocks=buf[8:8 + F]), dict(seq_lens=buf[(R - 1) * (W + 3):][:R]),
               dict(blocks_needed=buf[W + 3 + 1:][:1]), dict(query_lens=buf[W - 1:][:R])):
        with pytest.raises(ValueError, match="block_table"):
            call(block_table=table, **kw)
    assert not call.seen


def test_what_does_not_overlap_is_taken(call):
    """Inputs may share memory; results may lie next to each other, or between the rows of a table."""
    import torch

    lens = _buffer(R)
    call(context_lens=lens, query_lens=lens)
    buf = _buffer(R * (W + 3) + R)
    table = buf[: R * (W + 3)].view(R, W + 3)[:, :W]
    call(block_table=table, seq_lens=buf[R * (W + 3):])
    for row in range(R - 1):
        call(block_table=table, blocks_needed=buf[row * (W + 3) + W + 2:][:1])
    call(block_table=table, free_start=buf[W:][:1], blocks_needed=buf[W + 1:][:1])
    call(block_table=buf[: R * W].view(R, W)[:, :0], seq_lens=buf[2:2 + R])  # nothing of the table is touched
    slots = _buffer(2 * T).view(dtype=torch.int64)
    call(free_blocks=slots.view(lens.dtype)[6:6], slot_mapping=slots)  # an empty list has no memory
    call(block_table=buf[: R * (W + 3)].view(R, W + 3)[:, :W], free_blocks=buf[2:2])


@pytest.fixture
def attend(monkeypatch):
    import torch

    seen = []
    monkeypatch.setattr(at, "_call", lambda device, fn, *args: seen.append(args))

    def make(q, out, which="prompt"):
        i32, u8 = torch.int32, torch.uint8
        z = lambda n, dt=i32: torch.zeros(n, dtype=dt)  # noqa: E731
        a = dict(q=_Dev(q), key_cache=z((32, 128), u8), value_cache=z((32, 128), u8), key_scale=torch.ones(1), value_scale=torch.ones(1),
                 block_table=z((2, 3)), query_start=z(3), seq_lens=z(2), block_size=16, num_kv_heads=2, max_seq_len=48, out=out)
        if which == "tree":
            return nv.nvfp4_kv_fp8_tree_attention(**a, tree_mask=torch.zeros((q.shape[0], 1), dtype=torch.int64))
        return nv.nvfp4_kv_fp8_attention(**a)

    make.seen = seen
    return make


@pytest.mark.parametrize("which", ["prompt", "tree"])
def test_an_output_that_overlaps_the_query_is_refused(attend, which):
    """Rows are read and written by different workgroups in any order: the output is the query itself or elsewhere."""
    import torch

    tokens, heads, dim = 6, 4, 64
    n = heads * dim
    buf = torch.zeros(tokens * n + 8 * n, dtype=torch.bfloat16)
    q = buf[: tokens * n].view(tokens, heads, dim)
    for out in (buf[n:][: tokens * n].view(tokens, heads, dim),  # a token further
                buf[dim:][: tokens * n].view(tokens, heads, dim),  # a head further
                buf[tokens * n - 8:][: tokens * n].view(tokens, heads, dim),  # the last elements
                q.transpose(0, 1).reshape(-1)[:0].new_zeros(0).set_(buf.untyped_storage(), 0, (tokens, heads, dim), (dim, tokens * dim, 1))):
        with pytest.raises(ValueError, match="out"):
            attend(q, out, which)
    one = buf[:n].view(1, heads, dim).expand(tokens, heads, dim)  # one token's query for all
    with pytest.raises(ValueError, match="out"):
        attend(one, q, which)
    assert not attend.seen


@pytest.mark.parametrize("which", ["prompt", "tree"])
def test_outputs_beside_the_query_are_taken(attend, which):
    import torch

    tokens, heads, dim = 6, 4, 64
    n = heads * dim
    buf = torch.zeros(tokens * 3 * n, dtype=torch.bfloat16)
    rows = buf.view(tokens, 3 * heads, dim)
    q = rows[:, :heads]
    for out in (q, rows[:, heads:2 * heads], rows[:, 2 * heads:], torch.zeros(tokens, heads, dim, dtype=torch.bfloat16)):
        assert attend(q, out, which) is out
    assert attend(rows[:, 2 * heads:], rows[:, :heads], which) is not None  # before the query
    flat = buf[: 2 * tokens * n]
    attend(flat[: tokens * n].view(tokens, heads, dim), flat[tokens * n:].view(tokens, heads, dim), which)
    attend(flat[: tokens * n].view(heads, tokens, dim).transpose(0, 1), flat[tokens * n:].view(heads, tokens, dim).transpose(0, 1), which)
    head = buf[: tokens * 2 * n].view(heads, 2 * tokens, dim).transpose(0, 1)  # head-major, tokens of both in turn
    attend(head[:tokens], head[tokens:], which)
    attend(q[:0], q[:0], which)
    attend(q[:1], rows[1:2, :heads], which)


def test_the_rule_for_rows_against_their_elements():
    """Random layouts of both tensors in one small buffer, element by element."""
    import random

    import torch

    rng = random.Random(3)
    buf = torch.zeros(2000, dtype=torch.bfloat16)
    D = 8
    refused = 0
    for _ in range(3000):
        T, H = rng.randrange(1, 5), rng.randrange(1, 5)

        def layout():
            a, b = (T, H) if rng.random() < 0.5 else (H, T)
            inner = D + rng.choice([0, 0, 8, D])
            outer = (b - 1) * inner + D + rng.choice([0, 0, 8, 3 * D, b * inner])
            return rng.choice([(outer, inner) if a == T else (inner, outer), (rng.choice([0, D, 2 * D]), rng.choice([0, D]))])

        x = layout()
        y = layout() if rng.random() < 0.4 else x
        at_x, at_y = rng.randrange(40) * 8, rng.randrange(40) * 8 + rng.choice([0, 0, 0, 1, 4])
        places = [{o + t * ts + h * hs + d for t in range(T) for h in range(H) for d in range(D)} for o, (ts, hs) in ((at_x, x), (at_y, y))]
        effective = [(ts if T > 1 else H * D, hs if H > 1 else D) for ts, hs in (x, y)]
        want = bool(places[0] & places[1]) and not (at_x == at_y and effective[0] == effective[1])
        q, out = (buf.as_strided((T, H, D), (*s, 1), o) for o, s in ((at_x, x), (at_y, y)))
        if want:
            refused += 1
            with pytest.raises(ValueError):
                at._refuse_overlap_of_rows(q, effective[0], out, effective[1])
        else:
            at._refuse_overlap_of_rows(q, effective[0], out, effective[1])
    assert 300 < refused < 2700

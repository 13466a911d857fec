"""Results of nvfp4_kv_block_tables that share memory with its inputs or with one another: the workgroups of the one
launch read the lengths while others write results, so the binding refuses such calls (CPU: the library
call is replaced by a recorder; the tensors have memory, and claim to live on the GPU)."""

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

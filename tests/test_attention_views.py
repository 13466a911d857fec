"""Which views of block tables and drafted-tree masks the binding of the cache's attention operators takes, and
the row pitch that it hands to the library for them (CPU: the library call is replaced by a recorder).

Rows that share memory (an expanded row, overlapping windows) have no pitch that the library could take: a
pitch of the row's length instead would reach past the allocation."""

import os

import pytest

import bit_block_scaled_nvfp4_amd as nv
from bit_block_scaled_nvfp4_amd import attention as at

from .test_attention_abi import _Dev, _gpu_visible, _t

pytestmark = [
    pytest.mark.skipif(not os.path.exists(nv.LIB_PATH), reason="libnvfp4.so not built"),
    pytest.mark.skipif(_gpu_visible(), reason="host-only checks on tensors without memory"),
]


def _window(rows, width, pitch, dtype):
    return _t((max(1, rows) * max(1, pitch) + width,), dtype).as_strided((rows, width), (pitch, 1))


@pytest.fixture
def calls(monkeypatch):
    """The arguments of every library call, which is not made."""
    seen = []
    monkeypatch.setattr(at, "_call", lambda device, fn, *args: seen.append(args))
    return seen


def _tables(table, rows):
    import torch

    i32 = torch.int32
    return nv.nvfp4_kv_block_tables(_Dev(_t((rows,), i32)), _t((rows,), i32), _t((9,), i32), table, 16, 8)


def _attend(which, rows=8, table=None, mask=None):
    import torch

    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    a = dict(q=_Dev(_t((rows, 4, 64), torch.bfloat16)), key_cache=_t((32, 128), u8), value_cache=_t((32, 128), u8),
             key_scale=_t((1,), f32), value_scale=_t((1,), f32), block_table=_t((rows, 3), i32) if table is None else table,
             query_start=_t((rows + 1,), i32), seq_lens=_t((rows,), i32), block_size=16, num_kv_heads=2, max_seq_len=48)
    if which == "tree":
        a["tree_mask"] = _t((rows, 1), torch.int64) if mask is None else mask
        return nv.nvfp4_kv_fp8_tree_attention(**a)
    return nv.nvfp4_kv_fp8_attention(**a)


#: (rows, width, pitch) of views whose rows share elements
SHARED = [(8, 5, 0), (8, 5, 1), (8, 5, 4), (8, 1, 0), (2, 3, 2), (64, 1, 0)]
#: views that are taken, and the pitch that goes to the library
TAKEN = [((8, 5, 5), 5), ((8, 5, 9), 9), ((2, 1, 1), 1), ((1, 5, 0), 5), ((1, 5, 3), 5), ((1, 5, 9), 5), ((1, 1, 0), 1)]


@pytest.mark.parametrize("shape", SHARED)
def test_rows_that_share_memory_are_refused(calls, shape):
    import torch

    rows = shape[0]
    table, mask = _window(*shape, torch.int32), _window(*shape, torch.int64)
    with pytest.raises(ValueError, match="block_table"):
        _tables(table, rows)
    for which in ("prompt", "tree"):
        with pytest.raises(ValueError, match="block_table"):
            _attend(which, rows, table=table)
    with pytest.raises(ValueError, match="tree_mask"):
        _attend("tree", rows, mask=mask)
    assert not calls


def test_one_mask_row_expanded_to_all_tokens_is_refused(calls):
    """The mask of a plain decode step, written as an expanded one."""
    import torch

    with pytest.raises(ValueError, match="tree_mask"):
        _attend("tree", 64, mask=_t((1, 1), torch.int64).expand(64, 1))
    with pytest.raises(ValueError, match="block_table"):
        _tables(_t((1, 5), torch.int32).expand(8, 5), 8)
    assert not calls


@pytest.mark.parametrize("shape,pitch", TAKEN)
def test_pitch_of_the_views_that_are_taken(calls, shape, pitch):
    import torch

    rows, width, _ = shape
    table, mask = _window(*shape, torch.int32), _window(*shape, torch.int64)
    _tables(table, rows)
    assert calls[-1][8:10] == (width, pitch)
    for which in ("prompt", "tree"):
        _attend(which, rows, table=table)
        assert calls[-1][15:18] == (rows, width, pitch)
    _attend("tree", rows, mask=mask)
    assert calls[-1][25:27] == (width, pitch)
    assert len(calls) == 4


@pytest.mark.parametrize("rows", [0, 1, 4])
def test_tables_without_rows_or_columns(calls, rows):
    import torch

    for shape, pitch in (((rows, 0, 0), 1), ((rows, 0, 7), 7 if rows > 1 else 1)):
        _tables(_window(*shape, torch.int32), rows)
        assert calls[-1][8:10] == (0, pitch)
    _attend("tree", 0, table=_t((0, 3), torch.int32), mask=_t((0, 1), torch.int64))
    assert calls[-1][15:18] == (0, 3, 3) and calls[-1][25:27] == (1, 1)

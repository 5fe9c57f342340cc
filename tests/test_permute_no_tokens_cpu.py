"""A permutation of no token, whose outputs the grouped calls read; the library launches nothing for it."""
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi


@pytest.mark.parametrize("noalloc", [False, True])
@pytest.mark.parametrize("rows", [False, True])
def test_outputs_name_no_row(monkeypatch, noalloc, rows):
    monkeypatch.setattr(ffi, "_need", lambda *a: None)
    monkeypatch.setattr(ffi, "_stream", lambda s: None)
    out = ffi.alloc_permuted(0, 128, 2, 4, 16, "cpu", rows=rows)
    for t in (out.expert_counts, out.expert_offsets, out.num_tiles, out.row_src, out.tiles):
        t.fill_(12345)  # whatever the memory held
    x, idx = torch.zeros(0, 128, dtype=torch.bfloat16), torch.zeros(0, 2, dtype=torch.int32)
    if noalloc:
        assert ffi.moe_permute_noalloc(x if rows else None, idx, None, 128, 8, 0, 4, 1, 16, out) == 0
    else:
        assert ffi.moe_permute(x, idx, None, 8, 0, 4, 1, 16, out=out, copy_rows=rows) is out
    assert int(out.num_tiles) == 0 and out.expert_counts.tolist() == [0] * 4 and out.expert_offsets.tolist() == [0] * 5
    assert out.row_src.tolist() == [-1] * (4 * 15)

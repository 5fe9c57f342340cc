"""No token: a permutation's outputs, which the grouped calls read, and the calls that gather (nothing is launched)."""
import ctypes

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


def test_gathering_from_no_token():
    fake, L = ctypes.c_void_p(16 * 1024), ffi.lib()
    call = lambda x, T, H=512: L.moe_grouped_ffn_gather(x, fake, T, 2, fake, fake, fake, fake, fake, fake, fake, 8, H, 1024, 1, 64,  # noqa: E731
                                                        8 * 63, 8, fake, fake, None, 0, None)
    assert call(None, 0) == 0
    assert call(None, 1) == 1 and call(None, -1) == 1 and call(None, 0, H=576) == 2

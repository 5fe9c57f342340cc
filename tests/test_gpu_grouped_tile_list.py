"""Tile lists with entries that name no local expert, or rows outside the capacity, through the 4-bit grouped products:
such entries have no rows, and everything else comes out as without them."""
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi

import test_gpu_mxfp4 as M

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("tile_m", [16, 32, 64, 256])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("act,N", [("none", 100), ("swiglu", 2000)])
@pytest.mark.parametrize("count", ["the list's", "beyond the capacity", "none", "negative"])
def test_entries_that_are_none(tile_m, gather, act, N, count):
    T, k, E, K = 70, 2, 8, 384
    idx = M.choice("one", T, E, k, T)                       # few tiles: the list has places left
    p = M.permuted(idx, 0, E, tile_m, K)
    g = M.gen(N + tile_m)
    x, w = M.on(M.packed(g, (T if gather else p.R_cap, K))), M.on(M.packed(g, (E, N, K)))
    up = M.on(M.packed(g, (E, N, K))) if act == "swiglu" else None

    def run():
        out, check = M.guarded((p.R_cap, N), F32, -7.0)
        ffi.moe_grouped_linear_mxfp4(p, x, w, w_up=up, act=act, gather=gather, out=out)
        check()
        return out
    want = run()
    n = int(p.num_tiles)
    top = 2 ** 31 - 1
    bad = torch.tensor([[-1, 0], [E, 0], [top, 0], [-top - 1, 0], [0, -tile_m], [1, -top - 1], [2, p.R_cap], [3, top],
                        [7, int(p.expert_offsets[-1])]], dtype=torch.int32, device=M.dev())
    fill = p.tiles_cap - n
    assert fill > 0
    p.tiles[n:] = bad.repeat(fill // len(bad) + 1, 1)[:fill]
    # (those in front take the places of real ones, which come after them)
    order = torch.arange(p.tiles_cap, device=M.dev()).flip(0)
    p.tiles.copy_(p.tiles[order].contiguous())
    p.num_tiles.fill_({"the list's": p.tiles_cap, "beyond the capacity": top, "none": 0, "negative": -3}[count])
    got = run()
    assert bool((got == -7.0).all()) if count in ("none", "negative") else torch.equal(got, want)

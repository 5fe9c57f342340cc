"""The layer without a token, as a rank that gets none calls it."""
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from mixture_experts_layer_moe_amd import workloads as W
from mixture_experts_layer_moe_amd.layer import Gating, MoELayer, SharedExpert

import parity_helpers as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(fused_gather=True), dict(few_tokens=True), dict(gating=Gating())])
@pytest.mark.parametrize("tile_m", [16, 256])
def test_layer_without_a_token(kw, mx, tile_m):
    cfg = W.CONFIGS["decode"].with_(T=4, H=256, F=128, E=8, k=2, tile_m=tile_m)
    d = W.make_inputs(cfg, P.require_gpu())
    r = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=P.require_gpu())  # noqa: E731
    w, sh = [d[n] for n in ("w0", "w0_up", "w1")], [r(128, cfg.H), r(128, cfg.H), r(cfg.H, 128)]
    if mx:
        w, sh = [ffi.moe_mxfp4_quantize(t) for t in w], [ffi.moe_mxfp4_quantize(t) for t in sh]
    layer = MoELayer(cfg.with_(T=0), d["x"][:0], d["logits"][:0], None, *w, shared=SharedExpert(*sh), **kw)
    if not layer.few_tokens:
        layer.act_buf.fill_(-7.0), layer.y_perm.fill_(-7.0)
    assert layer.run().shape == (0, cfg.H)
    torch.cuda.synchronize()
    if not layer.few_tokens:
        assert int(layer.perm.num_tiles) == 0 and bool((layer.act_buf == -7.0).all()) and bool((layer.y_perm == -7.0).all())

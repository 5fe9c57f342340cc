"""The layer with 4-bit weights: its steps called by hand, its shared expert from the first product on, no token at all,
and the whole of it captured.  Tolerances as in test_gpu_mxfp4."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from mixture_experts_layer_moe_amd import workloads as W
from mixture_experts_layer_moe_amd.layer import MoELayer, SharedExpert
from oracle import mxfp4_oracle as X
from oracle import operators_oracle as Q

import parity_helpers as P
import test_gpu_mxfp4 as M

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def shared_expert(cfg, F=256):
    r = lambda *s: ffi.moe_mxfp4_quantize((torch.randn(*s, generator=M.gen(sum(s))) * 0.05).to(BF).to(M.dev()))  # noqa: E731
    return SharedExpert(r(F, cfg.H), r(F, cfg.H) if cfg.act == "swiglu" else None, r(cfg.H, F))


def small(**over):
    return W.CONFIGS["decode"].with_(**dict(dict(T=40, H=384, F=128, E=32, k=4, tile_m=16), **over))


@pytest.mark.parametrize("kind", ["experts", "experts and shared", "shared", "few and shared"])
def test_steps_by_hand(kind):
    """The layer's own methods, one after another, give what run() gives: nothing that a step reads is left from run()."""
    cfg = small()
    d = W.make_inputs(cfg, M.dev()) if kind == "shared" else M.mx_inputs(cfg)
    kw = dict(shared=shared_expert(cfg) if "shared" in kind else None, few_tokens=kind.startswith("few"))
    want = MoELayer.from_inputs(cfg, d, **kw).run().clone()
    layer = MoELayer.from_inputs(cfg, d, **kw)
    for q in (layer.x_q, getattr(layer, "act_q", None), getattr(layer, "shared_q", None)):
        if q is not None:
            q.codes.fill_(0x11), q.scales.fill_(120)
    if layer.few_tokens:
        layer.few()
    else:
        layer.route()
        layer.permute()
        layer.ffn()
        layer.combine()
    if layer.shared is not None:
        layer.shared_expert()
    assert torch.equal(layer.out, want)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("experts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("name,over", [("decode", {}), ("tiny", dict(T=60, H=512, F=256, E=8, k=2, tile_m=16))])
def test_shared_expert_from_its_first_product(name, over, experts, few):
    cfg = W.CONFIGS[name].with_(**over) if over else small()
    d = W.make_inputs(cfg, M.dev()) if experts == "bf16" else M.mx_inputs(cfg)
    sh = shared_expert(cfg)
    layer = MoELayer.from_inputs(cfg, d, shared=sh, few_tokens=few)
    out = M.n64(layer.run())
    plain = M.n64(MoELayer.from_inputs(cfg, d, few_tokens=few).run())
    code, s = X.quantize(M.n64(d["x"]))
    xv = X.values(X.pack(code), s)
    w0, up = M.host(sh.w0), None if sh.w0_up is None else M.host(sh.w0_up)
    want, z, u = Q.linear(xv, w0, up, act_name=cfg.act)
    tol = 1.2 * M.bound(xv, w0, cfg.H)
    if up is not None:
        du = M.bound(xv, up, cfg.H)
        tol = tol * (np.abs(u) + du) + np.abs(Q.act("silu", z)) * du
    tol = tol + 1e-6 * np.abs(want) + 1e-37
    h = M.n64(layer.shared_h)
    assert (np.abs(h - want) <= tol + M.BF_HALF * (np.abs(want) + tol)).all()
    code, s = X.quantize(h)
    assert np.array_equal(layer.shared_q.codes.cpu().numpy(), X.pack(code)) and np.array_equal(layer.shared_q.scales.cpu().numpy(), s)
    hq, w1 = X.values(X.pack(code), s), M.host(sh.w1)
    part = hq @ w1.T
    assert (np.abs(out - (plain + part)) <= M.bound(hq, w1, h.shape[1]) + M.U2 * (np.abs(plain) + np.abs(out))).all()


@pytest.mark.parametrize("kw", [dict(), dict(few_tokens=True)])
def test_the_whole_layer_captured(kw):
    """Replayed with other tokens, the program's own work between the replays."""
    cfg = small()
    d = M.mx_inputs(cfg)
    sh = shared_expert(cfg)
    layer, eager = (MoELayer.from_inputs(cfg, d, shared=sh, **kw) for _ in range(2))
    layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for i in range(4):
        d["x"].copy_(torch.randn(cfg.T, cfg.H, generator=M.gen(i)).to(BF))
        d["logits"].copy_(torch.randn(cfg.T, cfg.E, generator=M.gen(10 + i)))
        layer.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = layer.out.clone()
        assert torch.equal(got, eager.run()) and bool(torch.isfinite(got).all())
        torch.cuda.synchronize()

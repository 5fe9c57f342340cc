"""Which calls the layer's steps make with 4-bit weights, and in which order; no GPU and no library call."""
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from mixture_experts_layer_moe_amd import workloads as W
from mixture_experts_layer_moe_amd.layer import MoELayer, SharedExpert

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The names of the operators called, with those of the tensors that quantising reads and the products multiply."""
    log = []

    def record(name):
        def call(*args, out=None, **kw):
            log.append((name, args, out))
        return call
    for n in ("moe_route_topk", "moe_permute", "moe_mxfp4_quantize", "moe_grouped_linear_mxfp4", "moe_grouped_ffn", "moe_combine",
              "moe_linear_mxfp4", "moe_linear", "moe_few_tokens"):
        monkeypatch.setattr(ffi, n, record(n))
    for n in ("alloc_linear_workspace", "alloc_linear_mxfp4_workspace"):
        monkeypatch.setattr(ffi, n, lambda *a: None)
    return log


def layer_of(experts, shared, few):
    cfg = W.CONFIGS["decode"].with_(T=4, H=256, F=128, E=8, k=2)
    d = W.make_inputs(cfg)
    if experts == "mxfp4":
        d = dict(d, **{n: ffi.alloc_mxfp4(d[n].shape, "cpu") for n in ("w0", "w0_up", "w1")})
    sh = None
    if shared == "mxfp4":
        a = lambda *s: ffi.alloc_mxfp4(s, "cpu")  # noqa: E731
        sh = SharedExpert(a(128, 256), a(128, 256), a(256, 128))
    elif shared:
        z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
        sh = SharedExpert(z(128, 256), z(128, 256), z(256, 128))
    return MoELayer.from_inputs(cfg, d, shared=sh, few_tokens=few)


def by_hand(layer):
    if layer.few_tokens:
        layer.few()
    else:
        layer.route()
        layer.permute()
        layer.ffn()
        layer.combine()
    if layer.shared is not None:
        layer.shared_expert()


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("shared", [None, "bf16", "mxfp4"])
@pytest.mark.parametrize("experts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("way", [MoELayer.run, by_hand])
def test_tokens_are_quantised_once_and_before_they_are_read(calls, way, experts, shared, few):
    layer = layer_of(experts, shared, few)
    way(layer)
    quantised = [i for i, (n, args, out) in enumerate(calls) if n == "moe_mxfp4_quantize" and args[0] is layer.x and out is layer.x_q]
    reads = [i for i, (n, args, _) in enumerate(calls)
             if n in ("moe_grouped_linear_mxfp4", "moe_linear_mxfp4") and layer.x_q is not None and any(a is layer.x_q for a in args)]
    needed = (experts == "mxfp4" and not few) or shared == "mxfp4"
    assert len(reads) == (experts == "mxfp4" and not few) + (shared == "mxfp4")
    assert len(quantised) == (1 if needed else 0)
    if needed:
        assert quantised[0] < min(reads)

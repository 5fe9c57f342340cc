"""The layer for a few tokens on the GPU against the float64 oracle.

Tolerances: indices are compared exactly; gate weights are a quotient of an fp32 exponential and a sum of at most E of
them: within 4e-6 of their value for |logits| <= 16.  Outputs are within the oracle's bound, which counts the steps of
each product, of the activation and of the gate weight (computed with the library's own topk_w).  Those bounds grow with
the reduction's length times the terms' size; where rounding errors are independent they add as the root of it, so the
relative norm of the error is also held to 2e-5 (sqrt(7168) steps of 2^-24, four times over).
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from mixture_experts_layer_moe_amd import workloads as W
from mixture_experts_layer_moe_amd.layer import Gating, MoELayer, SharedExpert
from oracle import moe_oracle as O
from oracle import mxfp4_oracle as X
from oracle import operators_oracle as Q

import parity_helpers as P

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
INF, NAN = float("inf"), float("nan")


def dev():
    return P.require_gpu()


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def n64(t):
    return t.detach().cpu().double().numpy()


def guarded(shape, dtype, fill, pad=64):
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device=dev())

    def check():
        torch.cuda.synchronize()
        assert bool((whole[:pad] == fill).all()) and bool((whole[pad + n:] == fill).all()), "written out of range"
    return whole[pad:pad + n].view(shape), check


class Experts:
    """Weights on the device in bf16 or MXFP4, and in float64 expert by expert."""

    def __init__(self, g, El, H, F, act, mx, std=0.05):
        r = lambda *s: (torch.randn(*s, generator=g) * std).to(BF).to(dev())  # noqa: E731
        self.act, self.mx = act, mx
        self.t = [r(El, F, H), r(El, F, H) if act == "swiglu" else None, r(El, H, F)]
        if mx:
            self.t = [None if t is None else ffi.moe_mxfp4_quantize(t) for t in self.t]

    def __call__(self, e):
        f = lambda t: None if t is None else (X.values(t.codes[e].cpu().numpy(), t.scales[e].cpu().numpy()) if self.mx else n64(t[e]))  # noqa: E731
        return tuple(f(t) for t in self.t)


def run(x, w, logits=None, k=None, idx=None, gate=None, **kw):
    """Output, choice and gate weights of one call on guarded outputs, its workspace filled with NaN."""
    T, H = x.shape
    k = k or idx.shape[1]
    d = dev()
    out, c1 = guarded((T, H), F32, -7.0)
    ti, c2 = guarded((T, k), torch.int32, -7)
    tw, c3 = guarded((T, k), F32, -7.0)
    if logits is None:
        ti.copy_(idx), tw.copy_(gate)
    F = w.t[0].shape[1]
    ws, c4 = guarded((ffi.few_tokens_workspace_bytes(T, k, F),), U8, 0xFF)
    ffi.moe_few_tokens(x.to(d), *w.t, w.act, logits=None if logits is None else logits.to(d), topk_idx=ti, topk_w=tw, out=out,
                       ws=ws, **kw)
    c1(), c2(), c3(), c4()
    return n64(out), ti.cpu().numpy(), n64(tw)


def check_out(out, x, idx, gate, w, El, e0=0, norm=True):
    ref, bound = X.few_tokens(n64(x), idx, gate, w, w.act, e0, El)
    assert (np.abs(out - ref) <= bound).all()
    if norm and np.linalg.norm(ref) > 0:
        assert np.linalg.norm(out - ref) <= 2e-5 * np.linalg.norm(ref)
    return ref


SHAPES = [(1, 128, 128, 1, 1), (1, 256, 384, 8, 2), (1, 2048, 1408, 16, 6), (2, 128, 640, 8, 8), (3, 384, 128, 4, 1), (4, 512, 256, 60, 4),
          (5, 128, 128, 8, 2), (7, 512, 1024, 8, 2), (13, 256, 256, 64, 8), (16, 128, 256, 2, 2), (17, 256, 128, 4, 3),
          (31, 128, 128, 40, 32), (33, 640, 384, 16, 4), (64, 256, 256, 8, 2), (64, 128, 128, 256, 8), (64, 128, 128, 1, 1),
          (64, 128, 128, 1024, 5), (1, 7168, 256, 8, 2), (21, 1408, 2048, 6, 1)]


@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_shapes(T, H, F, E, k, mx, act):
    g = gen(T + H + E)
    w = Experts(g, E, H, F, act, mx)
    x = torch.randn(T, H, generator=g).to(BF)
    l = torch.randn(T, E, generator=g)
    renorm = (T + k) % 3 != 0
    out, idx, gate = run(x, w, l, k, renormalize=renorm)
    ridx, rw = X.route(l.numpy(), k, renorm)
    assert np.array_equal(idx, ridx)
    np.testing.assert_allclose(gate, rw, rtol=4e-6, atol=1e-37)
    check_out(out, x, idx, gate, w, E)


@pytest.mark.parametrize("T,E,k,given", [(64, 1024, 32, False), (64, 1024, 32, True), (1, 1024, 32, False), (64, 32, 32, True)])
def test_the_most_tokens_experts_and_choices(T, E, k, given):
    """The routing lists at their longest."""
    g = gen(T + E)
    w = Experts(g, E, 128, 128, "gelu", True)
    x = torch.randn(T, 128, generator=g).to(BF)
    l = torch.randn(T, E, generator=g)
    if given:
        idx, gate = X.route(l.numpy(), k, True)
        out, idx, gate = run(x, w, idx=torch.from_numpy(idx.astype(np.int32)), gate=torch.from_numpy(gate).float(), num_experts=E)
    else:
        out, idx, gate = run(x, w, l, k)
        assert np.array_equal(idx, X.route(l.numpy(), k, True)[0])
    check_out(out, x, idx, gate, w, E)


@pytest.mark.parametrize("T,H,F,E,k", [(5, 4096, 256, 16, 3), (40, 4096, 128, 4, 2), (9, 7168, 384, 16, 4), (64, 8192, 128, 64, 8),
                                       (30, 7168, 256, 8, 3), (2, 6144, 1408, 4, 2)])
@pytest.mark.parametrize("mx", [False, True])
def test_long_rows(T, H, F, E, k, mx):
    """Lengths of out that take more columns a workgroup."""
    g = gen(T + H)
    w = Experts(g, E, H, F, "swiglu", mx)
    x = torch.randn(T, H, generator=g).to(BF)
    out, idx, gate = run(x, w, torch.randn(T, E, generator=g), k)
    check_out(out, x, idx, gate, w, E)


def test_long_rows_beside_the_longest_lists():
    """A share of many experts: the lists leave less room for the sums."""
    T, H, E, El, k = 64, 8192, 704, 4, 32
    g = gen(0)
    w = Experts(g, El, H, 128, "gelu", True)
    x = torch.randn(T, H, generator=g).to(BF)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    idx[:, 5] = torch.arange(T) % 5 + 100
    gate = torch.rand(T, k, generator=g)
    out, i2, g2 = run(x, w, idx=idx, gate=gate, expert_begin=100, num_experts=E)
    check_out(out, x, i2, g2, w, El, 100)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 6, 40, 64])
@pytest.mark.parametrize("e0,El", [(0, 4), (4, 8), (15, 1)])
def test_a_share_of_given_choices(T, e0, El, mx):
    """Choices made elsewhere: padding tokens, slots of other ranks and beyond, gate weights of any sign and size."""
    g = gen(T + e0)
    w = Experts(g, El, 256, 384, "swiglu", mx)
    x = torch.randn(T, 256, generator=g).to(BF)
    idx = torch.stack([torch.randperm(16, generator=g)[:5] for _ in range(T)]).to(torch.int32)
    gate = torch.randn(T, 5, generator=g) * 2
    idx[T // 2, :] = -1
    if T > 1:
        idx[0, 0], gate[0, 1] = 1 << 30, 0.0
        idx[1, 2] = -5
    out, i2, g2 = run(x, w, idx=idx, gate=gate, expert_begin=e0, num_experts=16)
    assert np.array_equal(i2, idx.numpy()) and np.array_equal(g2, gate.double().numpy())
    check_out(out, x, i2, g2, w, El, e0)
    none = ~((i2 >= e0) & (i2 < e0 + El)).any(axis=1)
    assert none.any() and (out[none] == 0).all()


@pytest.mark.parametrize("mx", [False, True])
def test_no_token_has_a_local_expert(mx):
    w = Experts(gen(0), 2, 128, 128, "gelu", mx)
    for T in (1, 9):
        out, _, _ = run(torch.randn(T, 128, generator=gen(1)).to(BF), w, idx=torch.full((T, 3), -1, dtype=torch.int32), gate=torch.ones(T, 3))
        assert (out == 0).all()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 12, 64])
def test_an_expert_named_more_than_once(T, mx):
    g = gen(T)
    w = Experts(g, 3, 128, 256, "swiglu", mx)
    x = torch.randn(T, 128, generator=g).to(BF)
    idx = torch.randint(0, 3, (T, 7), generator=g, dtype=torch.int32)
    gate = torch.randn(T, 7, generator=g)
    out, i2, g2 = run(x, w, idx=idx, gate=gate)
    check_out(out, x, i2, g2, w, 3, norm=False)  # (weights of one expert may cancel)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,heavy", [(64, 64), (64, 33), (20, 17), (64, 5), (9, 9)])
def test_an_expert_with_many_tokens_among_others_with_few(T, heavy, mx):
    """More tokens on one expert than a pass takes, whichever form the averages choose."""
    g = gen(T + heavy)
    for E in (8, 96):
        w = Experts(g, E, 128, 128, "swiglu", mx)
        x = torch.randn(T, 128, generator=g).to(BF)
        l = torch.randn(T, E, generator=g)
        l[torch.randperm(T, generator=g)[:heavy], E // 2] = 9.0
        out, idx, gate = run(x, w, l, 2)
        check_out(out, x, idx, gate, w, E)


@pytest.mark.parametrize("renorm", [True, False])
def test_masks_ties_and_extremes_in_the_logits(renorm):
    E, k, T = 24, 4, 12
    g = gen(4)
    w = Experts(g, E, 128, 128, "swiglu", False)
    x = torch.randn(T, 128, generator=g).to(BF)
    l = torch.randn(T, E, generator=g)
    l[0] = -INF                       # padding token
    l[1] = NAN
    l[2, 2:] = -INF                   # fewer experts than slots
    l[3, ::2] = NAN
    l[4] = torch.finfo(F32).min       # masks of the type's lowest value: available, equal
    l[5, 3:] = torch.finfo(F32).min
    l[6, 20] = l[6, 7] = INF          # counts as the largest finite value
    l[7] = 0.25                       # all equal: lowest ids
    l[8] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0)
    l[9] = l[9].round()
    l[10] = -1000.0 + l[10]
    out, idx, gate = run(x, w, l, k, renormalize=renorm)
    ridx, rw = X.route(l.numpy(), k, renorm)
    assert np.array_equal(idx, ridx)
    np.testing.assert_allclose(gate, rw, rtol=4e-6, atol=1e-37)
    check_out(out, x, idx, gate, w, E)
    assert (out[:2] == 0).all()


def test_routes_as_the_plain_routing():
    g = gen(8)
    for T, E, k in ((64, 256, 8), (9, 64, 6), (33, 1000, 32)):
        l = torch.randn(T, E, generator=g)
        w = Experts(g, E, 128, 128, "gelu", True)
        _, idx, gate = run(torch.zeros(T, 128, dtype=BF), w, l, k)
        a, b = ffi.moe_route_topk(l.to(dev()), k)
        assert np.array_equal(idx, a.cpu().numpy())
        np.testing.assert_allclose(gate, n64(b), rtol=2e-6)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [3, 40])
def test_infinities_and_nan_reach_their_own_tokens_alone(T, mx):
    """An expert whose weights hold NaN, another with infinities, a token that holds one: all others stay finite."""
    g = gen(T)
    E, k = 8, 1
    w = Experts(g, E, 128, 128, "swiglu", mx)
    clean = [w(e) for e in range(E)]
    if mx:
        w.t[2].scales[1, ::2] = 255
        w.t[0].scales[2, 5] = 255
    else:
        w.t[2][1, 3], w.t[2][1, 4, 0] = NAN, INF
        w.t[0][2, 7, 3] = NAN
        w.t[1][2, 9] = -INF
    x = torch.randn(T, 128, generator=g).to(BF)
    x[T - 1, 5] = INF
    l = torch.full((T, E), -5.0)
    l[torch.arange(T), torch.arange(T) % E] = 5.0
    out, idx, gate = run(x, w, l, k)
    sick = (idx[:, 0] == 1) | (idx[:, 0] == 2)
    sick[T - 1] = True
    assert not np.isfinite(out[sick]).all(axis=1).any()
    ref, bound = X.few_tokens(n64(x)[~sick], idx[~sick], gate[~sick], lambda e: clean[e], "swiglu", 0, E)
    assert (np.abs(out[~sick] - ref) <= bound).all()


def test_an_infinite_activation_is_an_infinity_in_the_output():
    """Not the NaN that taking it apart into terms would make."""
    d = dev()
    w0, w1 = torch.zeros(1, 128, 128, dtype=BF, device=d), torch.zeros(1, 128, 128, dtype=BF, device=d)
    w0[0, 0, :] = 3e38                                   # z overflows to +inf in one column, the others are zero
    w1[0, :, 0] = torch.tensor([1.0, -2.0]).repeat(64).to(BF).to(d)
    for T in (1, 30):
        x = torch.ones(T, 128, dtype=BF, device=d)
        out = ffi.moe_few_tokens(x, w0, None, w1, "gelu", topk_idx=torch.zeros(T, 1, dtype=torch.int32, device=d),
                                 topk_w=torch.ones(T, 1, device=d))
        assert bool((out[:, ::2] == INF).all()) and bool((out[:, 1::2] == -INF).all())


@pytest.mark.parametrize("mx", [False, True])
def test_weights_past_4_gib(mx):
    """Experts whose weights begin past 2^32 bytes (2^28 bytes of scales)."""
    d = dev()
    El, H, F = (48, 8192, 8192) if not mx else (160, 8192, 8192)
    if mx:
        w = [ffi.Mxfp4(torch.zeros(El, F, H // 2, dtype=U8, device=d), torch.zeros(El, F, H // 32, dtype=U8, device=d)),
             ffi.Mxfp4(torch.zeros(El, H, F // 2, dtype=U8, device=d), torch.zeros(El, H, F // 32, dtype=U8, device=d))]
        for e in (0, El - 1):
            for m, v in zip(w, (0x11, 0x22)):
                m.codes[e], m.scales[e] = v, 120 + (e > 0)
        a, b = [0.5 * 2.0 ** -7, 0.5 * 2.0 ** -6], [2.0 ** -7, 2.0 ** -6]
    else:
        w = [torch.zeros(El, F, H, dtype=BF, device=d), torch.zeros(El, H, F, dtype=BF, device=d)]
        a, b = [2.0 ** -8, 2.0 ** -7], [2.0 ** -7, 2.0 ** -6]
        for j, e in enumerate((0, El - 1)):
            w[0][e], w[1][e] = a[j], b[j]
    x = torch.ones(2, H, dtype=BF, device=d)
    idx = torch.tensor([[0], [El - 1]], dtype=torch.int32, device=d)
    out = n64(ffi.moe_few_tokens(x, w[0], None, w[1], "gelu", topk_idx=idx, topk_w=torch.ones(2, 1, device=d)))
    for j in range(2):
        want = Q.act("gelu", np.array(H * a[j])) * F * b[j]
        np.testing.assert_allclose(out[j], want, rtol=1e-5)


@pytest.mark.parametrize("T,E,k", [(1, 16, 2), (40, 8, 2)])
def test_graphs_streams_and_repeats(T, E, k):
    """A captured call replayed with new inputs, two calls at once, and the same bits every time."""
    g = gen(T)
    d = dev()
    w = Experts(g, E, 256, 256, "swiglu", True)
    x = torch.randn(T, 256, generator=g).to(BF).to(d)
    l = torch.randn(T, E, generator=g).to(d)
    make = lambda: dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=d), topk_w=torch.empty(T, k, device=d),  # noqa: E731
                        out=torch.empty(T, 256, device=d), ws=ffi.alloc_few_tokens_workspace(T, k, 256, d))
    b = [make(), make()]
    call = lambda q, **kw: ffi.moe_few_tokens(x, *w.t, "swiglu", logits=l, **q, **kw)  # noqa: E731
    want = call(b[0]).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    for _ in range(20):
        for s, q in zip(streams, b):
            call(q, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(b[0]["out"], want) and torch.equal(b[1]["out"], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(b[0])
    for i in range(4):
        x.copy_(torch.randn(T, 256, device=d))
        l.copy_(torch.randn(T, E, device=d))
        b[0]["out"].fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        got = b[0]["out"].clone()
        eager = call(b[1])
        torch.cuda.synchronize()
        assert torch.equal(got, eager) and torch.equal(b[0]["topk_idx"], b[1]["topk_idx"])


def test_defaults_and_refusals_of_the_binding():
    d = dev()
    w = Experts(gen(0), 4, 128, 128, "swiglu", False)
    x, l = torch.randn(3, 128, device=d).to(BF), torch.randn(3, 4, device=d)
    out = ffi.moe_few_tokens(x, *w.t, "swiglu", logits=l, k=2)
    idx, gate = ffi.moe_route_topk(l, 2)
    torch.testing.assert_close(out, ffi.moe_few_tokens(x, *w.t, "swiglu", topk_idx=idx, topk_w=gate), rtol=1e-4, atol=1e-6)
    assert ffi.moe_few_tokens(x[:0], *w.t, "swiglu", logits=l[:0], k=2).shape == (0, 128)
    for bad in (dict(logits=l), dict(topk_idx=idx), dict(logits=l, k=2, ws=torch.empty(16, dtype=U8, device=d)),
                dict(logits=l.double(), k=2), dict(logits=l, topk_idx=idx[:2]), dict(logits=l.cpu(), k=2)):
        with pytest.raises((ValueError, TypeError, ffi.MoEError)):
            ffi.moe_few_tokens(x, *w.t, "swiglu", **bad)
    with pytest.raises(TypeError):
        ffi.moe_few_tokens(x, w.t[0], w.t[1], ffi.moe_mxfp4_quantize(w.t[2]), "swiglu", logits=l, k=2)
    with pytest.raises(ValueError):
        ffi.moe_few_tokens(x, w.t[0], w.t[1], w.t[2][:, :64], "swiglu", logits=l, k=2)
    with pytest.raises(ValueError):
        ffi.moe_few_tokens(x.t().contiguous().t(), *w.t, "swiglu", logits=l, k=2)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gating", [None, Gating(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)])
@pytest.mark.parametrize("T", [1, 24])
def test_the_layer_for_a_few_tokens(T, gating, mx):
    """MoELayer(few_tokens=True) beside the four-call path, both against the oracle, a shared expert in MXFP4 on top."""
    cfg = W.CONFIGS["decode"].with_(T=T, H=384, F=256, E=32, k=4)
    d = W.make_inputs(cfg, dev())
    host = P.host_weights64(d)
    e = d
    if mx:
        e = dict(d, **{n: ffi.moe_mxfp4_quantize(d[n]) for n in ("w0", "w0_up", "w1")})
        host = lambda i: tuple(X.values(e[n].codes[i].cpu().numpy(), e[n].scales[i].cpu().numpy()) for n in ("w0", "w0_up", "w1"))  # noqa: E731
    layer = MoELayer.from_inputs(cfg, e, few_tokens=True, gating=gating)
    out = n64(layer.run())
    idx, gate = layer.topk_idx.cpu().numpy(), n64(layer.topk_w)
    ref, bound = X.few_tokens(n64(d["x"]), idx, gate, host, "swiglu", 0, cfg.E)
    assert (np.abs(out - ref) <= bound).all()
    if not mx:
        four = MoELayer.from_inputs(cfg, d, gating=gating)
        P.assert_output_close(n64(four.run()), ref)
        assert np.array_equal(four.topk_idx.cpu().numpy(), idx)
    r = lambda *s: ffi.moe_mxfp4_quantize(torch.randn(*s, device=dev()).mul_(0.05).to(BF))  # noqa: E731
    sh = SharedExpert(r(128, cfg.H), r(128, cfg.H), r(cfg.H, 128))
    both = MoELayer.from_inputs(cfg, e, few_tokens=True, gating=gating, shared=sh)
    total = n64(both.run())
    h = X.values(*(t.cpu().numpy() for t in both.shared_q))
    w1 = X.values(*(t.cpu().numpy() for t in sh.w1))
    part, mag = h @ w1.T, np.abs(h) @ np.abs(w1).T
    assert (np.abs(total - (out + part)) <= 2.0 ** -23 * (128 * mag + np.abs(out) + np.abs(total))).all()
    idx2, _ = O.route_topk(d["logits"].cpu().numpy(), 4)
    if gating is None:
        assert np.array_equal(idx, idx2)

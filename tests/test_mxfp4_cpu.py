"""4-bit operands and the layer for a few tokens without a GPU: refusals of the C ABI and the binding, the oracle's pins.

No library call here reaches a kernel launch: each returns from host
validation.
"""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from mixture_experts_layer_moe_amd import workloads as W
from mixture_experts_layer_moe_amd.layer import MoELayer, SharedExpert
from oracle import moe_oracle as O
from oracle import mxfp4_oracle as X
from oracle import operators_oracle as Q

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
NULL = None


def at(n):
    """Aligned addresses far from one another (sizes here stay below 2^40); never dereferenced: validation fails first."""
    return ctypes.c_void_p((n + 1) << 44)


ODD = ctypes.c_void_p((1 << 44) + 4)


@pytest.fixture(scope="module")
def L():
    return ffi.lib()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

def quantize(L, **over):
    a = dict(x=at(0), R=10, K=64, dt=0, q=at(1), s=at(2))
    a.update(over)
    return L.moe_mxfp4_quantize(*a.values(), NULL)


def dequantize(L, **over):
    a = dict(q=at(1), s=at(2), R=10, K=64, dt=0, x=at(0))
    a.update(over)
    return L.moe_mxfp4_dequantize(*a.values(), NULL)


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("over,code", [
    (dict(R=0, x=NULL, q=NULL, s=NULL), OK), (dict(R=-1), INVALID), (dict(K=0), INVALID), (dict(K=-32), INVALID),
    (dict(dt=2), INVALID), (dict(dt=-1), INVALID), (dict(K=48), UNSUPPORTED), (dict(R=(1 << 31) + 1, K=32), UNSUPPORTED),
    (dict(R=(1 << 62), K=32), UNSUPPORTED), (dict(x=NULL), INVALID), (dict(q=NULL), INVALID), (dict(s=NULL), INVALID),
    (dict(x=ODD), INVALID), (dict(q=ODD), INVALID), (dict(s=ODD), INVALID), (dict(q=at(0)), INVALID), (dict(s=at(0)), INVALID),
    (dict(x=ctypes.c_void_p((2 << 44) + 304)), INVALID)])  # codes: 320 bytes, x begins 16 before their end
def test_quantize_refusals(L, call, over, code):
    assert call(L, **over) == code


def test_quantize_outputs_that_overlap(L):
    assert quantize(L, s=at(1)) == INVALID


def linear(L, **over):
    a = dict(xq=at(0), xs=at(1), wq=at(2), ws=at(3), uq=at(4), us=at(5), b=at(6), bu=at(7), r=at(8), M=10, N=20, K=128, act=1,
             dt=0, out=at(9), w=NULL, wb=0)
    a.update(over)
    return L.moe_linear_mxfp4(*a.values(), NULL)


NONE = dict(act=2, uq=NULL, us=NULL, bu=NULL)


@pytest.mark.parametrize("over,code", [
    (dict(M=0, xq=NULL, out=NULL), OK), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(dt=2), INVALID), (dict(K=64), UNSUPPORTED), (dict(K=192), UNSUPPORTED),
    (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 128), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(xq=NULL), INVALID), (dict(xs=NULL), INVALID), (dict(wq=NULL), INVALID), (dict(ws=NULL), INVALID),
    (dict(uq=NULL), INVALID), (dict(us=NULL), INVALID), (dict(out=NULL), INVALID), (dict(act=2), INVALID),
    (dict(act=0, uq=NULL), INVALID), (dict(NONE, bu=at(7)), INVALID), (dict(xq=ODD), INVALID), (dict(xs=ODD), INVALID),
    (dict(us=ODD), INVALID), (dict(b=ODD), INVALID), (dict(out=ODD), INVALID), (dict(out=at(0)), INVALID),
    (dict(out=at(3)), INVALID), (dict(out=at(6)), INVALID), (dict(w=at(0), wb=16), INVALID), (dict(w=at(9), wb=16), INVALID),
    (dict(NONE, r=NULL, M=(1 << 31) - 1, N=1 << 20), UNSUPPORTED)])
def test_linear_mxfp4_refusals(L, over, code):
    assert linear(L, **over) == code


def test_linear_mxfp4_workspace(L):
    for M, N, K, act in [(-1, 8, 128, 2), (8, 0, 128, 2), (8, 8, 64, 2), (8, 8, 128, 9), (1 << 31, 8, 128, 2)]:
        assert L.moe_linear_mxfp4_workspace_bytes(M, N, K, act) == 0
    for M, N, K in [(1, 2048, 7168), (300, 500, 14336), (1000, 1001, 1408)]:
        need = L.moe_linear_mxfp4_workspace_bytes(M, N, K, 2)
        if need:
            assert linear(L, **NONE, M=M, N=N, K=K, w=at(11), wb=need - 1) == WORKSPACE


def grouped(L, **over):
    a = dict(xq=at(0), xs=at(1), src=at(2), T=100, k=2, cnt=at(3), off=at(4), tiles=at(5), nt=at(6), wq=at(7), ws=at(8), uq=at(9),
             us=at(10), El=8, N=20, K=128, act=1, tm=64, R=1000, tc=20, dt=0, out=at(11))
    a.update(over)
    return L.moe_grouped_linear_mxfp4(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(R=0), OK), (dict(tc=0), OK), (dict(T=0), OK), (dict(R=-1), INVALID), (dict(tc=-1), INVALID), (dict(El=0), INVALID),
    (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(act=5), INVALID), (dict(dt=3), INVALID), (dict(T=-1), INVALID),
    (dict(k=0), INVALID), (dict(src=NULL, T=-1, k=0, act=2), INVALID), (dict(K=64), UNSUPPORTED), (dict(tm=48), UNSUPPORTED),
    (dict(tm=512), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(T=1 << 26), UNSUPPORTED), (dict(R=1 << 31), UNSUPPORTED),
    (dict(tc=1 << 28), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(xq=NULL), INVALID), (dict(xs=NULL), INVALID),
    (dict(cnt=NULL), INVALID), (dict(off=NULL), INVALID), (dict(tiles=NULL), INVALID), (dict(nt=NULL), INVALID),
    (dict(wq=NULL), INVALID), (dict(ws=NULL), INVALID), (dict(uq=NULL), INVALID), (dict(us=NULL), INVALID),
    (dict(out=NULL), INVALID), (dict(act=0), INVALID), (dict(src=ODD), INVALID), (dict(us=ODD), INVALID), (dict(wq=ODD), INVALID),
    (dict(out=at(2)), INVALID), (dict(out=at(7)), INVALID), (dict(out=at(5)), INVALID)])
def test_grouped_mxfp4_refusals(L, over, code):
    assert grouped(L, **over) == code


def few(L, **over):
    a = dict(x=at(0), l=at(1), T=10, E=64, k=4, rn=1, e0=0, El=64, w0=at(2), s0=NULL, up=at(3), su=NULL, w1=at(4), s1=NULL, H=256,
             F=128, act=1, idx=at(5), w=at(6), out=at(7), ws=at(8), wb=1 << 30)
    a.update(over)
    return L.moe_few_tokens(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(T=0, x=NULL, ws=NULL), OK), (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(El=0), INVALID), (dict(e0=-1), INVALID), (dict(e0=1), INVALID), (dict(H=0), INVALID), (dict(F=0), INVALID),
    (dict(act=2), INVALID), (dict(act=0), INVALID), (dict(up=NULL), INVALID), (dict(s0=at(9)), INVALID),
    (dict(s0=at(9), s1=at(10)), INVALID), (dict(s1=at(10)), INVALID), (dict(su=at(10)), INVALID),
    (dict(act=0, up=NULL, su=at(9)), INVALID), (dict(T=65), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(E=64, k=33), UNSUPPORTED), (dict(H=192), UNSUPPORTED), (dict(F=64), UNSUPPORTED),
    (dict(H=(1 << 20) + 128), UNSUPPORTED), (dict(x=NULL), INVALID), (dict(w0=NULL), INVALID), (dict(w1=NULL), INVALID),
    (dict(idx=NULL), INVALID), (dict(w=NULL), INVALID), (dict(out=NULL), INVALID), (dict(ws=NULL), INVALID),
    (dict(l=ODD), INVALID), (dict(x=ODD), INVALID), (dict(up=ODD), INVALID), (dict(s0=ODD, su=at(9), s1=at(10)), INVALID),
    (dict(out=at(0)), INVALID), (dict(out=at(4)), INVALID), (dict(ws=at(7)), INVALID), (dict(idx=at(1)), INVALID),
    (dict(l=NULL, w=at(5)), INVALID), (dict(l=NULL, out=at(5)), INVALID)])
def test_few_tokens_refusals(L, over, code):
    assert few(L, **over) == code


def test_few_tokens_workspace(L):
    need = L.moe_few_tokens_workspace_bytes(10, 4, 128)
    assert need >= 10 * 4 * 128 * 4
    assert few(L, wb=need - 1) == WORKSPACE
    for T, k, F in [(0, 4, 128), (65, 4, 128), (10, 0, 128), (10, 33, 128), (10, 4, 0)]:
        assert L.moe_few_tokens_workspace_bytes(T, k, F) == 0
    assert ffi.FEW_TOKENS == 64 and L.moe_few_tokens_workspace_bytes(ffi.FEW_TOKENS, 4, 128) > 0


def test_binding_refuses_host_tensors_and_other_types():
    q = ffi.alloc_mxfp4((4, 128), "cpu")
    with pytest.raises(ValueError):
        ffi.moe_mxfp4_quantize(torch.zeros(4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ffi.moe_mxfp4_dequantize(q)
    with pytest.raises(ValueError):
        ffi.moe_linear_mxfp4(q, q)
    with pytest.raises(TypeError):
        ffi.moe_linear_mxfp4(torch.zeros(4, 128), q)
    with pytest.raises(ValueError):
        ffi.moe_few_tokens(torch.zeros(4, 128, dtype=torch.bfloat16), None, None, None, "gelu")
    assert q.shape == (4, 128)


def test_layer_refusals():
    cfg = W.CONFIGS["decode"].with_(T=4, H=256, F=128, E=8, k=2)
    d = W.make_inputs(cfg)
    mx = {n: ffi.alloc_mxfp4(d[n].shape, "cpu") for n in ("w0", "w0_up", "w1")}
    args = (cfg, d["x"], d["logits"], None)
    with pytest.raises(ValueError):
        MoELayer(*args, mx["w0"], mx["w0_up"], d["w1"])          # some of the experts' weights
    with pytest.raises(ValueError):
        MoELayer(*args, mx["w0"], mx["w0_up"], mx["w1"], signalled=True)
    with pytest.raises(ValueError):
        MoELayer(*args, d["w0"], d["w0_up"], d["w1"], signalled=True, few_tokens=True)
    with pytest.raises(ValueError):
        MoELayer(*args, d["w0"], d["w0_up"], d["w1"], fused_gather=True, few_tokens=True)
    with pytest.raises(ValueError):
        MoELayer(cfg.with_(T=65), *args[1:], d["w0"], d["w0_up"], d["w1"], few_tokens=True)
    sh = SharedExpert(ffi.alloc_mxfp4((128, 256), "cpu"), ffi.alloc_mxfp4((128, 256), "cpu"), torch.zeros(256, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        MoELayer(*args, d["w0"], d["w0_up"], d["w1"], shared=sh)


# ---------------------------------------------------------------------------
# Pins of the oracle
# ---------------------------------------------------------------------------

def test_oracle_rounding_of_one_block():
    # 4 sets the scale to 1: halfway points go to the even code, 7 and up saturate
    x = np.array([4, .25, .250001, .75, .749999, 1.25, 1.250001, 1.75, 1.749999, 2.5, 2.500001, 3.5, 3.499999, 5, 5.000001, 7, 7.99,
                  -.25, -.75, -0.0, 0.0, -5, -6, 6, 0.1, 1, 2, 3, .5, 1.5, -1.5, -4])
    v = [4, 0, .5, 1, .5, 1, 1.5, 2, 1.5, 2, 3, 4, 3, 4, 6, 6, 6, -0.0, -1, -0.0, 0, -4, -6, 6, 0, 1, 2, 3, .5, 1.5, -1.5, -4]
    c, s = X.quantize(x[None])
    assert s[0, 0] == 127
    got = X.values(X.pack(c), s)[0]
    assert np.array_equal(got, v) and np.array_equal(np.signbit(got), np.signbit(np.array(v)))


def test_oracle_scales():
    for top, byte in [(1.0, 125), (1.999, 125), (2.0, 126), (4.0, 127), (7.99, 127), (2.0 ** -126, 0), (2.0 ** -125, 0),
                      (2.0 ** -124, 1), (2.0 ** -149, 0), (0.0, 0), (float(np.finfo(np.float32).max), 252), (np.inf, 255),
                      (np.nan, 255)]:
        x = np.zeros((1, 32))
        x[0, 7] = top
        c, s = X.quantize(x)
        assert s[0, 0] == byte
        assert (c == 0).all() or np.isfinite(top)


def test_oracle_codes_are_the_nearest_and_idempotent():
    r = np.random.default_rng(0)
    x = r.standard_normal((50, 96)) * np.exp2(r.integers(-20, 20, (50, 1)))
    c, s = X.quantize(x)
    v = X.values(X.pack(c), s)
    scale = np.exp2(s.astype(float) - 127).repeat(32, axis=1)
    every = np.concatenate((X.GRID, -X.GRID))[None, None] * scale[..., None]
    assert (np.abs(v - x) <= np.abs(every - x[..., None]).min(axis=2) + 1e-300).all()
    c2, s2 = X.quantize(v)
    assert np.array_equal(X.values(X.pack(c2), s2), v)
    assert np.array_equal(X.unpack(X.pack(c)), c)


def test_oracle_few_tokens_is_the_layer():
    cfg = W.CONFIGS["decode"].with_(T=6, H=128, F=128, E=8, k=3)
    d = W.make_inputs(cfg)
    f = lambda t: t.double().numpy()  # noqa: E731
    weights = lambda e: (f(d["w0"][e]), f(d["w0_up"][e]), f(d["w1"][e]))  # noqa: E731
    idx, w = X.route(d["logits"].numpy(), 3)
    ridx, rw = O.route_topk(d["logits"].numpy(), 3)
    assert np.array_equal(idx, ridx) and np.allclose(w, rw, rtol=1e-6)
    out, bound = X.few_tokens(f(d["x"]), idx, w, weights, "swiglu", 0, 8)
    ref = O.moe_layer(f(d["x"]), d["logits"].numpy(), 3, weights, "swiglu", route=(idx, w))
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-14) and (bound > 0).all() and (bound < 5e-3 * np.abs(out).max()).all()  # H sqrt(H) U2, a few times
    half = X.few_tokens(f(d["x"]), idx, w, lambda e: weights(e + 4), "swiglu", 4, 4)[0]
    rest = X.few_tokens(f(d["x"]), idx, w, weights, "swiglu", 0, 4)[0]
    assert np.allclose(half + rest, out, rtol=1e-12, atol=1e-14)
    assert Q.act("silu", np.array([0.0]))[0] == 0.0

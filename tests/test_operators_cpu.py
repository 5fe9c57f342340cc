"""Grouped routing, dense projection and the gradients without a GPU: refusals of the C ABI, and the oracle's pins.

No library call here reaches a kernel launch: each returns from host
validation.  The oracle's gradients are pinned by central differences, its
routing by closed forms and by the plain top-k routing's oracle.
"""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from oracle import moe_oracle as O
from oracle import operators_oracle as Q

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
NULL = None
FAKE = ctypes.c_void_p(16 * 1024)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(16 * 1024 + 4)


@pytest.fixture(scope="module")
def L():
    return ffi.lib()


def route(L, **over):
    a = dict(l=FAKE, b=NULL, T=10, E=64, k=4, score=1, G=8, tg=4, gt=2, rn=1, sc=1.0, i=FAKE, w=FAKE)
    a.update(over)
    return L.moe_route_grouped(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(T=0, l=NULL, i=NULL, w=NULL), OK), (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID),
    (dict(k=65), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(G=0), INVALID),
    (dict(G=7), INVALID), (dict(G=65), INVALID), (dict(tg=0), INVALID), (dict(tg=9), INVALID), (dict(gt=0), INVALID),
    (dict(gt=3), INVALID), (dict(G=64, gt=2), INVALID), (dict(tg=1, k=9), INVALID), (dict(sc=float("nan")), INVALID),
    (dict(sc=float("inf")), INVALID), (dict(E=2048), UNSUPPORTED), (dict(E=1024, G=1, tg=1, k=33), UNSUPPORTED),
    (dict(E=130, G=65, tg=2, gt=1), UNSUPPORTED), (dict(T=1 << 26), UNSUPPORTED), (dict(l=NULL), INVALID),
    (dict(i=NULL), INVALID), (dict(w=NULL), INVALID), (dict(l=ODD), INVALID), (dict(b=ODD), INVALID),
    (dict(i=ODD), INVALID), (dict(w=ODD), INVALID)])
def test_route_grouped_refusals(L, over, code):
    assert route(L, **over) == code


def route_bwd(L, **over):
    a = dict(l=FAKE, i=FAKE, g=FAKE, T=10, E=64, k=4, score=1, rn=1, sc=1.0, d=FAKE)
    a.update(over)
    return L.moe_route_grouped_backward(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(T=0, l=NULL), OK), (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(score=2), INVALID), (dict(sc=float("inf")), INVALID), (dict(E=1025), UNSUPPORTED), (dict(k=33), UNSUPPORTED),
    (dict(T=1 << 26), UNSUPPORTED), (dict(l=NULL), INVALID), (dict(i=NULL), INVALID), (dict(g=NULL), INVALID),
    (dict(d=NULL), INVALID), (dict(d=ODD), INVALID)])
def test_route_grouped_backward_refusals(L, over, code):
    assert route_bwd(L, **over) == code


def combine_bwd(L, **over):
    a = dict(g=FAKE, y=FAKE, i=FAKE, w=FAKE, T=10, k=2, H=64, R=40, dy=FAKE, dw=FAKE)
    a.update(over)
    return L.moe_combine_backward(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(T=0, g=NULL), OK), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(H=0), INVALID), (dict(R=-1), INVALID),
    (dict(H=66), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(g=NULL), INVALID),
    (dict(y=NULL), INVALID), (dict(i=NULL), INVALID), (dict(w=NULL), INVALID), (dict(dy=NULL), INVALID),
    (dict(dw=NULL), INVALID), (dict(dw=ODD), INVALID)])
def test_combine_backward_refusals(L, over, code):
    assert combine_bwd(L, **over) == code


def linear(L, **over):
    a = dict(x=FAKE, w=FAKE, wu=NULL, b=NULL, bu=NULL, r=NULL, M=10, N=64, K=64, act=2, od=0, z=NULL, zu=NULL, out=FAKE,
             ws=NULL, n=0)
    a.update(over)
    return L.moe_linear(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(M=0, x=NULL, w=NULL, out=NULL), OK), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(od=2), INVALID), (dict(K=60), UNSUPPORTED),
    (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(act=1), INVALID), (dict(act=0, wu=FAKE), INVALID), (dict(act=3, bu=FAKE), INVALID),
    (dict(act=2, zu=FAKE), INVALID), (dict(x=NULL), INVALID), (dict(w=NULL), INVALID), (dict(out=NULL), INVALID),
    (dict(x=ODD), INVALID), (dict(b=ODD), INVALID), (dict(r=ODD), INVALID), (dict(z=ODD), INVALID), (dict(out=ODD), INVALID)])
def test_linear_refusals(L, over, code):
    assert linear(L, **over) == code


def test_linear_workspace_refusal(L):
    # Sizes whose reduction is split need their workspace whole, if one is given.
    for M, N, K in [(1, 64, 8192), (130, 200, 4096), (4096, 64, 4096)]:
        need = ffi.linear_workspace_bytes(M, N, K, "none")
        if need:
            assert linear(L, M=M, N=N, K=K, ws=FAKE, n=need - 1) == WORKSPACE
    assert L.moe_linear_workspace_bytes(10, 64, 60, 2) == 0
    assert L.moe_linear_workspace_bytes(10, 64, 64, 9) == 0


def at(kib):
    return ctypes.c_void_p(kib << 10)


def test_overlaps_are_refused(L):
    """An output that shares bytes with an input or another output; addresses are told apart by KiB, none is read."""
    # [10, 64] logits take 2.5 KiB, [10, 4] choices 160 bytes
    r = dict(l=at(16), b=at(32), i=at(48), w=at(64))
    for o in (dict(i=at(18)), dict(w=at(16)), dict(w=at(48)), dict(i=at(32))):
        assert route(L, **{**r, **o}) == INVALID
    r = dict(l=at(16), i=at(32), g=at(48), d=at(64))
    for o in (dict(d=at(16)), dict(d=at(18)), dict(d=at(14)), dict(d=at(31)), dict(d=at(47))):
        assert route_bwd(L, **{**r, **o}) == INVALID
    # [10, 64] gradients 2.5 KiB, [40, 64] rows 10 KiB
    r = dict(g=at(16), y=at(32), i=at(64), w=at(80), dy=at(96), dw=at(128))
    for o in (dict(dy=at(32)), dict(dy=at(41)), dict(dy=at(18)), dict(dw=at(96)), dict(dw=at(80)), dict(dw=at(64))):
        assert combine_bwd(L, **{**r, **o}) == INVALID
    # x [10, 64] and outputs 1.25 KiB, weights [64, 64] 8 KiB
    r = dict(act=1, x=at(16), w=at(32), wu=at(64), b=at(96), bu=at(100), r=at(128), z=at(144), zu=at(160), out=at(176))
    for o in (dict(out=at(16)), dict(out=at(39)), dict(out=at(71)), dict(out=at(95)), dict(out=at(100)), dict(out=at(129)),
              dict(z=at(176)), dict(z=at(160)), dict(z=at(128)), dict(zu=at(177)), dict(zu=at(17)),
              dict(ws=at(176), n=1 << 20), dict(ws=at(8), n=1 << 14)):
        assert linear(L, **{**r, **o}) == INVALID
    r = dict(act=1, g=at(16), x=at(32), w=at(48), wu=at(64), z=at(80), zu=at(96), dx=at(112), dw=at(128), dwu=at(144),
             db=at(160), dbu=at(164), ws=at(1 << 12))
    for o in (dict(dx=at(16)), dict(dx=at(33)), dict(dx=at(128)), dict(dw=at(48)), dict(dw=at(137)), dict(dwu=at(71)),
              dict(db=at(80)), dict(dbu=at(160)), dict(dx=at(96)), dict(ws=at(150)), dict(ws=at(0x1000), dx=at(0x1001))):
        assert linear_bwd(L, **{**r, **o}) == INVALID


def test_layer_checks_its_shared_expert():
    from mixture_experts_layer_moe_amd import workloads as W
    from mixture_experts_layer_moe_amd.layer import MoELayer, SharedExpert
    cfg = W.CONFIGS["fine_grained"].with_(T=4, H=16, F=16, E=4, k=2, tile_m=16)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16)  # noqa: E731
    for sh in (SharedExpert(e(8, 16), None, e(16, 8)), SharedExpert(e(8, 16), e(8, 24), e(16, 8)),
               SharedExpert(e(8, 24), e(8, 24), e(16, 8)), SharedExpert(e(8, 16), e(8, 16), e(8, 16))):
        with pytest.raises(ValueError, match="shared"):
            MoELayer(cfg, e(4, 16), torch.empty(4, 4), None, e(4, 16, 16), e(4, 16, 16), e(4, 16, 16), shared=sh)


def linear_bwd(L, **over):
    a = dict(g=FAKE, x=FAKE, w=FAKE, wu=NULL, z=NULL, zu=NULL, M=10, N=64, K=64, act=2, od=0, dx=FAKE, dw=FAKE, dwu=NULL,
             db=NULL, dbu=NULL, ws=FAKE, n=1 << 30)
    a.update(over)
    return L.moe_linear_backward(*a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(M=0, g=NULL, ws=NULL, dw=NULL), OK), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(act=4), INVALID), (dict(od=2), INVALID), (dict(K=60), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(g=NULL), INVALID), (dict(ws=NULL), INVALID), (dict(z=FAKE), INVALID), (dict(act=0), INVALID),
    (dict(act=1, z=FAKE, wu=FAKE), INVALID), (dict(act=1, z=FAKE, zu=FAKE), INVALID), (dict(act=3, z=FAKE, zu=FAKE), INVALID),
    (dict(dwu=FAKE), INVALID), (dict(dbu=FAKE), INVALID), (dict(wu=FAKE), INVALID), (dict(w=NULL), INVALID),
    (dict(x=NULL), INVALID), (dict(g=ODD), INVALID), (dict(dx=ODD), INVALID), (dict(ws=ODD), INVALID), (dict(n=0), WORKSPACE)])
def test_linear_backward_refusals(L, over, code):
    assert linear_bwd(L, **over) == code


def test_binding_refuses_host_tensors_and_unknown_choices():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ffi.moe_linear(x, w)
    with pytest.raises(ValueError, match="device tensor"):
        ffi.moe_route_grouped(torch.zeros(4, 16), 2)
    with pytest.raises(ValueError, match="act"):
        ffi.linear_workspace_bytes(4, 8, 16, "relu")


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def test_oracle_routing_without_groups_is_the_plain_routing():
    rng = np.random.default_rng(0)
    l = rng.normal(size=(40, 24)).astype(np.float32)
    l[5] = l[5].round()  # equal logits
    for renorm in (True, False):
        a, b = Q.route_grouped(l, 5, renormalize=renorm), O.route_topk(l, 5, renorm)
        assert np.array_equal(a[0], b[0])
        np.testing.assert_allclose(a[1], b[1], rtol=1e-6)


def test_oracle_routing_closed_forms():
    inf, nan = np.inf, np.nan
    l = np.array([[0.0, 3.0, 1.0, 2.0, -1.0, 2.5, 2.5, -3.0]])
    # two groups of four: the sums of the two best are 5 (experts 0-3) and 5 (4-7): the lower group stays
    idx, _ = Q.route_grouped(np.log(np.array([[2.0, 3, 1, 1, 1, 2.5, 2.5, 1]])), 2, n_group=2, topk_group=1, group_top=1)
    assert idx.tolist() == [[1, 0]]
    idx, w = Q.route_grouped(l, 3, bias=np.array([9.0, 0, 0, 0, 0, 0, 0, 8.0]), score="sigmoid", renormalize=False, scale=2.0)
    assert idx.tolist() == [[0, 7, 1]]  # the bias chooses, and does not weigh
    np.testing.assert_allclose(w[0], 2 / (1 + np.exp(-np.array([0.0, -3.0, 3.0]))))
    idx, w = Q.route_grouped(np.array([[-inf, nan, 1.0, -inf], [-inf] * 4, [inf, 1.0, inf, -FMAX]]), 3)
    assert idx.tolist() == [[2, -1, -1], [-1, -1, -1], [0, 2, 1]]
    np.testing.assert_allclose(w, [[1, 0, 0], [0, 0, 0], [0.5, 0.5, 0]])
    idx, w = Q.route_grouped(np.full((1, 4), -1e6), 2, score="sigmoid")  # scores that underflow still weigh equally
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


FMAX = float(np.finfo(np.float32).max)


def _differences(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_oracle_router_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    l, d_w = rng.normal(size=(3, 7)), rng.normal(size=(3, 3))
    idx = np.array([[6, 0, 3], [1, 2, -1], [-1, -1, -1]], np.int32)
    got, _ = Q.route_grouped_backward(l, idx, d_w, score, renorm, 1.7)
    num = _differences(lambda x: float((Q.gate_weights(x, idx, score, renorm, 1.7) * d_w).sum()), l)
    np.testing.assert_allclose(got, num, atol=1e-8)


@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
def test_oracle_linear_gradients_against_differences(act):
    rng = np.random.default_rng(2)
    x, w, wu = rng.normal(size=(3, 4)), rng.normal(size=(5, 4)), rng.normal(size=(5, 4))
    b, bu, g = rng.normal(size=5), rng.normal(size=5), rng.normal(size=(3, 5))
    f = lambda x, w, wu, b, bu: float((Q.linear(x, w, wu, b, bu, act)[0] * g).sum())  # noqa: E731
    _, z, u = Q.linear(x, w, wu, b, bu, act)
    got = Q.linear_backward(g, x, w, wu, act, z, u)
    np.testing.assert_allclose(got["d_x"], _differences(lambda v: f(v, w, wu, b, bu), x), atol=1e-7)
    np.testing.assert_allclose(got["d_w"], _differences(lambda v: f(x, v, wu, b, bu), w), atol=1e-7)
    np.testing.assert_allclose(got["d_bias"], _differences(lambda v: f(x, w, wu, v, bu), b), atol=1e-7)
    if act == "swiglu":
        np.testing.assert_allclose(got["d_w_up"], _differences(lambda v: f(x, w, v, b, bu), wu), atol=1e-7)
        np.testing.assert_allclose(got["d_bias_up"], _differences(lambda v: f(x, w, wu, b, v), bu), atol=1e-7)


def test_oracle_combine_gradient_against_differences():
    rng = np.random.default_rng(3)
    y, g, w = rng.normal(size=(5, 4)), rng.normal(size=(2, 4)), rng.normal(size=(2, 2))
    inv = np.array([[3, -1], [0, 4]], np.int32)

    def f(y, w):
        out = np.zeros((2, 4))
        for t, j in np.ndindex(2, 2):
            if inv[t, j] >= 0:
                out[t] += w[t, j] * y[inv[t, j]]
        return float((out * g).sum())
    d_y, d_w, _ = Q.combine_backward(g, y, inv, w)
    assert np.isnan(d_y[[1, 2]]).all()
    np.testing.assert_allclose(np.nan_to_num(d_y), _differences(lambda v: f(v, w), y), atol=1e-8)
    np.testing.assert_allclose(d_w, _differences(lambda v: f(y, v), w), atol=1e-8)

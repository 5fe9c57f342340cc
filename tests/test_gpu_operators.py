"""Grouped routing, dense projection and the gradients on the GPU against the float64 oracle.

Tolerances (u = 2^-24, half an fp32 step; a bf16 result is within 2^-8 of its
value):
  * Indices and everything computed from small whole numbers (products whose
    fp32 sums are exact whatever their order, rounded once) are compared
    exactly.
  * Gate weights are a quotient of an fp32 exponential and a sum of at most k
    of them: exp 2 u, division 1 u, each addition 1 u of a sum of positive
    terms, the argument's rounding at most 2 u of |l| <= 16: within 2e-6.
  * Gradients of the router are sums of products of such weights: 4e-6 of the
    sum of the absolute terms.
  * d_topk_w: a thread adds ceil(H / 1024) groups of 4 products, then the
    block's 256 partial sums: (ceil(H / 1024) + 12) u of the sum of absolute
    products.
  * Products of arbitrary numbers: fp32 accumulation of R exact products in any
    order is within R 2^-23 of the sum of their absolute values (u doubled, in
    case the matrix unit truncates); activations add 1e-6 of the result (erf,
    hardware exp2 and reciprocal, a few u each), and pass an error of z on by
    at most 1.2.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from mixture_experts_layer_moe_amd import workloads as W
from mixture_experts_layer_moe_amd.layer import Gating, MoELayer, SharedExpert
from oracle import moe_oracle as O
from oracle import operators_oracle as Q

import parity_helpers as P

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
BF_HALF = 2.0 ** -8
INF, NAN, FMAX = float("inf"), float("nan"), float(torch.finfo(torch.float32).max)


def dev():
    return P.require_gpu()


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def guarded(shape, dtype, fill=-7.0, pad=64):
    """A tensor inside a larger one of `fill`; check() fails if anything around it was written."""
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device=dev())
    def check():
        torch.cuda.synchronize()
        assert bool((whole[:pad] == fill).all()) and bool((whole[pad + n:] == fill).all()), "written out of range"
    return whole[pad:pad + n].view(shape), check


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------

def check_route(logits, k, bias=None, **kw):
    T, E = logits.shape
    idx, c1 = guarded((T, k), torch.int32, -7)
    w, c2 = guarded((T, k), F32)
    d = dev()
    ffi.moe_route_grouped(logits.to(d), k, bias=None if bias is None else bias.to(d), topk_idx=idx, topk_w=w, **kw)
    c1(), c2()
    ridx, rw = Q.route_grouped(logits.numpy(), k, None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    np.testing.assert_allclose(n64(w), rw, rtol=2e-6, atol=1e-37)
    return idx, w


@pytest.mark.parametrize("T", [1, 3, 67])
@pytest.mark.parametrize("E,G,tg,gt,k", [
    (256, 8, 4, 2, 8), (256, 1, 1, 1, 8), (64, 8, 3, 1, 6), (64, 1, 1, 1, 1), (8, 1, 1, 1, 8), (160, 8, 3, 2, 6),
    (48, 3, 2, 2, 5), (60, 5, 5, 2, 7), (1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (96, 32, 7, 2, 9), (1024, 16, 4, 2, 32),
    (1024, 64, 64, 1, 32), (999, 27, 9, 2, 16), (128, 64, 9, 2, 12), (512, 16, 4, 2, 10), (20, 4, 2, 1, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_shapes(T, E, G, tg, gt, k, score, biased):
    g = gen(T * 1000 + E)
    l = torch.randn(T, E, generator=g) * 2
    b = torch.randn(E, generator=g) * 0.2 if biased else None
    check_route(l, k, b, score=score, n_group=G, topk_group=tg, group_top=gt, renormalize=(T + E) % 2 == 0, scale=2.5)


@pytest.mark.parametrize("E,G,tg,gt,k", [(256, 8, 4, 2, 8), (160, 8, 3, 2, 6), (256, 1, 1, 1, 16), (90, 3, 2, 1, 10), (192, 16, 5, 2, 9)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_many_tokens(E, G, tg, gt, k, score, biased):
    """Enough tokens for the form that shares a wavefront between four of them, with padding rows and masked experts."""
    g = gen(E)
    l = torch.randn(2051, E, generator=g) * 1.5
    l[::17] = -INF
    l[torch.rand(l.shape, generator=g) < 0.1] = -INF
    b = torch.randn(E, generator=g) * 0.1 if biased else None
    check_route(l, k, b, score=score, n_group=G, topk_group=tg, group_top=gt, renormalize=biased, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("G,tg,gt", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_and_extremes(score, renorm, G, tg, gt, biased):
    E, k = 32, 6
    g = gen(5)
    l = torch.randn(14, E, generator=g)
    l[0] = -INF                                # padding token
    l[1] = NAN
    l[2, 3:] = -INF                            # fewer than k experts left
    l[3, ::2] = -INF
    l[4] = -FMAX                               # masks of the type's lowest value: available, equal
    l[5, 4:] = -FMAX
    l[6, 7] = l[6, 20] = INF                   # counts as the largest finite value
    l[7] = 0.25                                # all equal: lowest ids, lowest groups
    l[8, 9:] = NAN
    l[9] = l[9].round()                        # many ties
    l[10] = -1000.0 + l[10]                    # every sigmoid underflows in fp32
    l[11] = 8.0 + l[11] * 0.1                  # sigmoids next to 1
    l[12, 8:] = -INF                           # one group only
    l[13, torch.arange(E) % 8 > 0] = -INF      # one expert per group
    b = (torch.randn(E // 2, generator=g) * 0.3).repeat_interleave(2) if biased else None
    if biased:
        b[5], b[6] = -INF, NAN                 # experts switched off by their bias
    check_route(l, k, b, score=score, n_group=G, topk_group=tg, group_top=gt, renormalize=renorm, scale=1.5)


def test_route_near_ties_are_decided_in_64_bits():
    """Scores that differ by far less than an fp32 step: the order is the exact one."""
    T, E, k = 512, 64, 8
    g = gen(9)
    base = torch.randn(T, E // 2, generator=g)
    l = torch.stack((base, torch.nextafter(base, base + 1)), dim=2).view(T, E)  # neighbours one fp32 step apart
    b = (torch.randn(E // 2, generator=g) * 0.1).repeat_interleave(2)
    for score in ("sigmoid", "softmax"):
        check_route(l, k, b, score=score, n_group=8, topk_group=4, group_top=2)
    check_route(l + 12.0, k, b, score="sigmoid")


def test_route_equals_the_plain_routing():
    l = torch.randn(1000, 64, generator=gen(1)).to(dev())
    a, b = ffi.moe_route_topk(l, 6), ffi.moe_route_grouped(l, 6, score="softmax")
    assert torch.equal(a[0], b[0])
    torch.testing.assert_close(a[1], b[1], rtol=2e-6, atol=0)


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (5, 8, 2), (33, 64, 6), (257, 160, 6), (3, 1024, 32), (9, 1, 1), (17, 37, 11),
                                   (2051, 256, 8), (2050, 130, 5), (2049, 260, 17)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(T, E, k, score, renorm):
    g = gen(E + k)
    l = torch.randn(T, E, generator=g) * 2
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    d_w = torch.randn(T, k, generator=g)
    if T > 4:
        idx[1] = -1                      # a padding token
        idx[2, max(1, k // 2):] = E + 3          # ids out of range take no part
        l[2] = -INF
        l[2, idx[2, 0]] = 0.5
        l[3, idx[3, 0]] = -INF           # a chosen expert that is not available
        l[4, idx[4, 0]] = INF
        l[0] = l[0] * 0 - FMAX
    out, check = guarded((T, E), F32)
    d = dev()
    ffi.moe_route_grouped_backward(l.to(d), idx.to(d), d_w.to(d), score=score, renormalize=renorm, scale=1.5, d_logits=out)
    check()
    ref, mag = Q.route_grouped_backward(l.numpy(), idx.numpy(), d_w.numpy(), score, renorm, 1.5)
    assert (np.abs(n64(out) - ref) <= 4e-6 * mag + 1e-37).all()


def test_route_backward_adds_up_a_repeated_expert():
    d = dev()
    l, idx = torch.randn(2, 8, generator=gen(0)), torch.tensor([[3, 3], [1, 0]], dtype=torch.int32)
    g = torch.tensor([[1.0, 2.0], [0.5, -1.0]])
    for score in ("softmax", "sigmoid"):
        out = ffi.moe_route_grouped_backward(l.to(d), idx.to(d), g.to(d), score=score, renormalize=False)
        ref, mag = Q.route_grouped_backward(l.numpy(), idx.numpy(), g.numpy(), score, False, 1.0)
        assert (np.abs(n64(out) - ref) <= 4e-6 * mag).all()


# ---------------------------------------------------------------------------
# Combine gradient
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,H,k,E,El,tm", [(1, 4, 1, 1, 1, 16), (1, 4096, 8, 8, 8, 16), (37, 64, 2, 8, 8, 16),
                                           (50, 1028, 6, 16, 4, 32), (21, 4100, 3, 4, 4, 16), (9, 128, 32, 40, 40, 16),
                                           (70, 260, 8, 64, 1, 64), (11, 2048, 11, 16, 8, 16)])
def test_combine_backward(T, H, k, E, El, tm):
    g = gen(T + H)
    idx = np.stack([np.random.default_rng(t).permutation(E)[:k] for t in range(T)]).astype(np.int32)
    perm = O.permute(idx, None, 0, El, tm)
    inv = np.asarray(perm["inv_perm"]).astype(np.int32).reshape(T, k)
    R = ffi.rows_capacity(T, k, El, tm)
    y, d_out, w = torch.randn(R, H, generator=g), torch.randn(T, H, generator=g), torch.rand(T, k, generator=g)
    d_y, c1 = guarded((R, H), F32)
    d_w, c2 = guarded((T, k), F32)
    d = dev()
    ffi.moe_combine_backward(d_out.to(d), y.to(d), torch.from_numpy(inv).to(d), w.to(d), d_y_perm=d_y, d_topk_w=d_w)
    c1(), c2()
    ref_y, ref_w, mag = Q.combine_backward(d_out.numpy(), y.numpy(), inv, w.numpy())
    got = d_y.cpu().numpy()
    named = ~np.isnan(ref_y)
    assert np.array_equal(got[named], ref_y[named].astype(np.float32))  # one product, rounded once
    assert (got[~named] == -7.0).all()                                  # rows behind the last token: as they were
    assert (np.abs(n64(d_w) - ref_w) <= (-(-H // 1024) + 12) * U * mag).all()


# ---------------------------------------------------------------------------
# Dense projection
# ---------------------------------------------------------------------------

def whole(shape, g, lim=3):
    return torch.randint(-lim, lim + 1, shape, generator=g).to(BF)


SHAPES = [(1, 1, 8), (1, 256, 64), (2, 17, 24), (5, 64, 1000), (16, 48, 512), (17, 100, 136), (31, 33, 72), (64, 64, 64),
          (65, 130, 200), (100, 7, 4096), (128, 128, 128), (129, 257, 320), (200, 512, 8), (255, 96, 1032), (256, 256, 256),
          (257, 1001, 456), (300, 64, 2048), (513, 384, 704), (1, 2048, 2056), (40, 1000, 3000), (700, 520, 136),
          (1030, 1100, 264), (1300, 1029, 136), (2051, 1536, 72)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("odt", [BF, F32])
def test_linear_whole_numbers(M, N, K, ws, odt):
    """Exact sums: every element is right to the last bit, in both types, split or not, and nothing else is written."""
    g = gen(M + N + K)
    x, w = whole((M, K), g), whole((N, K), g)
    bias, res = whole((N,), g).float(), whole((M, N), g).to(odt)
    d = dev()
    out, c1 = guarded((M, N), odt)
    z, c2 = guarded((M, N), BF)
    ffi.moe_linear(x.to(d), w.to(d), bias=bias.to(d), residual=res.to(d), out=out, z=z, use_workspace=ws)
    c1(), c2()
    zr = x.double() @ w.double().T + bias.double()
    assert torch.equal(out.cpu(), (zr + res.double()).float().to(odt))
    assert torch.equal(z.cpu(), zr.float().to(BF))
    plain = ffi.moe_linear(x.to(d), w.to(d), out_dtype=odt, use_workspace=ws)
    assert torch.equal(plain.cpu(), (x.double() @ w.double().T).float().to(odt))


# Sizes at which the launches choose each tile, split over the reduction or not, with a ragged edge in every direction.
@pytest.mark.parametrize("M,N,K", [(3001, 4100, 72), (1500, 4100, 520), (1500, 4100, 72), (4099, 130, 4104), (3600, 1029, 2056),
                                   (1795, 1029, 2056), (130, 513, 20488), (400, 770, 12296), (1500, 1300, 4104)])
def test_linear_tiles(M, N, K):
    g = gen(M + N + K)
    d = dev()
    x, w, res = whole((M, K), g).to(d), whole((N, K), g).to(d), whole((M, N), g).to(d).float()
    out, c1 = guarded((M, N), F32)
    out.copy_(res)
    z, c2 = guarded((M, N), BF)
    ffi.moe_linear(x, w, residual=out, out=out, z=z)
    c1(), c2()
    zr = torch.mm(x.double(), w.double().T)
    assert torch.equal(out, (zr + res).float())
    assert torch.equal(z, zr.float().to(BF))


@pytest.mark.parametrize("M,N,K", [(1500, 4100, 72), (1795, 4100, 520), (1500, 2050, 520), (1500, 2050, 72), (4099, 70, 4104),
                                   (4099, 1001, 520), (33, 33, 2056), (1300, 257, 72), (1500, 700, 4104)])
def test_linear_tiles_of_two_matrices(M, N, K):
    """The gate's bias lifts z to where its sigmoid is 1 in 32 bits, so that z u is whole too (below 2^24)."""
    g = gen(M + N + K)
    d = dev()
    x, w, wu, res = (whole(s, g).to(d) for s in ((M, K), (N, K), (N, K), (M, N)))
    bias, bu = torch.full((N,), 2048.0, device=d), whole((N,), g).float().to(d)
    out, c1 = guarded((M, N), F32)
    out.copy_(res)
    z, c2 = guarded((M, N), BF)
    zu, c3 = guarded((M, N), BF)
    ffi.moe_linear(x, w, w_up=wu, bias=bias, bias_up=bu, act="swiglu", residual=out, out=out, z=z, z_up=zu)
    c1(), c2(), c3()
    zr, ur = torch.mm(x.double(), w.double().T) + 2048.0, torch.mm(x.double(), wu.double().T) + bu
    assert float(zr.min()) > 64 and float((zr * ur).abs().max()) < 2 ** 24 - 64
    assert torch.equal(out, (zr * ur + res).float())
    assert torch.equal(z, zr.float().to(BF)) and torch.equal(zu, ur.float().to(BF))


@pytest.mark.parametrize("M,N,K", [(3001, 4104, 72), (1500, 4104, 520), (1500, 2056, 520), (1500, 4104, 72), (1500, 2056, 72),
                                   (203, 264, 136), (300, 268, 72)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("odt", [BF, F32])
def test_linear_rows_of_whole_pieces(M, N, K, act, odt):
    """Rows of 16-byte pieces on every tile, with and without a residual and the pre-activations, one or both."""
    g = gen(M + N + K)
    d = dev()
    dual = act == "swiglu"
    x, w, wu, r = (whole(s, g).to(d) for s in ((M, K), (N, K), (N, K), (M, N)))
    b = torch.full((N,), 2048.0, device=d) if dual else whole((N,), g).float().to(d)
    zr, ur = torch.mm(x.double(), w.double().T) + b, torch.mm(x.double(), wu.double().T)
    assert float((zr * ur).abs().max()) < 2 ** 24 - 64 and (not dual or float(zr.min()) > 64)
    for res, save in [(False, ""), (True, ""), (False, "z"), (True, "zu"), (True, "u"), (False, "zu")]:
        out, c1 = guarded((M, N), odt)
        z, c2 = guarded((M, N), BF)
        u, c3 = guarded((M, N), BF)
        ffi.moe_linear(x, w, w_up=wu if dual else None, bias=b, act=act, residual=r.to(odt) if res else None, out=out,
                       z=z if "z" in save else None, z_up=u if dual and "u" in save else None)
        c1(), c2(), c3()
        ref = (zr * ur if dual else zr) + (r.double() if res else 0)
        assert torch.equal(out, ref.float().to(odt)), (res, save)
        assert torch.equal(z, zr.float().to(BF) if "z" in save else torch.full_like(z, -7.0)), (res, save)
        assert torch.equal(u, ur.float().to(BF) if dual and "u" in save else torch.full_like(u, -7.0)), (res, save)


def act_bound(act, zb, z, u=None, ub=None):
    """Bound of the activation's error from z's (and u's)."""
    f = np.abs(Q.act(act, z))
    if act == "none":
        return zb
    own = 1.2 * zb + 1e-6 * f + 2e-7 * np.abs(z)
    if act != "swiglu":
        return own
    return own * np.abs(u) + (f + own) * ub + 1e-6 * f * np.abs(u)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (3, 200, 328), (16, 128, 512), (50, 33, 72), (130, 190, 520), (300, 257, 136),
                                   (600, 300, 1064), (1100, 1031, 72), (1029, 1152, 200)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("odt", [BF, F32])
def test_linear_activations(M, N, K, act, odt):
    g = gen(M * 7 + N)
    dual = act == "swiglu"
    x = torch.randn(M, K, generator=g).to(BF)
    w, wu = ((torch.randn(N, K, generator=g) * 2 / K ** 0.5).to(BF) for _ in range(2))
    b, bu = torch.randn(N, generator=g), torch.randn(N, generator=g)
    res = torch.randn(M, N, generator=g).to(odt)
    d = dev()
    z, c1 = guarded((M, N), BF)
    zu, c2 = guarded((M, N), BF)
    out, c3 = guarded((M, N), odt)
    ffi.moe_linear(x.to(d), w.to(d), w_up=wu.to(d) if dual else None, bias=b.to(d), bias_up=bu.to(d) if dual else None,
                   act=act, residual=res.to(d), out=out, z=z, z_up=zu if dual else None)
    c1(), c2(), c3()
    X, Wd, Wu = n64(x), n64(w), n64(wu)
    ref, zr, ur = Q.linear(X, Wd, Wu, n64(b), n64(bu), act, n64(res))
    zb = (K + 2) * 2 * U * (np.abs(X) @ np.abs(Wd).T + np.abs(n64(b)))
    ub = (K + 2) * 2 * U * (np.abs(X) @ np.abs(Wu).T + np.abs(n64(bu)))
    ob = act_bound(act, zb, zr, ur, ub) + 2 * U * (np.abs(ref) + np.abs(n64(res)))
    assert (np.abs(n64(out) - ref) <= ob * 1.01 + (BF_HALF * np.abs(ref) if odt is BF else 0)).all()
    assert (np.abs(n64(z) - zr) <= zb * 1.01 + BF_HALF * np.abs(zr)).all()
    if dual:
        assert (np.abs(n64(zu) - ur) <= ub * 1.01 + BF_HALF * np.abs(ur)).all()


@pytest.mark.parametrize("odt", [BF, F32])
@pytest.mark.parametrize("M", [3, 150, 400])
def test_linear_residual_in_place(odt, M):
    g = gen(3)
    N, K = 130, 1032
    x, w, res = whole((M, K), g), whole((N, K), g), whole((M, N), g).to(odt)
    d = dev()
    out = res.to(d)
    ffi.moe_linear(x.to(d), w.to(d), residual=out, out=out)
    assert torch.equal(out.cpu(), (x.double() @ w.double().T + res.double()).float().to(odt))


def test_linear_rows_do_not_touch_each_other():
    """Non-finite numbers stay in their own row; a NaN weight row stays in its own column."""
    g = gen(4)
    for M, N, K in [(20, 70, 136), (200, 300, 200), (3, 40, 2048)]:
        x, w = whole((M, K), g), whole((N, K), g)
        x[1, 3], w[2, K - 1] = NAN, INF
        d = dev()
        out = n64(ffi.moe_linear(x.to(d), w.to(d), out_dtype=F32))
        ref = x.double() @ w.double().T
        keep = np.ones((M, N), bool)
        keep[1], keep[:, 2] = False, False
        assert np.array_equal(out[keep], ref.numpy()[keep])
        assert np.isnan(out[1]).all()


BWD = [(1, 1, 8), (1, 64, 64), (3, 40, 72), (17, 100, 136), (64, 64, 64), (65, 130, 200), (128, 256, 128), (129, 257, 320),
       (300, 70, 264), (700, 257, 136), (70, 520, 1032), (260, 300, 520),
       (1030, 1100, 1064), (1100, 1027, 1288)]


@pytest.mark.parametrize("M,N,K", BWD)
@pytest.mark.parametrize("odt", [BF, F32])
def test_linear_backward_whole_numbers(M, N, K, odt):
    g = gen(M + N * K)
    d_out, x, w = whole((M, N), g).to(odt), whole((M, K), g), whole((N, K), g)
    d = dev()
    d_x, c1 = guarded((M, K), BF)
    d_w, c2 = guarded((N, K), BF)
    d_b, c3 = guarded((N,), F32)
    ffi.moe_linear_backward(d_out.to(d), x.to(d), w.to(d), d_x=d_x, d_w=d_w, d_bias=d_b)
    c1(), c2(), c3()
    G, X, Wd = d_out.double(), x.double(), w.double()
    assert torch.equal(d_x.cpu(), (G @ Wd).float().to(BF))
    assert torch.equal(d_w.cpu(), (G.T @ X).float().to(BF))
    assert torch.equal(d_b.cpu(), G.sum(0).float())


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 33, 72), (130, 190, 264), (300, 257, 136), (520, 64, 520), (1100, 1032, 1096)])
@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu"])
@pytest.mark.parametrize("odt", [BF, F32])
def test_linear_backward(M, N, K, act, odt):
    g = gen(M * 3 + N)
    dual = act == "swiglu"
    rb = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    x, w, wu, z, zu = rb(M, K), rb(N, K, std=0.1), rb(N, K, std=0.1), rb(M, N, std=2.0), rb(M, N)
    d_out = torch.randn(M, N, generator=g).to(odt)
    d = dev()
    outs = {n: guarded(s, t) for n, s, t in (("d_x", (M, K), BF), ("d_w", (N, K), BF), ("d_bias", (N,), F32))}
    if dual:
        outs |= {"d_w_up": guarded((N, K), BF), "d_bias_up": guarded((N,), F32)}
    ffi.moe_linear_backward(d_out.to(d), x.to(d), w.to(d), w_up=wu.to(d) if dual else None, act=act, z=z.to(d),
                            z_up=zu.to(d) if dual else None, **{n: t for n, (t, _) in outs.items()})
    G, X, Wd, Wu, Z, ZU = map(n64, (d_out, x, w, wu, z, zu))
    ref = Q.linear_backward(G, X, Wd, Wu, act, Z, ZU)
    # dz is off by 1e-6 of |d_out| (|act'| <= 1.2 and its terms) before its rounding to bf16.
    zb = {"dz": 1e-6 * np.abs(G) * (1 + np.abs(Z)) * (np.abs(ZU) if dual else 1.0)}
    if dual:
        zb["dz_up"] = 1e-6 * np.abs(G) * (1 + np.abs(Z))
    mats = [("dz", Wd, "d_w", "d_bias")] + ([("dz_up", Wu, "d_w_up", "d_bias_up")] if dual else [])
    xb = 0
    for name, weight, dw, db in mats:
        dz = np.abs(ref[name])
        eb = zb[name] + BF_HALF * dz
        xb = xb + eb @ np.abs(weight) + (len(mats) * N + 2) * 2 * U * (dz @ np.abs(weight))
        wb = eb.T @ np.abs(X) + (M + 2) * 2 * U * (dz.T @ np.abs(X))
        bb = zb[name].sum(0) + (M + 2) * U * dz.sum(0)
        for n, b, half in ((dw, wb, BF_HALF), (db, bb, U)):
            outs[n][1]()
            assert (np.abs(n64(outs[n][0]) - ref[n]) <= b * 1.01 + half * np.abs(ref[n])).all(), n
    outs["d_x"][1]()
    assert (np.abs(n64(outs["d_x"][0]) - ref["d_x"]) <= xb * 1.01 + BF_HALF * np.abs(ref["d_x"])).all()


# Sizes at which the launch chooses each tile, with each of its products split or not.
@pytest.mark.parametrize("M,N,K,act", [
    (1500, 1001, 4104, "none"), (2500, 130, 4104, "none"), (515, 1001, 4104, "none"), (4352, 700, 520, "none"),
    (257, 1300, 2056, "none"), (70, 1300, 4104, "none"), (4352, 70, 1032, "none"), (515, 3600, 520, "none"),
    (33, 1300, 72, "none"), (515, 1300, 72, "none"),
    (1300, 520, 4104, "swiglu"), (4352, 130, 2056, "swiglu"), (1300, 4100, 136, "swiglu"), (2500, 257, 2056, "swiglu"),
    (1500, 3600, 136, "swiglu"), (1300, 70, 2056, "swiglu"), (33, 2600, 1032, "swiglu"), (1500, 3100, 72, "swiglu"),
    (1300, 257, 72, "swiglu"), (33, 33, 72, "swiglu")])
def test_linear_backward_tiles(M, N, K, act):
    """Whole numbers throughout: with z of 32 or 64, silu(z) is z and silu'(z) is 1 in 32 bits."""
    g = gen(M + N + K)
    d = dev()
    G, x, w, wu, zu = (whole(s, g).to(d) for s in ((M, N), (M, K), (N, K), (N, K), (M, N)))
    z = (32 << torch.randint(0, 2, (M, N), generator=g)).to(BF).to(d)
    dual = act == "swiglu"
    dz, dzu = (G.double() * zu.double(), G.double() * z.double()) if dual else (G.double(), None)
    want = {"d_x": torch.mm(dz, w.double()) + (torch.mm(dzu, wu.double()) if dual else 0)}
    for s, v in (("", dz), ("_up", dzu))[:2 if dual else 1]:
        want |= {"d_w" + s: torch.mm(v.T.contiguous(), x.double()), "d_bias" + s: v.sum(0)}
    outs = {n: guarded(tuple(v.shape), F32 if "bias" in n else BF) for n, v in want.items()}
    up = dict(w_up=wu, z=z, z_up=zu) if dual else {}
    ffi.moe_linear_backward(G, x, w, act=act, **up, **{n: t for n, (t, _) in outs.items()})
    for n, (t, check) in outs.items():
        check()
        assert float(want[n].abs().max()) < 2 ** 24
        assert torch.equal(t, want[n].float().to(t.dtype)), n


def test_linear_backward_parts_and_empty_batch():
    """Gradients asked for one by one equal those asked for together; no rows: zero weight and bias gradients."""
    g = gen(8)
    M, N, K = 150, 72, 136
    d = dev()
    d_out, x, w, z = (t.to(d) for t in (whole((M, N), g), whole((M, K), g), whole((N, K), g), whole((M, N), g)))
    e = lambda *s, t=BF: torch.full(s, 5.0, dtype=t, device=d)  # noqa: E731
    full = dict(d_x=e(M, K), d_w=e(N, K), d_bias=e(N, t=F32))
    ffi.moe_linear_backward(d_out, x, w, act="silu", z=z, **full)
    for n, t in full.items():
        one = torch.full_like(t, 5.0)
        ffi.moe_linear_backward(d_out, x, w, act="silu", z=z, **{n: one})
        assert torch.equal(one, t), n
    empty = dict(d_x=e(0, K), d_w=e(N, K), d_w_up=e(N, K), d_bias=e(N, t=F32), d_bias_up=e(N, t=F32))
    ffi.moe_linear_backward(d_out[:0], x[:0], w, w_up=w, act="swiglu", z=z[:0], z_up=z[:0], **empty)
    assert all(not t.any() for t in empty.values())
    assert ffi.moe_linear(x[:0], w).shape == (0, N)
    assert ffi.moe_route_grouped(torch.empty(0, 8, device=d), 2)[0].shape == (0, 2)


def test_binding_refusals():
    d = dev()
    x, w = torch.zeros(4, 16, dtype=BF, device=d), torch.zeros(8, 16, dtype=BF, device=d)
    for kw, err in [(dict(bias=torch.zeros(7, device=d)), ValueError), (dict(bias=torch.zeros(8, dtype=BF, device=d)), TypeError),
                    (dict(bias=torch.zeros(8)), ValueError), (dict(act="swiglu"), ffi.MoEError),
                    (dict(out=torch.zeros(4, 8, dtype=torch.float16, device=d)), ValueError),
                    (dict(out=torch.zeros(8, 4, dtype=BF, device=d).T), ValueError),
                    (dict(residual=torch.zeros(4, 8, device=d)), TypeError), (dict(act="tanh"), ValueError)]:
        with pytest.raises(err):
            ffi.moe_linear(x, w, **kw)
    with pytest.raises(ValueError):
        ffi.moe_linear(x[:, ::2], w[:, :8].contiguous())
    with pytest.raises(ffi.MoEError):
        ffi.moe_linear(x[:, :12].contiguous(), w[:, :12].contiguous())
    with pytest.raises(ffi.MoEError):
        ffi.moe_route_grouped(torch.zeros(4, 10, device=d), 2, n_group=3)


# ---------------------------------------------------------------------------
# Together, captured, on other streams
# ---------------------------------------------------------------------------

def layer_inputs(seed=0, T=150):
    cfg = W.CONFIGS["fine_grained"].with_(T=T, H=256, F=128, E=32, k=4, tile_m=16, logits="normal", seed=seed)
    d = W.make_inputs(cfg, dev())
    g = gen(seed + 20)
    sh = [(torch.randn(*s, generator=g) * 0.05).to(BF).to(dev()) for s in ((192, 256), (192, 256), (256, 192))]
    d["logits"][3] = -INF  # a padding token
    bias = (torch.randn(32, generator=g) * 0.1).to(dev())
    return cfg, d, Gating(bias=bias, score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5), SharedExpert(*sh)


def layer_reference(cfg, d, gating, shared):
    idx, w = Q.route_grouped(d["logits"].cpu().numpy(), cfg.k, gating.bias.cpu().numpy(), gating.score, gating.n_group,
                             gating.topk_group, gating.group_top, True, gating.scale)
    x = n64(d["x"])
    out = np.zeros_like(x)
    W0, WU, W1 = (n64(d[n]) for n in ("w0", "w0_up", "w1"))
    for t, j in np.ndindex(*idx.shape):
        e = idx[t, j]
        if e >= 0:
            h = Q.act("silu", W0[e] @ x[t]) * (WU[e] @ x[t])
            out[t] += w[t, j] * (W1[e] @ h)
    h, _, _ = Q.linear(x, n64(shared.w0), n64(shared.w0_up), act_name="swiglu")
    return out + h @ n64(shared.w1).T


def test_layer_with_gating_and_shared_expert():
    cfg, d, gating, shared = layer_inputs()
    ref = layer_reference(cfg, d, gating, shared)
    outs = []
    for kw in (dict(), dict(fused_gather=True)):
        layer = MoELayer.from_inputs(cfg, d, gating=gating, shared=shared, **kw)
        out = layer.run()
        P.assert_output_close(n64(out), ref, "layer with gating and shared expert")
        outs.append(out.clone())
        assert torch.equal(layer.run(), outs[-1])  # nothing is left behind from call to call
    assert torch.equal(*outs)


def test_signalled_layer_with_gating_and_shared_expert():
    """The one-launch path adds the shared expert as the four calls do."""
    cfg, d, gating, shared = layer_inputs()
    cfg = cfg.with_(tile_m=256)
    layer = MoELayer.from_inputs(cfg, d, gating=gating, shared=shared, signalled=True)
    P.assert_output_close(n64(layer.run()), layer_reference(cfg, d, gating, shared), "signalled layer with shared expert")


def test_layer_replayed_from_a_graph_and_on_another_stream():
    cfg, d, gating, shared = layer_inputs()
    layer = MoELayer.from_inputs(cfg, d, gating=gating, shared=shared)
    eager = layer.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.out.fill_(NAN)
    s.wait_stream(torch.cuda.current_stream())
    layer.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(layer.out, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    _, d2, _, _ = layer_inputs(seed=7)
    for i in range(4):
        src = d2 if i % 2 else d
        layer.x.copy_(src["x"])
        layer.logits.copy_(src["logits"])
        want = layer.run().clone()
        layer.out.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, want), i


def test_gradients_replayed_from_a_graph():
    g = gen(11)
    d = dev()
    M, N, K = 300, 264, 520
    t = dict(d_out=torch.randn(M, N, generator=g).to(BF).to(d), x=torch.randn(M, K, generator=g).to(BF).to(d),
             w=torch.randn(N, K, generator=g).to(BF).to(d), w_up=torch.randn(N, K, generator=g).to(BF).to(d))
    z, zu = torch.empty(M, N, dtype=BF, device=d), torch.empty(M, N, dtype=BF, device=d)
    outs = dict(d_x=torch.empty(M, K, dtype=BF, device=d), d_w=torch.empty(N, K, dtype=BF, device=d),
                d_w_up=torch.empty(N, K, dtype=BF, device=d), d_bias=torch.empty(N, device=d), d_bias_up=torch.empty(N, device=d))
    out = torch.empty(M, N, dtype=BF, device=d)
    ws, wsb = ffi.alloc_linear_workspace(M, N, K, "swiglu", d), ffi.alloc_linear_backward_workspace(M, N, K, "swiglu", d)

    def step():
        ffi.moe_linear(t["x"], t["w"], w_up=t["w_up"], act="swiglu", z=z, z_up=zu, out=out, ws=ws, use_workspace=False)
        ffi.moe_linear_backward(t["d_out"], t["x"], t["w"], w_up=t["w_up"], act="swiglu", z=z, z_up=zu, ws=wsb, **outs)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        t["x"].add_(0.25)
        step()
        want = [v.clone() for v in (out, *outs.values())]
        for v in (out, *outs.values()):
            v.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (out, *outs.values()))), i


def test_router_gradients_replayed_from_a_graph():
    g = gen(14)
    d = dev()
    T, E, k, H = 67, 64, 6, 256
    logits, y, d_out = (torch.randn(*s, generator=g).to(d) for s in ((T, E), (T * k + 64 * 16, H), (T, H)))
    idx, w = torch.empty(T, k, dtype=torch.int32, device=d), torch.empty(T, k, device=d)
    inv = torch.randperm(y.shape[0], generator=g)[:T * k].view(T, k).to(torch.int32)
    inv[3, 2] = inv[5] = -1
    inv = inv.to(d)
    d_y, d_w, d_l = torch.zeros_like(y), torch.empty_like(w), torch.empty_like(logits)

    def step():
        ffi.moe_route_grouped(logits, k, score="sigmoid", n_group=8, topk_group=4, group_top=2, topk_idx=idx, topk_w=w)
        ffi.moe_combine_backward(d_out, y, inv, w, d_y, d_w)
        ffi.moe_route_grouped_backward(logits, idx, d_w, score="sigmoid", d_logits=d_l)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        logits.mul_(-1.25)
        step()
        want = [v.clone() for v in (idx, w, d_y, d_w, d_l)]
        for v in (w, d_y, d_w, d_l):
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (idx, w, d_y, d_w, d_l))), i


# ---------------------------------------------------------------------------
# Offsets past 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [3, 40])
def test_linear_longest_rows(M):
    """The longest reduction, and the widest weights of the input gradient; sums below 2^24."""
    N, K = 24, 1 << 20
    d = dev()
    g = torch.Generator(device=d).manual_seed(19)
    few = lambda *s: torch.randint(-2, 3, s, generator=g, device=d, dtype=torch.int8).to(BF)  # noqa: E731
    x, w, d_out = few(M, K), few(N, K), few(M, N)
    want = torch.mm(x.double(), w.double().T).float()
    for ws in (True, False):
        assert torch.equal(ffi.moe_linear(x, w, out_dtype=F32, use_workspace=ws), want)
    d_x, d_w = torch.empty_like(x), torch.empty_like(w)
    ffi.moe_linear_backward(d_out, x, w, d_x=d_x, d_w=d_w)
    assert torch.equal(d_x, torch.mm(d_out.double(), w.double()).float().to(BF))
    assert torch.equal(d_w, torch.mm(d_out.double().T.contiguous(), x.double()).float().to(BF))


def test_route_offsets_past_32_bits():
    """More than 2^31 logits: tokens at both ends and around the limit equal the same tokens alone."""
    d = dev()
    E, k = 1024, 4
    T = (1 << 21) + 300
    logits = torch.zeros(T, E, device=d)
    some = torch.cat([torch.arange(0, 64), torch.arange((1 << 20) - 64, (1 << 20) + 64), torch.arange(T - 364, T)]).to(d)
    part = torch.randn(len(some), E, generator=gen(15)).to(d)
    logits[some] = part
    kw = dict(score="sigmoid", n_group=8, topk_group=3, group_top=2)
    idx, w = ffi.moe_route_grouped(logits, k, **kw)
    pidx, pw = ffi.moe_route_grouped(part, k, **kw)
    assert torch.equal(idx[some], pidx) and torch.equal(w[some], pw)
    d_w = torch.zeros(T, k, device=d)
    pd = torch.randn(len(some), k, generator=gen(16)).to(d)
    d_w[some] = pd
    d_l = ffi.moe_route_grouped_backward(logits, idx, d_w, score="sigmoid")
    assert torch.equal(d_l[some], ffi.moe_route_grouped_backward(part, pidx, pd, score="sigmoid"))
    d_l[some] = 0
    assert not bool(d_l.any())


def test_combine_backward_offsets_past_32_bits():
    d = dev()
    H, R = 2048, (1 << 20) + 600
    rows = torch.tensor([0, 1, (1 << 19) - 1, 1 << 19, 1 << 20, (1 << 20) + 1, R - 2, R - 1])
    g = gen(17)
    y = torch.zeros(R, H, device=d)
    part = whole((len(rows), H), g).float().to(d)
    y[rows.to(d)] = part
    inv = rows.view(4, 2).to(torch.int32).to(d)
    d_out, w = whole((4, H), g).float().to(d), whole((4, 2), g).float().to(d)
    d_y, d_w = ffi.moe_combine_backward(d_out, y, inv, w, torch.full((R, H), 9.0, device=d))
    pos = torch.arange(8, dtype=torch.int32, device=d).view(4, 2)
    p_y, p_w = ffi.moe_combine_backward(d_out, part, pos, w)
    assert torch.equal(d_y[rows.to(d)], p_y) and torch.equal(d_w, p_w)
    d_y[rows.to(d)] = 9.0
    assert bool((d_y == 9.0).all())


@pytest.mark.parametrize("M,N,K", [((1 << 21) + 70, 8, 1032), ((1 << 21) + 70, 1032, 8), (2050, (1 << 20) - 1, 8)])
def test_linear_offsets_past_32_bits(M, N, K):
    """More than 2^31 elements of x, of out and its gradient; whole numbers, so every sum is exact."""
    d = dev()
    g = torch.Generator(device=d).manual_seed(18)
    big = lambda *s: torch.randint(-2, 3, s, generator=g, device=d, dtype=torch.int8).to(BF)  # noqa: E731
    x, w = big(M, K), big(N, K)
    out = ffi.moe_linear(x, w)
    rows = torch.tensor([0, 1, M // 2, M - 200, M - 2, M - 1], device=d)
    assert torch.equal(out[rows], torch.mm(x[rows].double(), w.double().T).float().to(BF))
    d_out = out.clamp_(-2, 2)
    d_x, d_w, d_b = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=d)
    ffi.moe_linear_backward(d_out, x, w, d_x=d_x, d_w=d_w, d_bias=d_b)
    assert torch.equal(d_x[rows], torch.mm(d_out[rows].double(), w.double()).float().to(BF))
    cols = torch.tensor([0, N // 2, N - 1], device=d)
    gc = d_out[:, cols].double()
    assert torch.equal(d_b[cols], gc.sum(0).float())
    want = torch.zeros(3, K, dtype=torch.float64, device=d)
    for i in range(0, M, 1 << 18):
        want += torch.mm(gc[i:i + (1 << 18)].T.contiguous(), x[i:i + (1 << 18)].double())
    assert torch.equal(d_w[cols], want.float().to(BF))


def test_router_training_step_against_differences():
    """route_grouped -> combine and back: the gradient of the logits is that of differences of the oracle's output."""
    T, E, k, H, El, tm = 6, 8, 3, 32, 8, 16
    g = gen(12)
    d = dev()
    l, b = torch.randn(T, E, generator=g), torch.randn(E, generator=g) * 0.1
    idx, w = ffi.moe_route_grouped(l.to(d), k, bias=b.to(d), score="sigmoid", n_group=2, topk_group=1, group_top=2, scale=2.5)
    x = torch.zeros(T, H, dtype=BF, device=d)
    p = ffi.moe_permute(x, idx, None, E, 0, El, 1, tm)
    y = torch.randn(p.R_cap, H, generator=g).to(d)
    d_out = torch.randn(T, H, generator=g).to(d)
    _, d_w = ffi.moe_combine_backward(d_out, y, p.inv_perm, w)
    d_l = ffi.moe_route_grouped_backward(l.to(d), idx, d_w, score="sigmoid", scale=2.5)
    I, INV, Y, G = idx.cpu().numpy(), p.inv_perm.cpu().numpy(), n64(y), n64(d_out)

    def loss(v):
        gw = Q.gate_weights(v, I, "sigmoid", True, 2.5)
        return float(sum(gw[t, j] * (Y[INV[t, j]] @ G[t]) for t, j in np.ndindex(T, k)))
    L64, num = n64(l), np.zeros((T, E))
    for i in np.ndindex(T, E):
        a, c = L64.copy(), L64.copy()
        a[i] += 1e-6
        c[i] -= 1e-6
        num[i] = (loss(a) - loss(c)) / 2e-6
    # differences are good to about 1e-8 of the loss's terms, fp32 to 1e-5 of the sum of the absolute terms
    mag = 2.5 * np.abs(n64(d_w)).sum(1, keepdims=True)
    assert (np.abs(n64(d_l) - num) <= 2e-5 * mag).all()


def test_two_calls_at_once_on_two_streams():
    g = gen(13)
    d = dev()
    M, N, K = 37, 520, 4104
    a, b, w = whole((M, K), g).to(d), whole((M, K), g).to(d), whole((N, K), g).to(d)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    r1, r2 = ffi.moe_linear(a, w, out_dtype=F32, stream=s1), ffi.moe_linear(b, w, out_dtype=F32, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(r1.cpu(), (a.double() @ w.double().T).float().cpu())
    assert torch.equal(r2.cpu(), (b.double() @ w.double().T).float().cpu())

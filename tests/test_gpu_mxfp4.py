"""4-bit operands (MXFP4) on the GPU against the float64 oracle.

Tolerances:
  * Codes, scales and values read back are compared exactly.
  * Products of codes and scales whose fp32 sums are exact whatever their order (multiples of 2^-4 below 2^20) are
    compared exactly, rounded once to bf16 where that is the output.
  * Other products: fp32 accumulation of K exact products in any order is within K 2^-23 of the sum of their absolute
    values (u = 2^-24 doubled, in case the matrix unit truncates); bias and residual add a step each; activations pass an
    error of z on by at most 1.2 and add 1e-6 of the result (erf, hardware exp2 and reciprocal, a few u each).  A bf16
    output adds half a step, 2^-8.
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
U2 = 2.0 ** -23
BF_HALF = 2.0 ** -8


def dev():
    return P.require_gpu()


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def guarded(shape, dtype, fill, pad=64):
    """A tensor inside a larger one of `fill`; check() fails if anything around it was written."""
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device=dev())

    def check():
        torch.cuda.synchronize()
        assert bool((whole[:pad] == fill).all()) and bool((whole[pad + n:] == fill).all()), "written out of range"
    return whole[pad:pad + n].view(shape), check


def n64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------
# Quantising and reading back
# ---------------------------------------------------------------------------

def check_quantize(x):
    codes, c1 = guarded((*x.shape[:-1], x.shape[-1] // 2), U8, 0xA5)
    scales, c2 = guarded((*x.shape[:-1], x.shape[-1] // 32), U8, 0xA5)
    q = ffi.moe_mxfp4_quantize(x.to(dev()), out=ffi.Mxfp4(codes, scales))
    c1(), c2()
    ref, s = X.quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), X.pack(ref))
    want = X.values(X.pack(ref), s)
    for dt in (BF, F32):
        out, c3 = guarded(x.shape, dt, -7.0)
        ffi.moe_mxfp4_dequantize(q, out=out)
        c3()
        got = n64(out)
        assert np.array_equal(got, want, equal_nan=True)
        fin = ~np.isnan(want)
        assert np.array_equal(np.signbit(got)[fin], np.signbit(want)[fin])


@pytest.mark.parametrize("R,K", [(1, 32), (1, 64), (3, 96), (7, 32), (5, 1440), (64, 7168), (129, 2048), (1003, 160)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_quantize_shapes(R, K, dt):
    g = gen(R + K)
    check_quantize((torch.randn(R, K, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))).to(dt))


@pytest.mark.parametrize("dt", [BF, F32])
def test_quantize_every_bf16_value_under_every_lead(dt):
    """All finite bf16 magnitudes below 8, both signs, in blocks whose scale a lead value fixes; then moved by powers of two."""
    v = torch.arange(0x0000, 0x4100, dtype=torch.int32).to(torch.int16).view(BF)
    v = torch.cat((v, -v))
    v = torch.cat((v, torch.zeros(-len(v) % 31, dtype=BF))).view(-1, 31)
    for lead in (4.0, 7.0):
        x = torch.cat((torch.full((len(v), 1), lead, dtype=BF), v), dim=1)
        check_quantize(x.to(dt))
    for e in (-131, -129, -100, -3, 5, 60, 124):
        check_quantize(torch.ldexp(torch.cat((torch.full((len(v), 1), 4.0, dtype=BF), v), dim=1).double(), torch.tensor(float(e))).to(dt)[::37])


@pytest.mark.parametrize("dt", [BF, F32])
def test_quantize_zeros_subnormals_infinities_and_nan(dt):
    x = torch.zeros(12, 64, dtype=dt)
    x[1] = -0.0
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4, 0], x[4, 1] = -float("inf"), 1.0
    x[5] = torch.finfo(dt).max
    x[6] = -torch.finfo(dt).max
    x[7] = torch.finfo(dt).tiny
    x[8] = torch.finfo(dt).tiny / 64                      # subnormal
    x[9, ::3] = 2.0 ** -127
    x[10] = torch.linspace(-1, 1, 64, dtype=torch.float64).to(dt) * 2.0 ** -126
    x[11, 31], x[11, 32] = 3.0, 1e-30
    check_quantize(x)


def test_dequantize_every_code_and_scale():
    c = torch.arange(256, dtype=torch.int32).to(U8).repeat(256, 1)             # [256, 256] bytes: 512 values a row
    s = torch.arange(256, dtype=torch.int32).to(U8)[:, None].repeat(1, 16)
    for dt in (BF, F32):
        got = n64(ffi.moe_mxfp4_dequantize(ffi.Mxfp4(c.to(dev()), s.contiguous().to(dev())), out_dtype=dt))
        want = X.values(c.numpy(), s.numpy())
        big = float(torch.finfo(dt).max)
        want = np.where(np.abs(want) > big, np.sign(want) * np.inf, want)
        assert np.array_equal(got, want, equal_nan=True)


def test_quantize_stacks_streams_and_large():
    x = torch.randn(3, 5, 96, generator=gen(0)).to(BF)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    xd = x.to(dev())
    torch.cuda.synchronize()
    q = ffi.moe_mxfp4_quantize(xd, stream=st)
    v = ffi.moe_mxfp4_dequantize(q, stream=st)
    st.synchronize()
    ref, s = X.quantize(x.double().numpy())
    assert q.shape == (3, 5, 96) and np.array_equal(n64(v), X.values(X.pack(ref), s))
    # more than 2^32 bytes of values, checked at both ends
    n = (1 << 31) // 4096 + 3
    big = torch.zeros(n, 4096, dtype=BF, device=dev())
    big[0], big[-1] = xd[0, 0, 0], torch.arange(4096, device=dev()).to(BF)
    q = ffi.moe_mxfp4_quantize(big)
    ref, s = X.quantize(big[-1:].cpu().double().numpy())
    assert np.array_equal(q.codes[-1:].cpu().numpy(), X.pack(ref)) and np.array_equal(q.scales[-1:].cpu().numpy(), s)
    out = ffi.moe_mxfp4_dequantize(q, out=big)
    assert np.array_equal(n64(out[-1:]), X.values(X.pack(ref), s)) and float(out[1:-1].abs().max()) == 0.0


# ---------------------------------------------------------------------------
# Dense products
# ---------------------------------------------------------------------------

def packed(g, shape, lo=126, hi=129):
    """Random codes, scales from lo to hi - 1."""
    K = shape[-1]
    c = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, dtype=torch.int32).to(U8)
    s = torch.randint(lo, hi, (*shape[:-1], K // 32), generator=g, dtype=torch.int32).to(U8)
    return ffi.Mxfp4(c, s)


def on(q):
    return None if q is None else ffi.Mxfp4(*(t.to(dev()) for t in q))


def vals(q):
    return None if q is None else X.values(q.codes.numpy(), q.scales.numpy())


def to_bf16(a):
    return torch.from_numpy(a).to(F32).to(BF).double().numpy()


SHAPES = [(1, 1, 128), (1, 2048, 256), (2, 17, 128), (3, 64, 384), (15, 33, 640), (16, 16, 512), (17, 100, 128), (31, 48, 1408),
          (32, 130, 256), (33, 16, 896), (64, 200, 512), (65, 128, 128), (127, 129, 384), (128, 128, 256), (129, 257, 640),
          (200, 1001, 1408), (257, 64, 128), (300, 383, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_exact(M, N, K, dt):
    g = gen(M * 7 + N + K)
    x, w = packed(g, (M, K)), packed(g, (N, K))
    out, check = guarded((M, N), dt, -7.0)
    ffi.moe_linear_mxfp4(on(x), on(w), out=out)
    check()
    ref = vals(x) @ vals(w).T
    assert np.array_equal(n64(out), ref if dt == F32 else to_bf16(ref))


def bound(x, w, K):
    return K * U2 * (np.abs(x) @ np.abs(w).T)


def check_linear(x, w, w_up=None, bias=None, bias_up=None, act="none", residual=None, dt=F32, in_place=False):
    M, N = x.codes.shape[0], w.codes.shape[0]
    K = w.shape[1]
    out, check = guarded((M, N), dt, -7.0)
    d = dev()
    f = lambda t: None if t is None else t.to(d)  # noqa: E731
    res = f(residual)
    if in_place:
        out.copy_(res)
        res = out
    ffi.moe_linear_mxfp4(on(x), on(w), w_up=on(w_up), bias=f(bias), bias_up=f(bias_up), act=act, residual=res, out=out)
    check()
    xv, wv, uv = vals(x), vals(w), vals(w_up)
    n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    ref, z, u = Q.linear(xv, wv, uv, n(bias), n(bias_up), act, n(residual))
    tol = 1.2 * (bound(xv, wv, K) + U2 * np.abs(z))
    if act == "swiglu":
        du = bound(xv, uv, K) + U2 * np.abs(u)
        tol = tol * (np.abs(u) + du) + np.abs(Q.act("silu", z)) * du
    plain = ref if residual is None else ref - n(residual)
    tol = tol + (1e-6 if act != "none" else U2) * np.abs(plain) + U2 * np.abs(ref) + 1e-37
    if dt == BF:
        tol = tol + BF_HALF * (np.abs(ref) + tol)
    assert (np.abs(n64(out) - ref) <= tol).all()


@pytest.mark.parametrize("M,N,K", [(1, 96, 1408), (5, 7, 384), (40, 100, 256), (150, 131, 640), (260, 512, 1024)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_epilogues(M, N, K, act, dt):
    g = gen(M + N + K)
    x, w = packed(g, (M, K), 122, 126), packed(g, (N, K), 118, 124)
    up = packed(g, (N, K), 118, 124) if act == "swiglu" else None
    b = torch.randn(N, generator=g)
    bu = torch.randn(N, generator=g) if act == "swiglu" else None
    r = torch.randn(M, N, generator=g).to(dt)
    check_linear(x, w, up, act=act, dt=dt)
    check_linear(x, w, up, b, bu, act, r, dt)
    check_linear(x, w, up, bias_up=bu, act=act, residual=r, dt=dt, in_place=True)


@pytest.mark.parametrize("M,N,K,act", [(4096, 4096, 384, "none"), (3000, 2500, 640, "none"), (2050, 3333, 384, "swiglu"),
                                       (2048, 4096, 256, "gelu")])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_large_tiles(M, N, K, act, dt):
    """Products that fill the card, against a float64 product on the device."""
    g = gen(M + N)
    x, w = packed(g, (M, K), 124, 127), packed(g, (N, K), 119, 122)
    up = packed(g, (N, K), 119, 122) if act == "swiglu" else None
    out, check = guarded((M, N), dt, -7.0)
    ffi.moe_linear_mxfp4(on(x), on(w), w_up=on(up), act=act, out=out)
    check()
    v = lambda q: torch.from_numpy(vals(q)).to(dev())  # noqa: E731
    xv, wv = v(x), v(w)
    ref = xv @ wv.T
    # (sums of products of multiples of 2^-4 and 2^-9 below 2^11: exact in fp32)
    if act == "none":
        assert torch.equal(out.double(), ref if dt == F32 else ref.to(F32).to(BF).double())
        return
    if act == "gelu":
        ref = torch.nn.functional.gelu(ref)
    else:
        ref = torch.nn.functional.silu(ref) * (xv @ v(up).T)
    tol = 1e-6 * ref.abs() + (BF_HALF * ref.abs() * (1 + 1e-6) if dt == BF else 0) + 1e-30
    if act == "gelu":
        tol = tol + 4e-7 * (xv @ wv.T).abs()  # (1 + erf cancels where z is far below 0: two steps of z / 2)
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("M,N,K,act", [
    (4000, 3990, 1152, "none"), (2001, 3991, 1152, "swiglu"),                               # 256 x 256
    (1500, 3801, 2176, "none"), (900, 2816, 2944, "swiglu"),                                # 256 x 128
    (2047, 2040, 896, "none"), (1100, 2001, 512, "none"), (1300, 1301, 640, "swiglu"),      # 128 x 128
    (2000, 2100, 384, "none"), (2001, 1990, 384, "swiglu"),                                 # several to a CU
    (65, 8000, 384, "none"), (200, 1500, 2176, "swiglu"),                                   # 64 rows
    (64, 64, 8192, "none"), (33, 50, 6272, "none"), (49, 40, 8192, "swiglu"),               # streamed, 64 rows
    (32, 500, 4096, "none"), (17, 333, 7168, "swiglu")])                                    # streamed, 32 rows
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_kinds_of_tiles(M, N, K, act, dt):
    """Rows and columns that end inside a tile, odd row lengths and half stages at its end, bias and residual; against a
    float64 product on the device."""
    g = gen(M + N + K)
    x, w = packed(g, (M, K), 124, 127), packed(g, (N, K), 119, 122)
    up = packed(g, (N, K), 119, 122) if act == "swiglu" else None
    b = torch.randint(-4, 5, (N,), generator=g).float()
    r = (torch.randint(-64, 65, (M, N), generator=g) / 8).to(dt)
    out, check = guarded((M, N), dt, -7.0)
    ffi.moe_linear_mxfp4(on(x), on(w), w_up=on(up), bias=b.to(dev()), act=act, residual=r.to(dev()), out=out)
    check()
    v = lambda q: torch.from_numpy(vals(q)).to(dev())  # noqa: E731
    xv = v(x)
    z, rd = xv @ v(w).T + b.double().to(dev()), r.double().to(dev())
    if act == "none":  # (multiples of 2^-13 below 2^11: exact in fp32)
        ref = z + rd
        assert torch.equal(out.double(), ref if dt == F32 else ref.to(F32).to(BF).double())
        return
    plain = torch.nn.functional.silu(z) * (xv @ v(up).T)
    tol = 1e-6 * plain.abs() + U2 * (plain + rd).abs() + 1e-30
    tol = tol + (BF_HALF * ((plain + rd).abs() + tol) if dt == BF else 0)
    assert bool(((out.double() - plain - rd).abs() <= tol).all())


@pytest.mark.parametrize("tile_m,T,k,E,N,K", [(256, 900, 4, 8, 1201, 384), (256, 600, 2, 8, 2100, 640), (256, 4000, 4, 8, 1999, 384),
                                              (256, 150, 2, 8, 1500, 1152), (256, 200, 2, 8, 2001, 2176),
                                              (128, 900, 2, 8, 2000, 640), (64, 300, 3, 16, 1500, 1152)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_kinds_of_tiles(tile_m, T, k, E, N, K, act, gather):
    """Experts whose rows end inside a tile, one without any, at sizes that take the larger tiles; exact where there is no
    activation."""
    idx = choice("even", T, E - 1, k, T + N)
    p = permuted(idx, 0, E, tile_m, K)
    g = gen(N + K)
    x, w = packed(g, (T if gather else p.R_cap, K), 124, 127), packed(g, (E, N, K), 119, 122)
    up = packed(g, (E, N, K), 119, 122) if act == "swiglu" else None
    out, check = guarded((p.R_cap, N), F32, -7.0)
    ffi.moe_grouped_linear_mxfp4(p, on(x), on(w), w_up=on(up), act=act, gather=gather, out=out)
    check()
    src, off, cnt = (t.cpu().numpy() for t in (p.row_src, p.expert_offsets, p.expert_counts))
    rows = np.concatenate([np.arange(off[e], off[e] + cnt[e]) for e in range(E)])
    assert len(rows) == T * k and (cnt == 0).any()
    untouched = torch.ones(p.R_cap, dtype=torch.bool, device=dev())
    untouched[torch.from_numpy(rows).to(dev())] = False
    assert bool((out[untouched] == -7.0).all())
    v = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
    xv = vals(x)
    for e in range(E):
        if cnt[e] == 0:
            continue
        at = np.arange(off[e], off[e] + cnt[e])
        xe, got = v(xv[src[at] // k if gather else at]), out[off[e]:off[e] + cnt[e]].double()
        z = xe @ v(X.values(w.codes[e].numpy(), w.scales[e].numpy())).T
        if up is None:
            assert torch.equal(got, z)
        else:
            want = torch.nn.functional.silu(z) * (xe @ v(X.values(up.codes[e].numpy(), up.scales[e].numpy())).T)
            assert bool(((got - want).abs() <= 1e-6 * want.abs() + 1e-30).all())


@pytest.mark.parametrize("M", [1, 20, 70, 300])
@pytest.mark.parametrize("K", [128, 384, 1408])
def test_linear_nan_and_extreme_scales_stay_in_their_rows(M, K):
    """A row next to one whose scales are 255, or 0, or 252: at a stage's half end the next row's scales are near."""
    N = 40
    g = gen(M + K)
    x, w = packed(g, (M, K)), packed(g, (N, K))
    w.scales[1::3] = 255
    w.scales[2::3, -1] = 0
    x.scales[M // 2] = 255
    if M > 2:
        x.scales[0, 0] = 252
        x.codes[0] = 0
    out = n64(ffi.moe_linear_mxfp4(on(x), on(w), out_dtype=F32))
    ref = vals(x) @ vals(w).T
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(out), nan) and nan.any()
    tol = K * U2 * (np.abs(np.nan_to_num(vals(x))) @ np.abs(np.nan_to_num(vals(w))).T)
    assert (np.abs(out - ref)[~nan] <= tol[~nan]).all()


def test_linear_scales_from_end_to_end():
    """Products near the largest and the smallest fp32 numbers, and sums that pass it."""
    x, w = packed(gen(1), (4, 256), 127, 128), packed(gen(2), (6, 256), 127, 128)
    x.codes.fill_(0x22), w.codes.fill_(0x22)                                     # all ones
    x.scales[:], w.scales[:] = 127, 127
    w.scales[0], w.scales[1], w.scales[2] = 254, 0, 244
    x.scales[1], x.scales[2], x.scales[3] = 0, 254, 120
    out = n64(ffi.moe_linear_mxfp4(on(x), on(w), out_dtype=F32))
    ref = vals(x) @ vals(w).T
    with np.errstate(over="ignore"):
        want = ref.astype(np.float32).astype(np.float64)
    ok = np.abs(want) >= 2.0 ** -126                                             # (below, subnormal results may be flushed)
    assert np.array_equal(out[ok], want[ok])
    assert (np.abs(out[~ok]) <= 2.0 ** -126).all()


def test_linear_out_past_4_gib():
    M, N, K = 70001, 16400, 128
    g = torch.Generator(device=dev()).manual_seed(0)
    r = lambda n, k: torch.randint(0, 256, (n, k), generator=g, device=dev(), dtype=torch.int32).to(U8)  # noqa: E731
    x, w = ffi.Mxfp4(r(M, K // 2), torch.full((M, K // 32), 126, dtype=U8, device=dev())), ffi.Mxfp4(r(N, K // 2), torch.full((N, K // 32), 127, dtype=U8, device=dev()))
    out = ffi.moe_linear_mxfp4(x, w, out_dtype=F32)
    for rows in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        ref = X.values(x.codes[rows].cpu().numpy(), x.scales[rows].cpu().numpy()) @ X.values(w.codes.cpu().numpy(), w.scales.cpu().numpy()).T
        assert np.array_equal(n64(out[rows]), ref)


def test_linear_streams_graph_and_two_at_once():
    g = gen(3)
    d = dev()
    x, w = on(packed(g, (200, 512))), on(packed(g, (300, 512)))
    want = ffi.moe_linear_mxfp4(x, w, out_dtype=F32).clone()
    outs = [torch.zeros_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            ffi.moe_linear_mxfp4(x, w, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    xb = torch.randn(64, 512, device=d).to(BF)
    q, out = ffi.alloc_mxfp4(xb.shape, d), torch.empty(64, 300, device=d)
    ws = ffi.alloc_linear_mxfp4_workspace(64, 300, 512, "none", d)

    def step():
        ffi.moe_mxfp4_quantize(xb, out=q)
        ffi.moe_linear_mxfp4(q, w, out=out, ws=ws, use_workspace=False)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        xb.copy_(torch.randn(64, 512, device=d))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and float(out.abs().max()) > 0


# ---------------------------------------------------------------------------
# Grouped products
# ---------------------------------------------------------------------------

def permuted(idx, expert_begin, E_loc, tile_m, K):
    """The library's own permutation of a choice (index-only)."""
    T, k = idx.shape
    x = torch.zeros(T, K, dtype=BF, device=dev())
    p = ffi.alloc_permuted(T, K, k, E_loc, tile_m, dev(), rows=False)
    E = max(int(idx.max()) + 1, expert_begin + E_loc, k)
    return ffi.moe_permute(x, torch.from_numpy(idx).to(dev()), None, E, expert_begin, E_loc, 1, tile_m, out=p, copy_rows=False)


def choice(kind, T, E, k, seed):
    r = np.random.default_rng(seed)
    if kind == "even":
        idx = np.stack([r.permutation(E)[:k] for _ in range(T)])
    elif kind == "one":                                    # every token on the same experts, the others empty
        idx = np.tile(np.arange(k)[::-1] + (E - k) // 2, (T, 1))
    else:                                                  # few tokens have an expert at all
        idx = np.stack([r.permutation(E)[:k] for _ in range(T)])
        idx[r.random((T, k)) < 0.8] = -1
    return idx.astype(np.int32)


@pytest.mark.parametrize("tile_m", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("T,E,k,e0,El,N,K,kind,act,dt", [
    (1, 8, 2, 0, 8, 128, 128, "even", "none", F32), (37, 8, 2, 0, 8, 100, 384, "even", "none", BF),
    (300, 16, 3, 4, 8, 257, 256, "even", "swiglu", F32), (90, 12, 2, 0, 12, 64, 1408, "one", "none", F32),
    (500, 4, 2, 1, 2, 48, 640, "sparse", "gelu", BF), (65, 64, 6, 0, 64, 33, 128, "even", "swiglu", BF)])
def test_grouped(tile_m, gather, T, E, k, e0, El, N, K, kind, act, dt):
    idx = choice(kind, T, E, k, T)
    p = permuted(idx, e0, El, tile_m, K)
    g = gen(T + N)
    x = packed(g, (T if gather else p.R_cap, K), 122, 125)
    w = packed(g, (El, N, K), 119, 122)
    up = packed(g, (El, N, K), 119, 122) if act == "swiglu" else None
    out, check = guarded((p.R_cap, N), dt, -7.0)
    ffi.moe_grouped_linear_mxfp4(p, on(x), on(w), w_up=on(up), act=act, gather=gather, out=out)
    check()
    ref = O.permute(idx, None, e0, El, tile_m)
    rows = np.nonzero(ref["row_src"] >= 0)[0]
    got = n64(out)
    untouched = np.ones(p.R_cap, bool)
    untouched[rows] = False
    assert (got[untouched] == -7.0).all()
    if not len(rows):
        return
    e = np.searchsorted(ref["offsets"], rows, side="right") - 1
    xv = vals(x)[ref["row_src"][rows] // k if gather else rows]
    wv, uv = vals(w), vals(up)
    for le in np.unique(e):
        sel = e == le
        want, z, u = Q.linear(xv[sel], wv[le], None if up is None else uv[le], act_name=act)
        tol = 1.2 * bound(xv[sel], wv[le], K)
        if up is not None:
            du = bound(xv[sel], uv[le], K)
            tol = tol * (np.abs(u) + du) + np.abs(Q.act("silu", z)) * du
        tol = tol + 1e-6 * np.abs(want) + 1e-37
        if dt == BF:
            tol = tol + BF_HALF * (np.abs(want) + tol)
        assert (np.abs(got[rows[sel]] - want) <= tol).all()


def test_grouped_weights_past_4_gib():
    """The last of 72 experts begins past 2^32 bytes of codes and 2^28 of scales."""
    T, El, N, K = 40, 72, 16384, 8192
    d = dev()
    idx = np.full((T, 1), El - 1, np.int32)
    idx[::2] = 0
    p = permuted(idx, 0, El, 16, K)
    w = ffi.Mxfp4(torch.empty(El, N, K // 2, dtype=U8, device=d), torch.empty(El, N, K // 32, dtype=U8, device=d))
    for e in (0, El - 1):
        w.codes[e], w.scales[e] = 0x22 + 0x11 * (e > 0), 127                        # ones, and 1.5
    x = packed(gen(0), (T, K), 124, 126)
    out = ffi.moe_grouped_linear_mxfp4(p, on(x), w, gather=True, out_dtype=F32)
    src = p.row_src.cpu().numpy()
    sums = vals(x).sum(axis=1)
    got = n64(out[:, ::4000])
    for r in np.nonzero(src >= 0)[0]:
        assert (got[r] == sums[src[r]] * (1.5 if idx[src[r], 0] else 1.0)).all()


# ---------------------------------------------------------------------------
# The layer
# ---------------------------------------------------------------------------

def mx_inputs(cfg):
    d = W.make_inputs(cfg, dev())
    for n in ("w0", "w0_up", "w1"):
        if d[n] is not None:
            d[n] = ffi.moe_mxfp4_quantize(d[n])
    return d


def host(q):
    return X.values(q.codes.cpu().numpy(), q.scales.cpu().numpy())


@pytest.mark.parametrize("name,over", [
    ("fine_grained", dict(T=300, H=256, F=384, E=16, k=3, tile_m=128)), ("tiny", dict(T=70, H=512, F=256, E=8, k=2, tile_m=16)),
    ("ep_share", dict(T=500, H=256, F=256, E=16, k=4, E_loc=4, tile_m=256)), ("decode", dict(T=40, H=384, F=128, E=32, k=4, tile_m=16))])
@pytest.mark.parametrize("gating", [None, Gating(score="sigmoid", n_group=4, topk_group=3, group_top=2, scale=2.5)])
def test_layer_with_mxfp4_experts(name, over, gating):
    """Every step of the layer from the step before it: tokens, gate and up products, activations, down product, combine."""
    cfg = W.CONFIGS[name].with_(**over)
    d = mx_inputs(cfg)
    sh = None
    if cfg.act == "swiglu":
        r = lambda *s: ffi.moe_mxfp4_quantize(torch.randn(*s, device=dev()).mul_(0.05).to(BF))  # noqa: E731
        sh = SharedExpert(r(128, cfg.H), r(128, cfg.H), r(cfg.H, 128))
    layer = MoELayer.from_inputs(cfg, d, gating=gating, shared=sh)
    out = n64(layer.run())
    idx, gate = layer.topk_idx.cpu().numpy(), n64(layer.topk_w)
    rank = None if d["src_rank"] is None else d["src_rank"].cpu().numpy()
    ref = O.permute(idx, rank, cfg.expert_begin, cfg.n_local, cfg.tile_m)
    rows = np.nonzero(ref["row_src"] >= 0)[0]
    e = np.searchsorted(ref["offsets"], rows, side="right") - 1
    code, s = X.quantize(n64(d["x"]))
    assert np.array_equal(layer.x_q.codes.cpu().numpy(), X.pack(code)) and np.array_equal(layer.x_q.scales.cpu().numpy(), s)
    xv = X.values(X.pack(code), s)
    act, y = n64(layer.act_buf), n64(layer.y_perm)
    code, s = X.quantize(act[rows])
    assert np.array_equal(layer.act_q.codes.cpu().numpy()[rows], X.pack(code)) and np.array_equal(layer.act_q.scales.cpu().numpy()[rows], s)
    aq = X.values(X.pack(code), s)
    w0, w1 = host(d["w0"]), host(d["w1"])
    w0u = None if d["w0_up"] is None else host(d["w0_up"])
    want_y = np.zeros((ref["row_src"].shape[0], cfg.H))
    for le in np.unique(e):
        sel = e == le
        xs = xv[ref["row_src"][rows[sel]] // cfg.k]
        want, z, u = Q.linear(xs, w0[le], None if w0u is None else w0u[le], act_name=cfg.act)
        tol = 1.2 * bound(xs, w0[le], cfg.H)
        if w0u is not None:
            du = bound(xs, w0u[le], cfg.H)
            tol = tol * (np.abs(u) + du) + np.abs(Q.act("silu", z)) * du
        tol = tol + 1e-6 * np.abs(want) + 1e-37
        assert (np.abs(act[rows[sel]] - want) <= tol + BF_HALF * (np.abs(want) + tol)).all()
        want_y[rows[sel]] = aq[sel] @ w1[le].T
        assert (np.abs(y[rows[sel]] - want_y[rows[sel]]) <= bound(aq[sel], w1[le], cfg.F_loc)).all()
    inv = ref["inv_perm"]
    total = np.where(inv[..., None] >= 0, gate[..., None] * y[np.maximum(inv, 0)], 0.0)
    want, mag = total.sum(axis=1), np.abs(total).sum(axis=1)
    if sh is not None:
        h = host(layer.shared_q)
        part = h @ host(sh.w1).T
        want, mag = want + part, mag + np.abs(part) + 128 * (np.abs(h) @ np.abs(host(sh.w1)).T)
    assert (np.abs(out - want) <= (cfg.k + 3) * U2 * mag + 1e-30).all()

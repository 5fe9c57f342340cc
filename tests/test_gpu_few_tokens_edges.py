"""The layer for a few tokens on the GPU where its weights, scales and logits are at their ends; tolerances as in
test_gpu_few_tokens."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi
from oracle import mxfp4_oracle as X

import test_gpu_few_tokens as F

pytestmark = pytest.mark.gpu

BF, U8 = torch.bfloat16, torch.uint8
INF = float("inf")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 3, 30])
@pytest.mark.parametrize("scale", [1.0, -1.0, 1.0 + 2.0 ** -20])
def test_infinite_weights_of_the_second_product(T, mx, scale):
    """Infinity times a nonzero activation is an infinity, also where the activation has few bits (128 exactly), and NaN
    only beside a zero one; in MXFP4, values past bf16's largest count as infinities."""
    d = F.dev()
    w0, w1 = torch.zeros(1, 128, 128), torch.zeros(1, 128, 128)
    w0[0, :64] = 1.0                       # z = 128: gelu(z) = 128; the other half of the activations is zero
    w1[0, 5, 9], w1[0, 6, 33] = INF, -INF
    w1[0, 7, 70] = INF                     # beside a zero activation
    w1[0, 8, :] = 1.0
    if mx:
        codes, s = X.quantize(np.nan_to_num(w1.double().numpy(), posinf=0.0, neginf=0.0))
        codes[0, 5, 9], codes[0, 6, 33], codes[0, 7, 70] = 7, 15, 7
        s[0, 5, 0] = s[0, 6, 1] = s[0, 7, 2] = 254
        w1 = ffi.Mxfp4(torch.from_numpy(X.pack(codes)).to(d), torch.from_numpy(s).to(d))
        w0 = ffi.moe_mxfp4_quantize(w0.to(BF).to(d))
    else:
        w0, w1 = w0.to(BF).to(d), w1.to(BF).to(d)
    x = torch.ones(T, 128, dtype=BF, device=d)
    out = F.n64(ffi.moe_few_tokens(x, w0, None, w1, "gelu", topk_idx=torch.zeros(T, 1, dtype=torch.int32, device=d),
                                   topk_w=torch.full((T, 1), scale, device=d)))
    sign = np.sign(scale)
    assert (out[:, 5] == sign * INF).all() and (out[:, 6] == -sign * INF).all()
    assert np.isnan(out[:, 7]).all()
    np.testing.assert_allclose(out[:, 8], 64 * 128 * scale, rtol=65 * 2.0 ** -23)
    rest = np.delete(out, [5, 6, 7, 8], axis=1)
    assert (rest == 0).all()


@pytest.mark.parametrize("T", [1, 4, 32])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_scale_bytes_from_end_to_end(T, act):
    """Blocks of codes under the bytes 0, 1, 252 and 254, brought to one size by the tokens and by the gate weights."""
    g = F.gen(T)
    E, H, K = 4, 128, 128
    ends = np.array([0, 1, 252, 254])
    w = F.Experts(g, E, H, K, act, True)

    def redo(q, byte):  # byte [..., blocks]; under 254 codes up to 1.5, the largest that bf16 holds
        c = torch.randint(0, 16, q.shape, generator=g).numpy()
        c = np.where(np.repeat(byte, 32, axis=-1) == 254, c & 11, c)
        q.codes.copy_(torch.from_numpy(X.pack(c)))
        q.scales.copy_(torch.from_numpy(byte.astype(np.uint8)))
    for q in w.t[:2]:
        if q is not None:
            redo(q, np.broadcast_to(ends, (E, K, 4)))
    redo(w.t[2], np.broadcast_to(ends[:, None, None], (E, H, 4)))   # one byte an expert
    x = torch.randn(T, H, generator=g).sign().double() * torch.from_numpy(np.exp2(np.minimum(127.0 - ends, 127.0).clip(-126.0)).repeat(32))
    x = x.to(BF)
    idx = (torch.arange(T, dtype=torch.int32) % E)[:, None]
    for first in range(E if T == 1 else 1):
        e = (idx + first) % E
        gate = torch.from_numpy(np.array([2.0 ** 100, 2.0 ** 100, 2.0 ** -100, 2.0 ** -100]))[e.long()].float()
        out, i2, g2 = F.run(x, w, idx=e.to(torch.int32), gate=gate, num_experts=E)
        ref = F.check_out(out, x, i2, g2, w, E, norm=False)
        assert (np.linalg.norm(out - ref, axis=1) <= 2e-5 * np.linalg.norm(ref, axis=1)).all() and (np.abs(ref) > 0).any(axis=1).all()


@pytest.mark.parametrize("T", [1, 4, 32])
@pytest.mark.parametrize("byte,code,value", [(252, 7, 6 * 2.0 ** 125), (253, 5, 3 * 2.0 ** 126), (253, 6, INF), (253, 7, INF), (254, 3, 1.5 * 2.0 ** 127),
                                             (254, 4, INF), (254, 15, -INF)])
def test_values_at_and_past_the_largest_bf16(T, byte, code, value):
    """MXFP4 values past bf16's largest are infinities in both products, as read back."""
    d = F.dev()
    one = lambda: X.quantize(np.ones((1, 128, 128)))  # noqa: E731
    for which in (0, 1):
        q = [one(), one()]
        q[which][0][0, 3, 40], q[which][1][0, 3, 1] = code, byte
        q[which][0][0, 3, 32:40] = q[which][0][0, 3, 41:64] = 0
        w0, w1 = (ffi.Mxfp4(torch.from_numpy(X.pack(c)).to(d), torch.from_numpy(s).to(d)) for c, s in q)
        assert F.n64(ffi.moe_mxfp4_dequantize((w0, w1)[which]))[0, 3, 40] == value
        x, scale = torch.zeros(T, 128, dtype=BF, device=d), 1.0
        if which == 0:  # z[3] = 768 or infinite, gelu(z) = z (of -inf: NaN); the others vanish beside it
            x[:, 40] = 2.0 ** -118
            want = np.full(128, value * 2.0 ** -118 if value > 0 else np.nan)
        else:           # every activation is 128 2^-100
            x[:], scale = 1.0, 2.0 ** -100
            want = np.full(128, 128.0 * 128 * scale)
            want[3] = (96 + value) * 128 * scale
        out = F.n64(ffi.moe_few_tokens(x, w0, None, w1, "gelu", topk_idx=torch.zeros(T, 1, dtype=torch.int32, device=d),
                                       topk_w=torch.full((T, 1), scale, device=d)))
        np.testing.assert_allclose(out, np.broadcast_to(want, out.shape), rtol=130 * 2.0 ** -23)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("renorm", [True, False])
def test_masks_and_ties_in_small_calls(n, renorm):
    """Rows that leave slots empty, ties and infinities, n tokens a call: routed by one wavefront, by the workgroups of the
    first launch, or by a launch of their own."""
    E, k, T = 24, 4, 12
    g = F.gen(n)
    w = F.Experts(g, E, 128, 128, "swiglu", False)
    x = torch.randn(T, 128, generator=g).to(BF)
    l = torch.randn(T, E, generator=g)
    l[0] = -INF
    l[1] = float("nan")
    l[2, 2:] = -INF
    l[3, ::2] = float("nan")
    l[4] = torch.finfo(torch.float32).min
    l[5, 3:] = torch.finfo(torch.float32).min
    l[6, 20] = l[6, 7] = INF
    l[7] = 0.25
    l[8] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0)
    l[9] = l[9].round()
    l[10, :] = -INF
    l[10, 23] = -1000.0
    ridx, rw = X.route(l.numpy(), k, renorm)
    for t in range(0, T, n):
        rows = slice(t, t + n)
        out, idx, gate = F.run(x[rows], w, l[rows].contiguous(), k, renormalize=renorm)
        assert np.array_equal(idx, ridx[rows])
        np.testing.assert_allclose(gate, rw[rows], rtol=4e-6, atol=1e-37)
        F.check_out(out, x[rows], idx, gate, w, E)
        assert (out[(idx < 0).all(axis=1)] == 0).all()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 2, 4, 9, 64])
@pytest.mark.parametrize("e0,El", [(0, 3), (9, 7)])
def test_a_share_with_logits_over_all_experts(T, e0, El, mx):
    """Tokens routed here over every expert, of which a few are local."""
    g = F.gen(T + e0)
    E, k = 16, 5
    w = F.Experts(g, El, 256, 128, "swiglu", mx)
    x = torch.randn(T, 256, generator=g).to(BF)
    l = torch.randn(T, E, generator=g)
    l[T // 2, e0:e0 + El] = -20.0                       # no local expert
    out, idx, gate = F.run(x, w, l, k, expert_begin=e0, num_experts=E)
    ridx, rw = X.route(l.numpy(), k, True)
    assert np.array_equal(idx, ridx)
    np.testing.assert_allclose(gate, rw, rtol=4e-6, atol=1e-37)
    F.check_out(out, x, idx, gate, w, El, e0)
    assert (out[T // 2] == 0).all()


def test_arguments_that_contradict_one_another():
    d = F.dev()
    w = F.Experts(F.gen(0), 4, 128, 128, "swiglu", False)
    x, l = torch.randn(3, 128, device=d).to(BF), torch.randn(3, 8, device=d)
    idx, gate = ffi.moe_route_topk(l, 2)
    for bad in (dict(logits=l, k=2, num_experts=9), dict(logits=l, k=2, num_experts=4), dict(logits=l, k=3, topk_idx=idx),
                dict(topk_idx=idx, topk_w=gate, k=3), dict(topk_idx=idx, topk_w=gate, k=1)):
        with pytest.raises(ValueError):
            ffi.moe_few_tokens(x, *w.t, "swiglu", **bad)
    a = ffi.moe_few_tokens(x, *w.t, "swiglu", logits=l, k=2, num_experts=8)
    b = ffi.moe_few_tokens(x, *w.t, "swiglu", topk_idx=idx, topk_w=gate, k=2, num_experts=8)
    torch.testing.assert_close(a, b, rtol=1e-4, atol=1e-6)

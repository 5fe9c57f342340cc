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

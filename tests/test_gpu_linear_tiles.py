"""GELU and SiLU in the dense projection's epilogue on every tile, split over the reduction or not, against fp64.

Tolerances (u = 2^-24): z is an fp32 sum of K exact products in any order, within (K + 2) 2u of the sum of their absolute
values (u doubled, in case the matrix unit truncates); the activation adds 1e-6 of its result (erf, hardware exp2 and
reciprocal, a few u each) and 2e-7 |z| (GELU's 1 + erf cancels for negative z: u of 1 each from erf, its argument and the
sum, times |z| / 2), and passes an error of z on by at most 1.2; the residual adds 2u; a bf16 output is within 2^-8 of itself.
"""
import pytest
import torch

from mixture_experts_layer_moe_amd import ffi

import parity_helpers as P
from linear_tile_cases import CASES

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("M,N,K,kind,slices,streamed", CASES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("odt", [BF, F32])
def test_activations_on_every_tile(M, N, K, kind, slices, streamed, act, odt):
    d = P.require_gpu()
    if torch.cuda.get_device_properties(d).multi_processor_count == 256:
        assert (ffi.linear_workspace_bytes(M, N, K, act) > 0) == (slices > 1)
    g = torch.Generator(device=d).manual_seed(M + N + K)
    r = lambda *s: torch.randn(*s, device=d, generator=g)  # noqa: E731
    x, w = r(M, K).to(BF), (r(N, K) * 2 / K ** 0.5).to(BF)
    b, res = r(N), r(M, N).to(odt)
    out, z = torch.full((M, N), 99.0, dtype=odt, device=d), torch.full((M, N), 99.0, dtype=BF, device=d)
    ffi.moe_linear(x, w, bias=b, act=act, residual=res, out=out, z=z)
    X, W = x.double(), w.double()
    ref_z = torch.mm(X, W.T.contiguous()) + b
    zb = (K + 2) * 2 * U * (torch.mm(X.abs(), W.abs().T.contiguous()) + b.abs())
    y = ref_z * (0.5 * torch.erfc(-ref_z / 2 ** 0.5) if act == "gelu" else torch.sigmoid(ref_z))
    ref = y + res.double()
    bound = 1.2 * zb + 1e-6 * y.abs() + 2e-7 * ref_z.abs() + 2 * U * (ref.abs() + res.double().abs())
    half = 2.0 ** -8 if odt is BF else 0.0
    assert bool(((out.double() - ref).abs() <= bound * 1.01 + half * ref.abs()).all())
    assert bool(((z.double() - ref_z).abs() <= zb * 1.01 + 2.0 ** -8 * ref_z.abs()).all())
    again = torch.empty_like(out)
    ffi.moe_linear(x, w, bias=b, act=act, residual=res, out=again)
    assert torch.equal(again, out)

"""Sizes that no launch takes are refused on the host, before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

from mixture_experts_layer_moe_amd import ffi

UNSUPPORTED = 2
NULL = None
FAKE = ctypes.c_void_p(16 * 1024)   # aligned, never dereferenced: validation fails first


def test_permute_of_more_tokens_than_one_launch_takes():
    for T in ((1 << 26) - 15, 1 << 26, (1 << 26) + 70):
        args = [FAKE, FAKE, NULL, T, 8, 1, 8, 0, 8, 1, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
        assert ffi.lib().moe_permute(*args, FAKE, 1 << 40, NULL) == UNSUPPORTED
        assert ffi.lib().moe_permute_noalloc(*args, NULL) == UNSUPPORTED


FAR = [ctypes.c_void_p(p << 56) for p in (1, 2, 3, 4)]  # sizes here pass 2^48 bytes


@pytest.mark.parametrize("M,N,K,act", [((1 << 31) - 1, 1, 8, 2), ((1 << 31) - 1, 1024, 8, 0), ((1 << 31) - 20, 130, 8, 1),
                                       (1 << 28, 1 << 20, 64, 2)])
def test_linear_of_more_tiles_than_one_launch_takes(M, N, K, act):
    up = FAKE if act == 1 else NULL
    w, out = FAR[:2]
    assert ffi.lib().moe_linear(FAKE, w, up, NULL, NULL, NULL, M, N, K, act, 0, NULL, NULL, out, NULL, 0, NULL) == UNSUPPORTED
    assert ffi.lib().moe_linear_workspace_bytes(M, N, K, act) == 0


@pytest.mark.parametrize("M,N,K,act", [((1 << 31) - 1, 1, 8, 2), ((1 << 31) - 1, 8, 1024, 0), (1 << 28, 130, 1 << 20, 1),
                                       (1, 1 << 20, 1 << 20, 2)])
def test_linear_backward_of_more_tiles_than_one_launch_takes(M, N, K, act):
    w, g, d_x, ws = FAR
    up, z, z_up = FAKE if act == 1 else NULL, FAKE if act != 2 else NULL, FAKE if act == 1 else NULL
    args = [g, FAKE, w, up, z, z_up, M, N, K, act, 0, d_x, NULL, NULL, NULL, NULL]
    assert ffi.lib().moe_linear_backward(*args, ws, 1 << 55, NULL) == UNSUPPORTED

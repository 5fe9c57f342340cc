"""Sizes that no launch takes are refused on the host, before anything is enqueued (no GPU needed)."""
import ctypes

from mixture_experts_layer_moe_amd import ffi

UNSUPPORTED = 2
NULL = None
FAKE = ctypes.c_void_p(16 * 1024)   # aligned, never dereferenced: validation fails first


def test_permute_of_more_tokens_than_one_launch_takes():
    for T in ((1 << 26) - 15, 1 << 26, (1 << 26) + 70):
        args = [FAKE, FAKE, NULL, T, 8, 1, 8, 0, 8, 1, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
        assert ffi.lib().moe_permute(*args, FAKE, 1 << 40, NULL) == UNSUPPORTED
        assert ffi.lib().moe_permute_noalloc(*args, NULL) == UNSUPPORTED

"""Limits of the 4-bit operators' calls without a GPU; no library call here reaches a kernel launch."""
from test_mxfp4_cpu import L, UNSUPPORTED, dequantize  # noqa: F401


def test_dequantize_to_fp32_stays_below_two_to_the_32_threads(L):  # noqa: F811
    """Four values a thread and four units: 2^36 values are 2^24 workgroups of 256, one thread more than a grid can hold."""
    assert dequantize(L, R=1 << 31, K=32, dt=1) == UNSUPPORTED
    assert dequantize(L, R=(1 << 31) - 127, K=32, dt=1) == UNSUPPORTED
    assert dequantize(L, R=(1 << 31) + 1, K=32, dt=0) == UNSUPPORTED

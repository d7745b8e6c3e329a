"""Largest sizes of bfp8_attn_latent: products with the heads are held to their limit, not factors to its quotient."""
import ctypes

import pytest

from block_scaled_fp8_04_amd import _lib

FAKE = ctypes.c_void_p(0x10000)


def status(T, max_new, heads):
    """Without a query: a size that is allowed is refused for that alone, before any HIP call."""
    return _lib.library().bfp8_attn_latent(
        None, 0, 0, FAKE, 0, 0, FAKE, FAKE, FAKE, 8, 64, FAKE, 4, FAKE, FAKE, 2, T, max_new, heads, 1.0, FAKE, 512, 512,
        None, None, 0, None)


@pytest.mark.parametrize("heads", [1, 2, 3, 7, 16, 100, 128, 65535])
def test_products_up_to_their_limit(heads):
    last = (2 ** 29 - 1) // heads
    assert status(last, 1, heads) == _lib.BFP8_ERR_NULL
    assert status(last + 1, 1, heads) == _lib.BFP8_ERR_SHAPE
    last = (2 ** 31 - 1) // heads
    assert status(1, last, heads) == _lib.BFP8_ERR_NULL
    assert status(1, last + 1, heads) == _lib.BFP8_ERR_SHAPE


def test_factors_far_past_the_limit():
    for huge in (2 ** 31, 2 ** 32, 2 ** 61, 2 ** 63 - 1):
        assert status(huge, 1, 8) == status(1, huge, 8) == _lib.BFP8_ERR_SHAPE

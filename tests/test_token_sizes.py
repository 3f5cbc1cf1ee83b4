"""Sizes past what the token calls take (no GPU: refused before anything is launched)."""
import pytest

import block_scaled_fp8_grouped_amd as bs

P, SHAPE = 1 << 20, -4  # an address that nothing reads


@pytest.mark.parametrize("tokens,cols", [(1 << 22, 8192), (1 << 23, 3500), (1 << 29, 33), (1 << 30, 32)])
def test_rows_past_a_launch_are_refused(tokens, cols):
    """2^35 elements, a row's rounded up to whole 1024s, or below to 8 times a power of two."""
    lib = bs.lib()
    assert lib.bsfp8_dispatch(P, bs.BF16, tokens, cols, P, 1, None, P, 8, None) == SHAPE
    assert lib.bsfp8_combine(P, bs.BF16, 8, cols, P, tokens, 1, None, None, P, None) == SHAPE

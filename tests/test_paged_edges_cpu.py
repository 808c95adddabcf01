"""Paged cache and log probabilities without a GPU: launches at the ends of 32 bits (every call
here returns before a launch)."""
import ctypes

import pytest

FAKE = 4096  # never dereferenced


@pytest.fixture(scope="module")
def ft():
    from int4_weight_kv_gb300 import build as b
    b.build()
    import int4_weight_kv_gb300 as m
    return m


def test_attention_grids_past_32_bits_are_refused(ft):
    """More CTAs than a launch may have, in the joining kernel of few rows and the kernel of many: refused before any launch."""
    lib, n = ft.lib(), 43690
    c = ft.make_cfg(512, n, n, 64, 512)
    call = lambda B, total, max_q: lib.ft_attn_paged_int4(  # noqa: E731
        ctypes.byref(c), FAKE, 8, 16, FAKE, n * 64, FAKE, FAKE, FAKE, 1, B, total, max_q, 0.1, FAKE, n * 64, FAKE, 2 ** 60, None, None)
    assert call(8192, 8192, 20) == ft.FT_ERR_UNSUPPORTED
    assert call(1, 2 ** 30, 2 ** 30) == ft.FT_ERR_UNSUPPORTED

"""Shapes that the decode calls accept, by their host checks (CPU only): a call with no workspace is refused for that, and
not as a shape without a kernel, wherever there is one."""
import ctypes

import pytest

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import _lib

FAKE = 1 << 20  # never dereferenced: every call below fails host validation first
UNSUPPORTED, WORKSPACE = 3, 4


def answer(call, heads, T, D, P):
    pool = _lib.nk_kv_pool(FAKE, 16, P, 1, D)
    return getattr(nk.lib(), call)(ctypes.byref(pool), FAKE, FAKE, 4, FAKE, 1, T, heads, 0.1, 4 * P, 0, FAKE, 0, FAKE, None,
                                   None)


@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_fp16_scales_at_head_dim_256_on_128_key_pages(T):
    """33 to 40 rows leave two stages of 128-key pages, to within some hundred bytes of shared memory."""
    for heads in range(1, 41):
        assert answer("nk_i8f16_decode_attn", heads, T, 256, 128) == WORKSPACE, heads
    assert answer("nk_i8f16_decode_attn", 41, T, 256, 128) == UNSUPPORTED  # (six tiles of rows: one stage)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("call", ["nk_paged_decode_attn", "nk_i8f16_decode_attn"])
def test_up_to_48_heads_on_pages_of_up_to_64_keys(call, D):
    for P in (16, 32, 48, 64):
        for heads in (1, 8, 24, 32, 33, 40, 48):
            assert answer(call, heads, 1, D, P) == WORKSPACE, (P, heads)

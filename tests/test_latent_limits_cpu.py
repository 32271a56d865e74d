"""Sizes past the limits of the latent cache's calls and of page allocation, which a 32-bit count in a kernel would pass, are
refused before any CUDA call."""
import ctypes

import pytest

import flash_attention_forward_gb300 as fa
from flash_attention_forward_gb300 import build as libbuild

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation
F, SZ, I64 = ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
PAST = [(1 << 30) + 1, (1 << 31) - 1000, (1 << 31) - 1]


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return fa.library()


@pytest.mark.parametrize("n", PAST)
def test_page_allocation(lib, n):
    def call(B, total):
        return lib.sdpa_cache_resize(*[FAKE] * 10, B, total, 64, 64, 100, I64(64), FAKE, SZ(1 << 40), None)
    assert call(2, n) == call(n, 2) == fa.SDPA_ERR_UNSUPPORTED
    assert fa.sdpa_cache_resize_workspace_size(2, n, 64) == fa.sdpa_cache_resize_workspace_size(n, 2, 64) == 0
    assert fa.sdpa_cache_resize_workspace_size(2, 1 << 30, 64) == 3 * 16


@pytest.mark.parametrize("n", PAST)
def test_latent_write(lib, n):
    assert lib.sdpa_latent_write(*[FAKE] * 6, n, 64, 4, 512, 64, 0, F(1.0), None, fa.SDPA_BF16, None) == fa.SDPA_ERR_UNSUPPORTED


@pytest.mark.parametrize("n", PAST)
@pytest.mark.parametrize("Hq", [1, 128])
def test_attention(lib, n, Hq):
    def absorbed(B, total):
        return lib.sdpa_fwd_latent_paged(*[FAKE] * 6, None, B, Hq, total, 1, 64, 8, 20, 512, 64, None, F(0.1), 1, FAKE, SZ(1 << 62),
                                         fa.SDPA_BF16, None)

    def expanded(B, total, total_k=20):
        return lib.sdpa_fwd_latent(*[FAKE] * 7, None, B, Hq, 1, total, total_k, 1, 128, 64, 128, None, F(0.1), 1, FAKE, SZ(1 << 62),
                                   fa.SDPA_BF16, None)
    assert absorbed(2, n) == absorbed(n, 2) == expanded(2, n) == expanded(n, 2) == expanded(2, 2, n) == fa.SDPA_ERR_UNSUPPORTED
    assert fa.sdpa_fwd_latent_paged_workspace_size(2, Hq, n, 1, 512) == fa.sdpa_fwd_latent_paged_workspace_size(n, Hq, 2, 1, 512) == 0
    assert fa.sdpa_fwd_latent_workspace_size(2, Hq, 1, n, 1, 20) == fa.sdpa_fwd_latent_workspace_size(n, Hq, 1, 2, 1, 20) == 0


@pytest.mark.parametrize("n", PAST)
def test_rope_of_too_many_heads(lib, n):
    def call(Hq, Hk):
        return lib.sdpa_rope(*[FAKE] * 6, 1, Hq, Hk, 16, 16, 0, F(1.0), None, fa.SDPA_BF16, None)
    assert call(n, 1) == call(1, n) == call(1 << 30, 1) == fa.SDPA_ERR_UNSUPPORTED


def test_rope_of_too_many_units(lib):
    # 2^27 tokens of 16 units: 2^31; half pairs are two vectors a unit, and what is not turned is left alone in place
    def call(total, rot, inter):
        return lib.sdpa_rope(FAKE, None, FAKE, None, FAKE, FAKE, total, 1, 0, 128, rot, inter, F(1.0), None, fa.SDPA_BF16, None)
    assert call(1 << 27, 128, 1) == call(1 << 28, 128, 0) == call((1 << 31) - 1, 16, 1) == fa.SDPA_ERR_UNSUPPORTED

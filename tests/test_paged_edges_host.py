"""CPU: refusals at the ends of what the paged cache's calls take."""
import ctypes

import pytest

from bit_fp8_attention_means_gb300 import build, vc

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    build.build()
    return vc.lib()


def attn(L, scale=0.0):
    cache = vc.VcCacheShape(10, 16, 2, 128, 2 * 16 * 128, 16 * 128, 128, 32, 16)
    batch = vc.VcBatch(0x10000, 0x10000, 0x10000, 3, 7, 4, 4)
    return L.vc_attn_paged(FAKE, 512, 128, 4, cache, FAKE, FAKE, FAKE, FAKE, batch, scale, 1, 0, 0, FAKE, 512, 128, FAKE,
                           None, 0, None, None)


def test_softmax_scale_beyond_fp32_in_log2_units(L):
    assert attn(L) == attn(L, 2.3e38) == 3     # as far as the workspace, which is not there
    for scale in (2.4e38, 3.4e38):
        assert attn(L, scale) == 1, scale


def test_timeout_hook_refusals(L):
    cache = vc.VcCacheShape(10, 16, 2, 128, 2 * 16 * 128, 16 * 128, 128, 32, 16)
    batch = vc.VcBatch(0x10000, 0x10000, 0x10000, 3, 7, 4, 4)

    def call(status=FAKE, skip=0, heads=4, ws=None):
        return L.vc_debug_attn_paged_timeout(FAKE, 512, 128, heads, cache, FAKE, FAKE, FAKE, FAKE, batch, 0, FAKE, 512, 128,
                                             ws, 0, status, None, skip)
    assert call() == 3                         # as far as the workspace
    for kw in (dict(status=None), dict(skip=-1), dict(heads=3)):
        assert call(**kw) == 1, kw

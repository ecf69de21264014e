"""CPU: what the test hooks of the shared passes refuse before any launch."""
import ctypes

import pytest

from bit_fp8_attention_means_gb300 import build, vc
from test_rope_pages_host import FAKE, batch, cache


@pytest.fixture(scope="module")
def L():
    build.build()
    return vc.lib()


def test_shared_timeout_hook_refusals(L):
    def call(skip_pass=1, skip_unit=0, status=FAKE, groups=FAKE, N=2, ws=FAKE, b=batch()):
        return L.vc_debug_attn_paged_shared_timeout(FAKE, 512, 128, 4, cache(), FAKE, FAKE, FAKE, FAKE, b, groups, FAKE, N, 0, 0, FAKE, 512, 128, FAKE, ws, 1 << 40,
                                                    status, None, skip_pass, skip_unit)
    for bad in (dict(skip_pass=0), dict(skip_pass=3), dict(skip_unit=-1), dict(status=None), dict(groups=None), dict(N=-1), dict(b=batch(B=0)), dict(N=0)):
        assert call(**bad) == 1, bad
    assert call() == 1                         # so small a call takes one pass
    assert call(ws=ctypes.c_void_p(0x10080)) == 3

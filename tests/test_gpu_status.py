"""GPU: a status word that several calls share: the largest number stays, and a timeout beside a refused reservation."""
import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from test_gpu_pages import DEV, Device, ints
from pool_model import Model

pytestmark = pytest.mark.gpu
INVALID, TIMEOUT, PAGES = 1, 5, 6


def refused(status):
    """A reservation of more pages than there are."""
    m = Model(2, 16, 1, 4)
    dev = Device(m)
    vc.vc_pages_reserve(dev.cache, dev.pool, ints([0, 40]), ints([40]), dev.table, 40, dev_status=status)


def invalid(status):
    """A copy of a page that is not there."""
    dev = Device(Model(2, 16, 1, 4))
    vc.vc_cache_copy(dev.cache, dev.cache, ints([5]), ints([1]), dev_status=status)


def timeout(status):
    """A bounded wait that runs out."""
    vc.vc_debug_wait_timeout(status, 1000)


@pytest.mark.parametrize("calls,left", [((timeout, refused), TIMEOUT), ((invalid, refused), PAGES), ((refused, invalid), PAGES), ((invalid, timeout), TIMEOUT),
                                        ((timeout, invalid), TIMEOUT), ((refused,), PAGES), ((invalid,), INVALID), ((invalid, timeout, refused, invalid), TIMEOUT)],
                         ids=lambda x: "_".join(f.__name__ for f in x) if isinstance(x, tuple) else str(x))
def test_a_refused_reservation_replaces_no_timeout(calls, left):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in calls:
        call(status)
    assert int(status) == left

"""GPU: page calls (vc_pages_*) on tables that break a pool's rules: equal to the calls on lists (pool_model.py) but
for what is reported."""
import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from test_gpu_pages import DEV, Device, grown

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [0, 1, 3, 255])
def test_compacting_gives_a_free_page_no_second_owner(fill):
    """Entries that name free pages into which others are moved: reported, and -1 afterwards, whatever lies in the
    workspace; nothing else differs, and what is ended later takes no page from its owner."""
    for hole in (0, 3, 6):
        m = grown(seed=8)
        m.trim([0, -1, -1, -1, -1, -1])                          # pages 0 .. 6: all of them are moved into
        used = sum(r > 0 for r in m.refs)
        assert hole < used and not m.refs[hole]
        dev = Device(m)
        dev.table[0, 0], dev.table[3, 1], dev.table[1, 7] = hole, -2 - hole, hole
        ws = torch.full((8 * m.pages + 8,), fill, dtype=torch.uint8, device=DEV)
        assert int(vc.vc_pages_compact(dev.cache, dev.pool, dev.table, workspace=ws, dev_status=dev.status)) == m.compact() == used
        dev.same(m, 1)
        dev.trim([0, -1, -1, 0, -1, -1])
        m.trim([0, -1, -1, 0, -1, -1])
        dev.same(m)

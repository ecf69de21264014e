"""GPU: attention over shared prefixes where a group's sequences end, waits run out, strides are wide: against the
definition of attention in fp64 (paged_case.py), with its bars."""
import pytest
import torch

from shared_case import Shared
from test_gpu_shared import attend

pytestmark = pytest.mark.gpu

ENDED = {  # groups, and the sequences that ended
    "first": (dict(groups=[(777, [(3, 0), (5, 1), (300, 2), (2, 1)])], H=2, G=4, page=32), [0]),
    "first_three": (dict(groups=[(40, [(1, 0), (9, 0), (3, 0), (7, 3), (1, 1)])], H=1, d=64), [0, 1, 2]),
    "between": (dict(groups=[(500, [(7, 1), (9, 0), (9, 0), (3, 2)])], H=2, G=2), [1, 2]),
    "of_several": (dict(groups=[(1000, [(20, 0), (9, 4)]), (129, [(200, 0)] * 3 + [(200, 7)] * 2), (2000, [(1, 0)] * 9 + [(1, 1)] * 20)], H=2, G=3, page=64), [0, 2, 3, 4, *range(7, 16)]),
    "all_of_one": (dict(groups=[(64, [(3, 0), (4, 0)]), (300, [(8, 0), (6, 2), (2, 2)])], H=1, G=2), [0, 1, 2]),
    "chunks": (dict(groups=[(400, [(130, 0), (200, 90), (130, 130)]), (33, [(9, 0), (300, 300)])], H=1, G=2, page=128), [0, 3]),
    "behind_others": (dict(before=[(300, 2), (50, 0)], groups=[(64, [(10, 0), (3, 3), (4, 4)])], H=2, G=4, d=64, tail=5), [2]),
    "many": (dict(groups=[(300, [(20, 0)] * 70 + [(20, 3)] * 30)], H=1, G=2, page=64), list(range(70))),
}


def ended(kw, who, seed=1):
    """The batch after vc_pages_trim of the sequences `who`: no tokens, no pages."""
    c = Shared(seed=seed, **kw)
    assert all(c.n[b] == 0 for b in who)
    for b in who:
        c.kv[b] = 0
        c.kv_len[b] = 0
        c.table[b] = -1
    return c


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("case", ENDED)
def test_sequences_of_a_group_that_have_ended(case, wide):
    """The others' prefix is found without them, in two passes and in one."""
    c = ended(*ENDED[case])
    c.check(attend(c, wide=wide), c.cache())
    for hints in ((1, 1), (33, 300), (300, 5000)):
        c.check(attend(c, wide=wide, max_q=hints[0], max_rows=hints[1]), c.cache())

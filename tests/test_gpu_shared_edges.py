"""GPU: attention over shared prefixes where a group's sequences end, waits run out, strides are wide: against the
definition of attention in fp64 (paged_case.py), with its bars."""
import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from shared_case import Shared
from test_gpu_shared import DEV, attend, tables

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


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("prefix", [0, 5000, 2 ** 31 - 1, -1, -2 ** 31])
def test_groups_without_tokens_have_any_prefix(prefix, wide):
    """Groups without sequences, and such whose sequences all ended: their prefix is not looked at, and nothing is
    reported."""
    c = ended(dict(groups=[(200, [(9, 1), (3, 2)]), (0, []), (0, [(1, 0), (2, 0)]), (90, [(5, 5)]), (0, [])], H=2, G=2), [2, 3])
    c.prefix = [c.prefix[0], prefix, prefix, c.prefix[3], prefix]
    c.check(attend(c, wide=wide), c.cache())


LOST = {  # groups, hints that choose the tiles of both passes
    "few_few": (dict(groups=[(5000, [(300, 1)] * 12)], H=8, G=1, d=64, page=64), 1, 8),
    "many_few": (dict(groups=[(5000, [(600, 2)] * 20)], H=8, G=4, page=16, tail=3), 2, 64),
    "many_many": (dict(groups=[(4000, [(700, 70)] * 4), (900, [(500, 70)] * 3)], H=8, G=1, page=128), 70, 300),
    "many_many_of_d_64": (dict(groups=[(4000, [(700, 70)] * 4), (900, [(500, 70)] * 3)], H=8, G=1, d=64, page=128), 70, 300),
    "many_short": (dict(groups=[(3000, [(400, 70)] * 5)], H=8, G=1, page=32), 70, 100),
}


@pytest.mark.parametrize("skip_pass,skip_unit", [(1, 0), (2, 0), (1, 1)])
@pytest.mark.parametrize("case", LOST)
def test_wait_timeout_and_recovery(case, skip_pass, skip_unit):
    """Loaders that leave out a unit's keys: the wait for them runs out and is recorded, both passes end, every row of the
    call says that it is none, and the next call with the same workspace is right."""
    kw, max_q, max_rows = LOST[case]
    c = Shared(seed=20, **kw)
    Q, cache, args, groups = c.Q.to(DEV), c.cache(DEV), tables(c, True), c.shared_args(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.zeros(vc.attn_paged_shared_workspace_bytes(cache, c.H * c.G, c.B, c.T, len(c.prefix), max_q, max_rows), dtype=torch.uint8, device=DEV)
    hints = dict(max_q=max_q, max_rows=max_rows, workspace=ws)
    c.check(vc.vc_attn_paged_shared(Q, cache, *args, *groups, dev_status=status, **hints), c.cache())
    assert int(status) == 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    O, lse = vc.vc_debug_attn_paged_shared_timeout(Q, cache, *args, *groups, status, skip_pass, skip_unit, **hints)
    end.record()
    torch.cuda.synchronize()
    assert int(status) == 5
    # 2^16 attempts of 3.7 us, or twice that where something in flight never arrives
    assert start.elapsed_time(end) < 1000
    assert torch.isnan(O[:sum(c.n)]).all() and torch.isnan(lse[:sum(c.n)]).all()
    status.zero_()
    c.check(vc.vc_attn_paged_shared(Q, cache, *args, *groups, dev_status=status, **hints), c.cache())
    assert int(status) == 0


def test_the_hook_is_for_two_passes():
    c = Shared([(40, [(1, 1)] * 3)], H=1, d=64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(vc.VcError):
        vc.vc_debug_attn_paged_shared_timeout(c.Q.to(DEV), c.cache(DEV), *c.args(DEV), *c.shared_args(DEV), status, 1, 0)
    assert int(status) == 0

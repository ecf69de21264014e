"""GPU: the pages of a cache (vc_pages_*, vc_cache_copy) against the calls on lists (pool_model.py): equal in every
number and every byte."""
import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import Case
from pool_model import Model, rng_of, walk

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def offsets(n):
    return ints([sum(n[:i]) for i in range(len(n) + 1)])


class Device:
    """The state of a model on the GPU."""

    def __init__(self, m):
        self.cache = {k: v.to(DEV) for k, v in m.cache.items()}
        self.pool = vc.alloc_pool(m.pages, DEV)
        self.pool["refs"].copy_(ints(m.refs))
        self.pool["free"].copy_(ints(m.bits()))
        self.table, self.kv, self.status = ints(m.table), ints(m.kv), torch.zeros(1, dtype=torch.int32, device=DEV)

    def same(self, m, status=0, data=True):
        assert self.table.tolist() == m.table and self.kv.tolist() == m.kv
        assert self.pool["refs"].tolist() == m.refs and self.pool["free"].tolist() == m.bits()
        assert int(self.status) == status
        self.status.zero_()
        if data:
            for k, v in m.cache.items():
                assert torch.equal(self.cache[k].cpu(), v), k

    def reserve(self, n, **kw):
        vc.vc_pages_reserve(self.cache, self.pool, offsets(n), self.kv, self.table, sum(n), dev_status=self.status, **kw)

    def trim(self, lens):
        vc.vc_pages_trim(self.cache, self.pool, self.table, self.kv, ints(lens), dev_status=self.status)

    def compact(self):
        return vc.vc_pages_compact(self.cache, self.pool, self.table, dev_status=self.status)


def grown(pages=40, page=16, rows=6, cols=8, lens=(100, 40, 16, 0, 1, 33), seed=0, **kw):
    m = Model(pages, page, rows, cols, seed=seed, **kw)
    m.kv = list(lens)
    assert m.reserve(lens)
    return m


@pytest.mark.parametrize("seed", range(12))
def test_random_walks(seed):
    """Growing, taking back, forking, ending and moving together in any order, with too few pages at times."""
    rng = rng_of(seed)
    page = rng.choice([16, 32])
    m = Model(rng.choice([9, 14, 33, 97]), page, 6, 8, H=rng.choice([1, 3]), d=rng.choice([64, 128]), seed=seed)
    dev, failed = Device(m), 0
    for op, arg in walk(m, rng, 40):
        if op == "reserve":
            m.kv = [k + n for k, n in zip(m.kv, arg)]
            dev.kv += ints(arg)
            dev.reserve(arg)
            ok = m.reserve(arg)
            dev.same(m, 0 if ok else 6)
            if not ok:                                   # the tokens that found no page are taken back
                failed += 1
                lens = [k - n for k, n in zip(m.kv, arg)]
                m.trim(lens)
                dev.trim(lens)
        elif op == "trim":
            m.trim(arg)
            dev.trim(arg)
        elif op == "compact":
            assert int(dev.compact()) == m.compact()
        else:
            parents, rows, lens = arg
            none = [0 if r in rows else -1 for r in range(6)]
            m.trim(none)
            dev.trim(none)
            # forks of the other half of the rows
            base, other = (0, 3) if rows[0] == 0 else (3, 0)
            dev_parents = ints([p if p < 0 else p - other for p in parents])
            vc.vc_pages_fork(dev.cache, dev.pool, dev.table[other:other + 3], dev.kv[other:other + 3], dev_parents, dev.table[base:base + 3],
                             dev.kv[base:base + 3], lens=None if lens is None else ints(lens), dev_status=dev.status)
            m.fork(parents, rows, lens)
        assert m.consistent()
        dev.same(m)


@pytest.mark.parametrize("page,H,d", [(16, 1, 64), (128, 3, 128)])
def test_last_writer_keeps_the_page(page, H, d):
    """Five names of a page that begins to be written: all five write, all but a later one, or only some."""
    for who in ([1] * 5, [1, 1, 1, 1, 0], [0, 1, 0, 1, 0], [0, 0, 0, 0, 1]):
        m = Model(60, page, 5, 4, H=H, d=d, seed=1)
        m.kv[0] = page + 5
        assert m.reserve([page + 5, 0, 0, 0, 0])
        m.fork([0, 0, 0, 0], [1, 2, 3, 4])
        dev = Device(m)
        m.kv = [k + w for k, w in zip(m.kv, who)]
        dev.kv += ints(who)
        dev.reserve(who)
        assert m.reserve(who)
        dev.same(m)
        if who[0] and all(who):
            assert m.table[4][1] == 1 and m.refs[1] == 1        # the old page: the last one's
        dev.reserve(who)                                        # once more: nothing is left to do
        dev.same(m)


def test_too_few_pages_take_none():
    """The state stays, entries that needed a copy are marked, an append behind it writes nowhere, and a second
    call with enough pages makes up for it."""
    m = grown(pages=17)
    m.trim([-1, -1, -1, -1, 0, -1])
    m.fork([0, 1], [3, 4])
    kv, n, refs = list(m.kv), [1, 50, 0, 1, 1, 50], list(m.refs)
    m.kv = [k + x for k, x in zip(kv, n)]
    dev = Device(m)
    dev.reserve(n)
    assert not m.reserve(n) and m.refs == refs
    dev.same(m, 6)
    assert [m.table[b][j] < -1 for b, j in ((0, 6), (1, 2), (3, 6), (4, 2), (5, 2))] == [True] * 4 + [False]
    # the tokens that found no page go nowhere
    c = Case(n=n, kv=m.kv, H=2, d=64, seed=2)
    written = torch.zeros(m.pages, m.page, dtype=torch.bool)
    for b, k in enumerate(m.kv):
        for p in range(k - n[b], k):
            if m.table[b][p // 16] >= 0:
                written[m.table[b][p // 16], p % 16] = True
    vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), dev.cache, offsets(n), dev.kv, dev.table, dev_status=dev.status)
    assert int(dev.status) == 1 and int(written.sum()) == 15
    dev.status.zero_()
    for k, v in m.cache.items():
        same = (dev.cache[k].cpu() == v).transpose(1, 2)
        assert same[~written].all(), k
        dev.cache[k].copy_(v)
    # taken back, three sequences ended: now the marked entries get theirs
    for x in (m, dev):
        x.trim([kv[0], 0, 0, kv[3], kv[4], 0])
    dev.same(m)
    n = [1, 0, 0, 1, 1, 0]
    m.kv = [k + x for k, x in zip(m.kv, n)]
    dev.kv += ints(n)
    dev.reserve(n)
    assert m.reserve(n) and m.consistent()
    dev.same(m)
    assert all(e >= -1 for row in m.table for e in row)


def test_marked_entries_move_fork_and_end_like_others():
    m = grown(pages=16, seed=3)
    m.fork([0], [3])
    m.kv[0] += 25
    assert not m.reserve([25, 0, 0, 0, 0, 0]) and any(e < -1 for e in m.table[0])
    m.kv[0] -= 25
    m.trim([-1, 0, -1, -1, -1, -1])
    dev = Device(m)
    assert int(dev.compact()) == m.compact()
    dev.same(m)
    vc.vc_pages_fork(dev.cache, dev.pool, dev.table[:1], dev.kv[:1], ints([0]), dev.table[1:2], dev.kv[1:2], dev_status=dev.status)
    m.fork([0], [1])
    dev.same(m)
    m.trim([0, -1, -1, -1, -1, -1])
    dev.trim([0, -1, -1, -1, -1, -1])
    assert m.consistent()
    dev.same(m)


def test_broken_batches_and_pools_are_reported():
    """cu, kv_len, entries, parents and lengths out of range: reported, nothing outside is touched, and a broken batch
    reserves nothing."""
    m = grown(seed=4)
    for cu, kv in (([0, 4, 2, 12, 12, 12, 12], m.kv), ([0, 4, 8, 12, 12, 12, 2 ** 31 - 1], m.kv), ([-1, 0, 0, 0, 0, 0, 0], m.kv),
                   ([0, 1, 1, 1, 1, 1, 1], [129] + m.kv[1:]), ([0, 1, 1, 1, 1, 1, 1], [-1] + m.kv[1:])):
        dev = Device(m)
        vc.vc_pages_reserve(dev.cache, dev.pool, ints(cu), ints(kv), dev.table, 12, dev_status=dev.status)
        dev.same(m, 1)
    for e in (40, 2 ** 31 - 1, -42, -2 ** 31):          # numbers of no page
        dev = Device(m)
        dev.table[0, 0] = e
        dev.trim([0, -1, -1, -1, -1, -1])
        assert int(dev.status) == 1 and dev.table[0].tolist() == [-1] * 8
        assert dev.pool["refs"].tolist() == [r if p in (0,) or not any(p == x for x in m.table[0]) else 0 for p, r in enumerate(m.refs)]
        dev = Device(m)
        dev.table[0, 0] = e
        vc.vc_pages_fork(dev.cache, dev.pool, dev.table[:3], dev.kv[:3], ints([0, -1, 7]), dev.table[3:], dev.kv[3:], dev_status=dev.status)
        assert int(dev.status) == 1 and dev.table[3, 0] == -1 and dev.table[3, 1:].tolist() == m.table[0][1:]
        assert dev.table[4:].eq(-1).all() and dev.kv[3:].tolist() == [100, 0, 0]
        dev = Device(m)
        dev.table[0, 0] = e
        assert int(dev.compact()) == sum(r > 0 for r in m.refs) and int(dev.status) == 1
        assert dev.table[0].tolist() == [e] + m.table[0][1:]
    dev = Device(m)
    dev.table[3, 0] = 39                                  # named and counted nowhere
    dev.compact()
    assert int(dev.status) == 1 and int(dev.table[3, 0]) == 39
    dev = Device(m)
    dev.table[3, 0] = 39
    dev.trim([-1, -1, -1, 0, -1, -1])
    m2 = grown(seed=4)
    dev.same(m2, 1)
    for kv, lens in (([-5, 40, 16], None), ([129, 40, 16], None), ([100, 40, 16], [-3, 1, 1])):
        dev = Device(m)
        dev.kv[:3] = ints(kv)
        vc.vc_pages_fork(dev.cache, dev.pool, dev.table[:3], dev.kv[:3], ints([0, 1, 2]), dev.table[3:], dev.kv[3:],
                         lens=None if lens is None else ints(lens), dev_status=dev.status)
        assert int(dev.status) == 1 and int(dev.kv[3]) == 0 and dev.table[3].eq(-1).all() and int(dev.kv[4]) == (1 if lens else 40)


def test_free_pages_that_a_table_names_get_no_second_owner():
    """An entry that names a free page: a fork leaves it out, reserving replaces it; both report it."""
    m = grown(seed=7)
    free = max(p for p in range(m.pages) if not m.refs[p])
    for entry in (free, -2 - free):
        dev = Device(m)
        dev.table[1, 1] = entry
        vc.vc_pages_fork(dev.cache, dev.pool, dev.table[:3], dev.kv[:3], ints([1]), dev.table[3:4], dev.kv[3:4], dev_status=dev.status)
        assert int(dev.status) == 1 and int(dev.kv[3]) == 40
        assert dev.table[3].tolist() == [m.table[1][0], -1, m.table[1][2]] + [-1] * 5
        m2 = grown(seed=7)
        m2.refs[m.table[1][0]] += 1
        m2.refs[m.table[1][2]] += 1
        assert dev.pool["refs"].tolist() == m2.refs and dev.pool["free"].tolist() == m2.bits()

        m2 = grown(seed=7)
        dev = Device(m)
        n = [0, 20, 0, 0, 0, 0]                                  # positions 20 .. 39: columns 1 and 2
        dev.table[1, 1] = entry
        dev.reserve(n)
        m2.refs[m2.table[1][1]] = 1                              # its own page before, still counted
        lowest = min(p for p in range(m.pages) if not m.refs[p])
        m2.table[1][1], m2.refs[lowest] = lowest, 1
        dev.same(m2, 1)


def test_fork_into_fewer_columns():
    m = grown(seed=5)
    dev = Device(m)
    table, kv = torch.full((3, 3), 9, dtype=torch.int32, device=DEV), ints([7, 7, 7])
    vc.vc_pages_fork(dev.cache, dev.pool, dev.table, dev.kv, ints([1, 5, 0]), table, kv, dev_status=dev.status)
    assert int(dev.status) == 1 and kv.tolist() == [40, 33, 0]           # 100 tokens do not fit in 3 pages of 16
    assert table.tolist() == [m.table[1][:3], m.table[5][:3], [-1] * 3]


def test_positions_below_zero_and_rows_without_tokens():
    m = Model(30, 16, 4, 6, seed=6)
    m.kv = [5, 0, 96, 20]
    dev = Device(m)
    n = [9, 3, 96, 0]
    dev.reserve(n)
    assert m.reserve(n)
    dev.same(m)
    dev.reserve([0, 0, 0, 0])
    dev.same(m)


@pytest.mark.parametrize("rows,pages", [(1500, 4000), (6000, 9000)])
def test_many_sequences(rows, pages):
    """More sequences than the planning block has threads, and than its shared memory has room for; more than 2^12
    forks of one page, all of which then write."""
    m = Model(pages, 16, rows, 3, H=1, seed=7)
    n = [(b * 7) % 20 if b < 500 else 0 for b in range(rows)]
    m.kv = list(n)
    dev = Device(m)
    dev.reserve(n)
    assert m.reserve(n)
    dev.same(m)
    dev.trim([-1] * 500 + [0] * (rows - 500))
    vc.vc_pages_fork(dev.cache, dev.pool, dev.table[:500], dev.kv[:500], ints([5] * (rows - 500)), dev.table[500:], dev.kv[500:])
    m.fork([5] * (rows - 500), range(500, rows))
    dev.same(m)
    n = [0] * 500 + [1] * (rows - 500)
    m.kv = [k + x for k, x in zip(m.kv, n)]
    dev.kv += ints(n)
    dev.reserve(n)
    assert m.reserve(n) and m.consistent()
    dev.same(m)
    assert int(dev.compact()) == m.compact()
    dev.same(m)


def test_large_pools():
    """2^20 + 5 pages: the free ones behind a long stretch of used ones, and moved from the far end."""
    pages = (1 << 20) + 5
    cache, pool = vc.alloc_cache(pages, 16, 1, 64, DEV), vc.alloc_pool(pages, DEV)
    table = torch.full((2, 600), -1, dtype=torch.int32, device=DEV)
    used = torch.zeros(pages, dtype=torch.int32, device=DEV)
    used[:pages - 700] = 1
    pool["refs"].copy_(used)
    bits = torch.zeros(-(-pages // 32) * 32, dtype=torch.int64, device=DEV)
    bits[:pages] = 1 - used
    words = lambda b: ((b.view(-1, 32) << torch.arange(32, device=DEV)).sum(1) + (1 << 31)) % (1 << 32) - (1 << 31)  # noqa: E731
    pool["free"].copy_(words(bits))
    kv, cu = ints([16 * 600, 16 * 50]), ints([0, 16 * 600, 16 * 650])
    vc.vc_pages_reserve(cache, pool, cu, kv, table, 16 * 650)
    at = pages - 700
    assert table[0].tolist() == list(range(at, at + 600)) and table[1, :50].tolist() == list(range(at + 600, at + 650))
    cache["K8"][at:at + 650] = torch.randint(0, 100, (650, 1, 16, 64), device=DEV).to(torch.uint8)
    cache["sv"][at:at + 650] = torch.rand(650, 1, 16, device=DEV)
    K8, sv = cache["K8"][at:at + 650].clone(), cache["sv"][at:at + 650].clone()
    # what the other pages stand for ends, all but every third of the last ones
    left = torch.arange(pages, device=DEV) >= at
    pool["refs"].mul_(left)
    bits[:pages] = pool["refs"] == 0
    pool["free"].copy_(words(bits))
    assert int(vc.vc_pages_compact(cache, pool, table)) == 650
    assert table[0].tolist() == list(range(600)) and table[1, :50].tolist() == list(range(600, 650)) and table[1, 50:].eq(-1).all()
    assert torch.equal(cache["K8"][:650], K8) and torch.equal(cache["sv"][:650], sv)
    assert pool["refs"][:650].eq(1).all() and not pool["refs"][650:].any()
    bits[:pages] = pool["refs"] == 0
    assert torch.equal(pool["free"].long(), words(bits))


@pytest.mark.parametrize("H,page,d", [(1, 16, 64), (3, 32, 128), (5, 256, 64)])
def test_copy_between_caches(H, page, d):
    """Other strides on the other side; -1 leaves a pair out; numbers out of range are reported."""
    a, b = (Model(50, page, 1, 1, H=H, d=d, seed=8 + i) for i in range(2))
    src = {k: v.to(DEV) for k, v in a.cache.items()}
    dst = {}
    for k, v in b.cache.items():
        big = torch.full([50, page + 4, H + 1, d + 16] if k in ("K8", "V8") else [50, H, page + 4], 3, dtype=v.dtype, device=DEV)
        dst[k] = big[:, 2:2 + page, 1:, 16:].transpose(1, 2) if k in ("K8", "V8") else big[:, :, 4:]
        dst[k].copy_(v)
    g = torch.Generator().manual_seed(9)
    pages = torch.randperm(50, generator=g)[:33].to(torch.int32)
    to = torch.randperm(50, generator=g)[:33].to(torch.int32)
    pages[4], to[7] = -1, -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert vc.vc_cache_copy(src, dst, pages.to(DEV), to.to(DEV), dev_status=status) is dst
    for x, y in zip(pages.tolist(), to.tolist()):
        if x >= 0 and y >= 0:
            for k in a.cache:
                b.cache[k][y] = a.cache[k][x]
    assert int(status) == 0
    for k, v in b.cache.items():
        assert torch.equal(dst[k].cpu(), v), k
    for bad in ([50], [-2], [2 ** 31 - 1]):
        for args in ((ints(bad), ints([1])), (ints([1]), ints(bad))):
            status.zero_()
            vc.vc_cache_copy(src, dst, *args, dev_status=status)
            assert int(status) == 1 and all(torch.equal(dst[k].cpu(), v) for k, v in b.cache.items())
    # within one cache
    vc.vc_cache_copy(src, src, ints([3, 4]), ints([40, 41]))
    for k, v in a.cache.items():
        v[40], v[41] = v[3].clone(), v[4].clone()
        assert torch.equal(src[k].cpu(), v)
    vc.vc_cache_copy(src, src, ints([]), ints([]))


@pytest.mark.parametrize("G,d", [(1, 128), (4, 64)])
def test_continuations_of_a_prompt(G, d):
    """As used, in a captured graph: a prompt is cached, forked, and each continuation reserves, writes and attends,
    token by token; every one gives what a sequence of its own gives."""
    H, page, N, prompt, steps = 2, 16, 3, 37, 20
    whole = [Case(n=[prompt + steps], kv=[prompt + steps], H=H, G=G, d=d, page=page, seed=30) for _ in range(N)]
    for i, c in enumerate(whole[1:]):
        other = Case(n=[prompt + steps], kv=[prompt + steps], H=H, G=G, d=d, page=page, seed=31 + i)
        for k in ("Q", "K", "V"):
            getattr(c, k)[prompt:] = getattr(other, k)[prompt:]
    pages = 24
    cache, pool = vc.alloc_cache(pages, page, H, d, DEV), vc.alloc_pool(pages, DEV)
    table, kv = torch.full((N + 1, 6), -1, dtype=torch.int32, device=DEV), torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu, kv[0] = ints([0, prompt]), prompt
    vc.vc_pages_reserve(cache, pool, cu, kv[:1], table[:1], prompt, dev_status=status)
    vc.vc_cache_append(whole[0].K[:prompt].to(DEV), whole[0].V[:prompt].to(DEV), cache, cu, kv[:1], table[:1])
    vc.vc_pages_fork(cache, pool, table[:1], kv[:1], ints([0] * N), table[1:], kv[1:], dev_status=status)
    vc.vc_pages_trim(cache, pool, table[:1], kv[:1], ints([0]), dev_status=status)     # only its forks hold the prompt now
    one = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    Q = torch.zeros((N, H * G, d), dtype=torch.bfloat16, device=DEV)
    K, V = (torch.zeros((N, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        kv[1:] += 1
        vc.vc_pages_reserve(cache, pool, one, kv[1:], table[1:], N, dev_status=status)
        vc.vc_cache_append(K, V, cache, one, kv[1:], table[1:], dev_status=status)
        return vc.vc_attn_paged(Q, cache, one, kv[1:], table[1:], max_q=1, dev_status=status)

    graph, outs = None, []
    for t in range(prompt, prompt + steps):
        for i, c in enumerate(whole):
            Q[i], K[i], V[i] = (x[t].to(DEV) for x in (c.Q, c.K, c.V))
        if t == prompt + 2:
            graph, keep = torch.cuda.CUDAGraph(), kv.clone()
            with torch.cuda.graph(graph):
                out = step()
            kv.copy_(keep)
        if graph is None:
            outs.append([x.clone() for x in step()])
        else:
            graph.replay()
            outs.append([x.clone() for x in out])
    assert int(status) == 0
    held = [set(r) - {-1} for r in table[1:].tolist()]
    assert len(set.intersection(*held)) == prompt // page and sum(pool["refs"].tolist()) == sum(len(h) for h in held)
    for i, c in enumerate(whole):
        want = c.appended()
        O, tol, lse, told = c.attend(want)
        got = torch.stack([o[0][i] for o in outs]).double().cpu(), torch.stack([o[1][i] for o in outs]).double().cpu()
        assert torch.all((got[0] - O[prompt:]).abs() <= tol[prompt:]) and torch.all((got[1] - lse[prompt:]).abs() <= told[prompt:])
    # all end: the pool is as new
    vc.vc_pages_trim(cache, pool, table, kv, ints([0] * (N + 1)), dev_status=status)
    new = vc.alloc_pool(pages, DEV)
    assert torch.equal(pool["refs"], new["refs"]) and torch.equal(pool["free"], new["free"]) and table.eq(-1).all() and int(status) == 0


def test_on_another_stream_and_with_a_workspace():
    m = grown(seed=10)
    m.fork([0, 1], [3, 4])
    side = torch.cuda.Stream()
    n = [1, 1, 1, 1, 1, 1]
    for kw in (dict(stream=side), dict(workspace=torch.empty(vc.pages_reserve_workspace_bytes(Device(m).cache, 6, 6), dtype=torch.uint8, device=DEV))):
        dev, want = Device(m), grown(seed=10)
        want.fork([0, 1], [3, 4])
        want.kv = [k + 1 for k in want.kv]
        dev.kv += 1
        side.wait_stream(torch.cuda.current_stream())
        dev.reserve(n, **kw)
        assert want.reserve(n)
        torch.cuda.synchronize()
        dev.same(want)
        kw.pop("workspace", None)
        side.wait_stream(torch.cuda.current_stream())
        used = vc.vc_pages_compact(dev.cache, dev.pool, dev.table, dev_status=dev.status, **kw)
        torch.cuda.synchronize()
        assert int(used) == want.compact()
        dev.same(want)

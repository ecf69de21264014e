"""GPU: the calls around a paged cache on caches that are parts of larger allocations: heads of several layers in the same
pages, which share a table and a pool, and pages, heads and tokens apart.  Equal, bit for bit, to the same calls on a cache of
its own, and nothing else is written."""
import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import Case
from pool_model import Model, rng_of, walk
from shared_case import Shared
from test_gpu_pages import DEV, Device, ints, offsets
from test_gpu_shared import same_bits, tables

pytestmark = pytest.mark.gpu
KEYS = ("K8", "sk", "V8", "sv")


def apart(cache, fill=3):
    """A copy of `cache` ({K8: [pages, H, page, d], ..}) with room between its pages, heads, tokens and channels; the larger
    tensors, and where in them it lies."""
    pages, H, page, d = cache["K8"].shape
    views, wholes = {}, {}
    for k in KEYS:
        codes = k in ("K8", "V8")
        big = torch.full([pages + 1, page + 3, H + 2, d + 32] if codes else [pages + 1, H + 1, page + 8], fill, dtype=cache[k].dtype, device=DEV)
        at = (lambda b: b[1:, 2:2 + page, 1:1 + H, 16:16 + d].transpose(1, 2)) if codes else (lambda b, p=page: b[1:, :H, 4:4 + p])
        at(big).copy_(cache[k])
        views[k], wholes[k] = at(big), (big, at)
    return views, wholes


def untouched(wholes, fill=3):
    """Whether all but the cache itself is as it was."""
    for big, at in wholes.values():
        rest = big.clone()
        at(rest).fill_(fill)
        if not torch.all(rest == fill):
            return False
    return True


def layers(cache, count):
    """`count` layers of the cache's heads in the same pages: one cache of all heads, and each layer's part of it."""
    whole = {k: torch.cat([v] * count, 1).contiguous().to(DEV) for k, v in cache.items()}
    H = cache["K8"].shape[1]
    return whole, [{k: v[:, i * H:(i + 1) * H] for k, v in whole.items()} for i in range(count)]


@pytest.mark.parametrize("seed", range(6))
def test_random_walks_with_pages_apart(seed):
    rng = rng_of(100 + seed)
    m = Model(rng.choice([14, 33]), rng.choice([16, 64]), 6, 8, H=rng.choice([1, 3]), d=rng.choice([64, 128]), seed=seed)
    dev = Device(m)
    dev.cache, wholes = apart(dev.cache)
    for op, arg in walk(m, rng, 25):
        if op == "reserve":
            m.kv = [k + n for k, n in zip(m.kv, arg)]
            dev.kv += ints(arg)
            dev.reserve(arg)
            ok = m.reserve(arg)
            dev.same(m, 0 if ok else 6)
            if not ok:
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
            base, other = (0, 3) if rows[0] == 0 else (3, 0)
            vc.vc_pages_fork(dev.cache, dev.pool, dev.table[other:other + 3], dev.kv[other:other + 3], ints([p if p < 0 else p - other for p in parents]),
                             dev.table[base:base + 3], dev.kv[base:base + 3], lens=None if lens is None else ints(lens), dev_status=dev.status)
            m.fork(parents, rows, lens)
        dev.same(m)
    assert untouched(wholes)


@pytest.mark.parametrize("page,G,d,layout", [(16, 1, 128, "halves"), (64, 4, 64, "pairs"), (256, 2, 128, "pairs")])
def test_rows_turned_into_pages_apart(page, G, d, layout):
    c = Case(n=[5, 0, 1, 70], kv=[33, 4, 1, 300], H=3, G=G, d=d, page=page, seed=60, tail=2)
    rope = vc.make_rope(d, layout=layout, device=DEV)
    want = c.cache(DEV)
    q = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), want, *c.args(DEV), rope)
    views, wholes = apart(c.cache(DEV))
    got = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), views, *c.args(DEV), rope)
    rows = int(c.cu[-1])
    assert same_bits(got[:rows], q[:rows]) and all(same_bits(views[k], want[k]) for k in KEYS) and untouched(wholes)


SHARED = {
    "one_each": dict(groups=[(777, [(3, 1)] * 9 + [(300, 1)])], H=2, G=4, page=32),
    "drafts": dict(groups=[(1000, [(20, 1), (9, 4)]), (129, [(200, 7)] * 5), (2000, [(1, 1)] * 20)], H=3, G=3, d=64, page=64),
    "chunks": dict(groups=[(400, [(130, 130), (200, 90)]), (33, [(300, 300)])], H=2, G=2, page=256),
}


@pytest.mark.parametrize("case", SHARED)
def test_attention_over_pages_apart(case):
    c = Shared(seed=61, **SHARED[case])
    for wide in (True, False):
        args = (*tables(c, wide), *c.shared_args(DEV))
        hints = dict(max_q=max(c.n), max_rows=c.most())
        want = vc.vc_attn_paged_shared(c.Q.to(DEV), c.cache(DEV), *args, **hints)
        c.check(want, c.cache())
        views, wholes = apart(c.cache(DEV))
        got = vc.vc_attn_paged_shared(c.Q.to(DEV), views, *args, **hints)
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1]) and untouched(wholes)


def test_layers_share_a_table_and_a_pool():
    """A model of three layers: their heads lie side by side in the same pages, so one reservation, fork, trim or move is for
    all of them; each layer appends to and attends over its own heads.  Every layer gives what a cache of its own gives."""
    count, H, G, d, page, N = 3, 2, 2, 64, 16, 4
    prompt, steps = 37, 5
    rope = vc.make_rope(d, device=DEV)
    g = torch.Generator().manual_seed(62)
    bf = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    first = [(bf(prompt, H * G, d), bf(prompt, H, d), bf(prompt, H, d)) for _ in range(count)]
    more = [[(bf(N, H * G, d), bf(N, H, d), bf(N, H, d)) for _ in range(count)] for _ in range(steps)]

    def run(cache, parts, which):
        """The outputs of the layers `which`, whose heads are parts of `cache`, and its state at the end."""
        pool = vc.alloc_pool(24, DEV)
        table, kv, status, out = torch.full((N + 1, 1800), -1, dtype=torch.int32, device=DEV), ints([prompt] + [0] * N), ints([0]), []
        vc.vc_pages_reserve(cache, pool, ints([0, prompt]), kv[:1], table[:1], prompt, dev_status=status)
        for part, i in zip(parts, which):
            q = vc.vc_cache_append_rope(*first[i], part, ints([0, prompt]), kv[:1], table[:1], rope, dev_status=status)
            out += [q, *vc.vc_attn_paged(q, part, ints([0, prompt]), kv[:1], table[:1], max_q=prompt, dev_status=status)]
        vc.vc_pages_fork(cache, pool, table[:1], kv[:1], ints([0] * N), table[1:], kv[1:], dev_status=status)
        vc.vc_pages_trim(cache, pool, table[:1], kv[:1], ints([0]), dev_status=status)
        for step in more:
            kv[1:] += 1
            vc.vc_pages_reserve(cache, pool, offsets([1] * N), kv[1:], table[1:], N, dev_status=status)
            for part, i in zip(parts, which):
                q = vc.vc_cache_append_rope(*step[i], part, offsets([1] * N), kv[1:], table[1:], rope, dev_status=status)
                out += [q, *vc.vc_attn_paged_shared(q, part, offsets([1] * N), kv[1:], table[1:], ints([0, N]), ints([prompt]), max_q=1, max_rows=N, dev_status=status)]
            if step is more[2]:
                vc.vc_pages_trim(cache, pool, table[1:], kv[1:], ints([0, -1, -1, -1]), dev_status=status)
                vc.vc_pages_compact(cache, pool, table, dev_status=status)
                vc.vc_pages_fork(cache, pool, table[2:3], kv[2:3], ints([0]), table[1:2], kv[1:2], dev_status=status)
        assert int(status) == 0
        return out, (table, kv, pool["refs"], pool["free"])

    whole, parts = layers(vc.alloc_cache(24, page, H, d, "cpu"), count)
    out, state = run(whole, parts, range(count))
    for i in range(count):
        own = vc.alloc_cache(24, page, H, d, DEV)
        alone, end = run(own, [own], [i])
        assert all(torch.equal(a, b) for a, b in zip(state, end))
        per = [out[j:j + 3] for j in range(0, len(out), 3)][i::count]
        assert all(same_bits(a, b) for a, b in zip([x for y in per for x in y], alone))
        slots = {(int(state[0][b, p // page]), p % page) for b in range(1, N + 1) for p in range(int(state[1][b]))}
        for k in KEYS:
            for p, t in slots:
                assert torch.equal(parts[i][k][p, :, t], own[k][p, :, t]), (k, p, t)

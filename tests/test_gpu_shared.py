"""GPU: attention over shared prefixes against the definition of attention in fp64 (paged_case.py), with that one's bars:
the prefix's and the own keys' parts are joined in fp32, as parts of one pass are."""
import math

import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import Case
from shared_case import Shared

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def tables(c, wide):
    """The batch's arguments; wide: a table with so many columns that the work could be large, without which calls of few
    keys take one pass over all of them."""
    cu, kv, table = c.args(DEV)
    if wide:
        more = -(-1600 * 128 // (c.B * c.H * c.page)) + 1
        table = torch.cat([table, torch.full((c.B, more), -1, dtype=torch.int32, device=DEV)], 1)
    return cu, kv, table


def attend(c, cache=None, status=0, wide=True, **kw):
    seen = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw.setdefault("max_q", max(c.n))
    kw.setdefault("max_rows", c.most())
    groups = kw.pop("groups", c.shared_args(DEV))
    out = vc.vc_attn_paged_shared(c.Q.to(DEV), cache or c.cache(DEV), *tables(c, wide), *groups, dev_status=seen, **kw)
    torch.cuda.synchronize()
    assert int(seen) == status
    return out


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


CASES = {
    "one": dict(groups=[(40, [(1, 1)])], H=1, d=64),
    "two": dict(groups=[(128, [(1, 1), (5, 1)])], H=2, G=2, d=64),
    "short": dict(groups=[(3, [(9, 1), (2, 2), (1, 0), (30, 4)])], H=2, G=2),
    "page border": dict(groups=[(256, [(1, 1), (16, 1), (17, 1)])], H=1, G=4),
    "mid page": dict(groups=[(777, [(3, 1)] * 9 + [(300, 1)])], H=2, G=4, page=32),
    "no prefix": dict(groups=[(0, [(70, 1), (5, 5)]), (100, [(3, 3)]), (0, [(1, 1)])], H=2, G=2, d=64),
    "many rows": dict(groups=[(300, [(20, 3)] * 30)], H=1, G=2, page=64),
    "all rows": dict(groups=[(500, [(7, 1)] * 70)], H=1, G=8, d=64),
    "groups": dict(groups=[(1000, [(20, 1), (9, 4)]), (129, [(200, 7)] * 5), (2000, [(1, 1)] * 20)], H=2, G=3, page=64),
    "alone too": dict(before=[(300, 2), (0, 0), (50, 50)], groups=[(64, [(10, 1), (3, 3)])], H=2, G=4, d=64, tail=5),
    "chunks": dict(groups=[(400, [(130, 130), (200, 90)]), (33, [(300, 300)])], H=1, G=2, page=128),
    "chunks of d 64": dict(groups=[(1500, [(257, 257), (1, 1), (40, 40)])], H=2, d=64, page=256),
    "long": dict(groups=[(12000, [(40, 1), (3, 2)])], H=1, G=2, d=64, page=64),
    "long, many rows": dict(groups=[(9000, [(33, 3)] * 20)], H=1, G=4, page=128),
}


def name(k):
    return k.replace(" ", "_").replace(",", "")


@pytest.mark.parametrize("causal,wide", [(1, True), (0, True), (1, False)])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_attention(case, causal, wide):
    c = Shared(seed=1, **CASES[case])
    c.check(attend(c, causal=causal, wide=wide), c.cache(), causal=causal)


@pytest.mark.parametrize("hints", [(0, 0), (1, 1), (5, 5), (10, 20), (60, 9), (9, 60), (33, 300), (65, 90), (300, 5000), (2 ** 32, 2 ** 40)], ids=str)
def test_hints_choose_kernels_only(hints):
    """Tiles of 8 to 256 rows in both passes, whatever the batch."""
    for case in ("groups", "chunks of d 64"):
        c = Shared(seed=2, **CASES[case])
        c.check(attend(c, max_q=hints[0], max_rows=hints[1]), c.cache())


@pytest.mark.parametrize("case", ["groups", "many rows", "chunks"], ids=name)
def test_same_as_every_sequence_by_itself(case):
    """The same numbers as vc_attn_paged on the same batch, within both bars; same call, same bits."""
    c = Shared(seed=3, **CASES[case])
    got = attend(c)
    again = attend(c)
    assert same_bits(got[0], again[0]) and same_bits(got[1], again[1])
    cache = c.cache(DEV)
    alone = vc.vc_attn_paged(c.Q.to(DEV), cache, *c.args(DEV), max_q=max(c.n))
    c.check(alone, c.cache())
    _, tol, _, told = c.attend(c.cache())
    T = int(c.cu[-1])
    assert torch.all((got[0] - alone[0]).abs().double().cpu()[:T] <= 2 * tol[:T]) and torch.all((got[1] - alone[1]).abs().double().cpu()[:T] <= 2 * told[:T])


@pytest.mark.parametrize("case", ["two", "many rows"], ids=name)
def test_peaked_scores_and_value_scales(case):
    """Large scores, so that one part has all of the weight, a softmax scale, and values of very different sizes."""
    c = Shared(seed=4, qmul=6.0, **CASES[case])
    f = torch.exp2(torch.randint(-30, 30, c.sv.shape, generator=torch.Generator().manual_seed(1)).float())
    for g, p in enumerate(c.prefix):                       # the prefix's last page stays the same for all
        if p % c.page:
            pages = [int(c.table[b, p // c.page]) for b in range(c.groups[g], c.groups[g + 1])]
            f[pages, :, :p % c.page] = f[pages[0], :, :p % c.page].clone()
    c.sv *= f
    c.check(attend(c), c.cache())
    c.check(attend(c, softmax_scale=0.5), c.cache(), scale=0.5)


@pytest.mark.parametrize("case", ["mid page", "many rows"], ids=name)
def test_values_all_zero_and_not_finite_numbers(case):
    """A prefix without values, own tokens that are not numbers in one sequence, and a query that is none: as in
    vc_attn_paged, only the rows that see them."""
    c = Shared(seed=5, **CASES[case])
    whole = c.prefix[0] // c.page
    for p in c.table[0, :whole].tolist():
        c.V8[p], c.sv[p] = 0, 0.0
    b = c.B - 1
    page, at = int(c.table[b, (c.kv[b] - 1) // c.page]), (c.kv[b] - 1) % c.page
    c.sv[page, 0, at] = math.nan
    c.Q[0, 0, 7] = math.inf
    got = attend(c)
    O, tol, lse, told = c.attend(c.cache())
    # a query that sees a token of NaN scale gets NaN, in lse as in O (the definition's lse goes by the keys alone)
    spoilt = torch.isnan(O).any(-1)
    assert torch.equal(torch.isnan(got[0].cpu()).all(-1), spoilt) and torch.equal(torch.isnan(got[1].cpu()), spoilt)
    assert torch.all((got[0].double().cpu() - O).abs()[~spoilt] <= tol[~spoilt]) and torch.all((got[1].double().cpu() - lse).abs()[~spoilt] <= told[~spoilt])
    assert spoilt[0, 0] and spoilt[int(c.cu[-1]) - 1, 0] and int(spoilt.sum()) < spoilt.numel() // 2


@pytest.mark.parametrize("case", ["mid page", "many rows"], ids=name)
def test_garbage_behind_the_last_token(case):
    c = Shared(seed=6, **CASES[case])
    clean, used = c.cache(), torch.zeros(c.sk.shape, dtype=torch.bool)
    for b in range(c.B):
        for p in range(c.kv[b]):
            used[c.table[b, p // c.page], :, p % c.page] = True
    for k in ("K8", "V8"):
        getattr(c, k)[~used] = 0x7F
    c.sk[~used], c.sv[~used] = math.nan, math.inf
    c.check(attend(c), clean)


def test_rows_of_no_sequence_stay():
    c = Shared(seed=7, **CASES["alone too"])
    O = torch.full((c.T, c.H * c.G, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.T, c.H * c.G), 7.0, device=DEV)
    attend(c, O=O, lse=lse)
    c.check((O, lse), c.cache())
    n = sum(c.n)
    assert torch.all(O[n:] == 7.0) and torch.all(lse[n:] == 7.0)


def test_without_groups():
    c = Case(n=[3, 0, 40], kv=[300, 20, 90], H=2, G=2, seed=8)
    none = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    c.check(vc.vc_attn_paged_shared(c.Q.to(DEV), c.cache(DEV), *c.args(DEV), *none), c.cache())
    empty = Case(n=[0], kv=[5], H=2)
    O, lse = vc.vc_attn_paged_shared(empty.Q.to(DEV), empty.cache(DEV), *empty.args(DEV), *none)
    assert O.shape == (0, 2, 128) and lse.shape == (0, 2)


def test_rows_without_keys():
    """kv_len 0 and 0 of a prefix: O = 0, lse = -inf."""
    c = Shared([(0, [(4, 4), (9, 1)]), (200, [(1, 1), (2, 1)])], H=2, G=2, seed=9)
    c.kv[0] = 0
    c.kv_len[0] = 0
    got = attend(c)
    c.check(got, c.cache())
    assert torch.all(got[0][:4] == 0) and torch.all(got[1][:4] == -math.inf)


def test_pages_that_are_not_there():
    """Missing pages of a prefix (of the group's first sequence) and of a sequence's own, behind the one that the prefix
    ends in: unseen, and reported."""
    for case, b in (("mid page", 9), ("groups", 2)):
        c = Shared(seed=10, **CASES[case])
        c.table[:, 1] = -1
        assert (c.kv[b] - 1) // c.page > (c.kv[b] - 190) // c.page
        c.table[b, (c.kv[b] - 1) // c.page] = c.pages
        c.check(attend(c, status=1), c.cache())


def test_broken_groups_are_reported_and_touch_nothing_outside():
    c = Shared(seed=11, **CASES["alone too"])
    guard, T, Hq = 64, c.T, c.H * c.G
    for groups, prefix in (([3, 9], [64]), ([-4, 5], [64]), ([5, 3], [64]), ([2 ** 31 - 1, -2 ** 31], [64]), ([3, 5], [66]), ([3, 5], [-1]), ([3, 5], [2 ** 31 - 1]),
                           ([0, 5], [64])):
        g = tuple(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (groups, prefix))
        for max_q, max_rows in ((1, 1), (50, 50), (500, 500)):
            O = torch.full((T + 2 * guard, Hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
            lse = torch.full((T + 2 * guard, Hq), 7.0, device=DEV)
            attend(c, groups=g, status=1, O=O[guard:-guard], lse=lse[guard:-guard], max_q=max_q, max_rows=max_rows)
            for x in (O, lse):
                assert torch.all(x[:guard] == 7.0) and torch.all(x[-guard:] == 7.0)
    for cu, kv in (([0, 2, 1, 52, 53, 56], c.kv), ([-3, 2, 2, 52, 53, 56], c.kv), ([0, 2, 2, 52, 53, 2 ** 31 - 1], c.kv), ([0, 2, 2, 52, 53, 56], [300, -1, 50, 74, 67]),
                   ([0, 2, 2, 52, 53, 56], [2 ** 31 - 1, 0, 50, 74, 67])):
        args = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, kv)]
        for max_q, max_rows in ((1, 1), (500, 500)):
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            O = torch.full((T + 2 * guard, Hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
            vc.vc_attn_paged_shared(c.Q.to(DEV), c.cache(DEV), *args, tables(c, max_q == 1)[2], *c.shared_args(DEV), O=O[guard:-guard], max_q=max_q, max_rows=max_rows, dev_status=status)
            assert int(status) == 1 and torch.all(O[:guard] == 7.0) and torch.all(O[-guard:] == 7.0)


@pytest.mark.parametrize("case", ["two", "groups", "many rows"], ids=name)
def test_given_outputs_and_streams(case):
    """Strided Q and O, a workspace of the caller's with anything in it, another stream, and the C entry without lse."""
    c = Shared(seed=12, **CASES[case])
    cache, args, groups, Q, Hq = c.cache(DEV), tables(c, True), c.shared_args(DEV), c.Q.to(DEV), c.H * c.G
    hints = dict(max_q=max(c.n), max_rows=c.most())
    want = vc.vc_attn_paged_shared(Q, cache, *args, *groups, **hints)
    c.check(want, c.cache())
    big = torch.full((c.T, Hq + 1, c.d + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    size = vc.attn_paged_shared_workspace_bytes(cache, Hq, c.B, c.T, len(c.prefix), **hints)
    wide_q = torch.full((c.T, Hq, 2, c.d), math.nan, dtype=torch.bfloat16, device=DEV)
    wide_q[:, :, 1] = Q
    assert same_bits(vc.vc_attn_paged_shared(wide_q[:, :, 1], cache, *args, *groups, **hints)[0], want[0])
    for fill in (0, 255, 170):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        vc.vc_attn_paged_shared(Q, cache, *args, *groups, O=big[:, :Hq, :c.d], workspace=ws, **hints)
        assert same_bits(big[:, :Hq, :c.d], want[0]) and torch.all(big[:, Hq] == 3.0) and torch.all(big[:, :, c.d:] == 3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        there = vc.vc_attn_paged_shared(Q, cache, *args, *groups, stream=side, **hints)
        here = vc.vc_attn_paged_shared(Q, cache, *args, *groups, **hints)
        torch.cuda.synchronize()
        assert same_bits(there[0], want[0]) and same_bits(here[1], want[1])
    O = torch.zeros_like(want[0])
    shape, batch = vc.cache_shape_of(cache), vc._batch_of(*args, c.T, 0)
    rc = vc.lib().vc_attn_paged_shared(Q.data_ptr(), Hq * c.d, c.d, Hq, shape, cache["K8"].data_ptr(), cache["sk"].data_ptr(), cache["V8"].data_ptr(),
                                       cache["sv"].data_ptr(), batch, groups[0].data_ptr(), groups[1].data_ptr(), len(c.prefix), 0.0, 1, hints["max_q"], hints["max_rows"],
                                       O.data_ptr(), Hq * c.d, c.d, None, ws.data_ptr(), ws.numel(), None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and same_bits(O, want[0])


def test_many_sequences_and_groups():
    """More sequences than a block has threads, in more groups than it has warps."""
    groups = [(20 + 7 * (g % 30), [(1 + (g + i) % 9, min(1 + (g + i) % 9, (g + i) % 3)) for i in range(1 + g % 13)]) for g in range(200)]
    c = Shared(groups, H=1, G=2, d=64, seed=13)
    assert c.B > 1200
    c.check(attend(c), c.cache())
    c.check(attend(c, max_q=200, max_rows=200), c.cache())


@pytest.mark.parametrize("G,d", [(1, 128), (4, 64)])
def test_generation_from_forks(G, d):
    """As used: a prompt's keys are turned and cached, forked, and every step of the continuations reserves, turns and
    writes, and attends with the prompt read once; in a captured graph from the third step on."""
    H, page, N, prompt, steps = 2, 16, 5, 149, 12
    rope = vc.make_rope(d, device=DEV)
    whole = [Case(n=[prompt + steps], kv=[prompt + steps], H=H, G=G, d=d, page=page, seed=40) for _ in range(N)]
    for i, c in enumerate(whole[1:]):
        other = Case(n=[prompt + steps], kv=[prompt + steps], H=H, G=G, d=d, page=page, seed=41 + i)
        for k in ("Q", "K", "V"):
            getattr(c, k)[prompt:] = getattr(other, k)[prompt:]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pages = 40
    cache, pool = vc.alloc_cache(pages, page, H, d, DEV), vc.alloc_pool(pages, DEV)
    table, kv, status = torch.full((N + 1, 2000), -1, dtype=torch.int32, device=DEV), torch.zeros(N + 1, dtype=torch.int32, device=DEV), ints([0])
    cu, kv[0] = ints([0, prompt]), prompt
    vc.vc_pages_reserve(cache, pool, cu, kv[:1], table[:1], prompt, dev_status=status)
    vc.vc_cache_append_rope(None, whole[0].K[:prompt].to(DEV), whole[0].V[:prompt].to(DEV), cache, cu, kv[:1], table[:1], rope)
    vc.vc_pages_fork(cache, pool, table[:1], kv[:1], ints([0] * N), table[1:], kv[1:], dev_status=status)
    one, groups, prefix = torch.arange(N + 1, dtype=torch.int32, device=DEV), ints([0, N]), ints([prompt])
    Q = torch.zeros((N, H * G, d), dtype=torch.bfloat16, device=DEV)
    K, V = (torch.zeros((N, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        kv[1:] += 1
        vc.vc_pages_reserve(cache, pool, one, kv[1:], table[1:], N, dev_status=status)
        q = vc.vc_cache_append_rope(Q, K, V, cache, one, kv[1:], table[1:], rope, dev_status=status)
        return (q, *vc.vc_attn_paged_shared(q, cache, one, kv[1:], table[1:], groups, prefix, max_q=1, max_rows=N, dev_status=status))

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
    for i, c in enumerate(whole):
        # each sequence by itself, from what its own pages hold
        c.table, c.pages = table[1 + i:2 + i].cpu(), pages
        c.Q[prompt:] = torch.stack([o[0][i] for o in outs]).cpu()
        for k, v in cache.items():
            setattr(c, k, v.cpu())
        O, tol, lse, told = c.attend(c.cache())
        got = [torch.stack([o[j][i] for o in outs]).double().cpu() for j in (1, 2)]
        assert torch.all((got[0] - O[prompt:]).abs() <= tol[prompt:]) and torch.all((got[1] - lse[prompt:]).abs() <= told[prompt:])


def test_captured_graphs_do_not_share():
    """Two graphs captured in turn, with other groups put into their buffers, replayed one after the other."""
    shapes = [dict(groups=[(200, [(9, 1)] * 4), (90, [(3, 1)] * 2)]), dict(groups=[(30, [(70, 1)]), (300, [(2, 1)] * 5)])]
    cases = [Shared(H=2, G=4, seed=50 + i, cols=2200, **kw) for i, kw in enumerate(shapes)]
    pages = max(c.pages for c in cases)
    graphs = []
    for c in cases:
        buf = [t.to(DEV) for t in (c.Q, *c.args("cpu"), *c.shared_args("cpu"))]
        cache = vc.alloc_cache(pages, 16, 2, 128, DEV)
        vc.vc_attn_paged_shared(buf[0], cache, *buf[1:], max_q=1, max_rows=6)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = vc.vc_attn_paged_shared(buf[0], cache, *buf[1:], max_q=1, max_rows=6)
        graphs.append((graph, out, buf, cache))
    for which in (0, 1, 1, 0):
        for k, (graph, out, buf, cache) in enumerate(graphs):
            c = cases[which ^ k]
            for t, new in zip(buf, (c.Q, *c.args("cpu"), *c.shared_args("cpu"))):
                t.copy_(new)
            for name_, v in c.cache().items():
                cache[name_][:c.pages].copy_(v)
            graph.replay()
        torch.cuda.synchronize()
        for k, (graph, out, buf, cache) in enumerate(graphs):
            cases[which ^ k].check(out, cases[which ^ k].cache())

"""GPU: the paged FP8 cache and its attention against their definitions in fp64 (paged_case.py).

Codes and scales bit-exact; values read back bit-exact; attention within the
bars that Case.attend derives."""
import math

import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import LOG2E, Case, quantize

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def same_cache(got, want):
    for k in ("K8", "V8"):
        assert torch.equal(got[k].cpu(), want[k]), k
    for k in ("sk", "sv"):
        x = got[k].cpu()
        assert torch.equal(torch.isnan(x), torch.isnan(want[k])), k
        assert torch.equal(torch.nan_to_num(x, -1.0), torch.nan_to_num(want[k], -1.0)), k


def attend(c, cache=None, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw.setdefault("max_q", max(c.n))
    out = vc.vc_attn_paged(c.Q.to(DEV), cache or c.cache(DEV), *c.args(DEV), dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    return out


# ---------------------------------------------------------------- writing and reading

CACHE_CASES = [dict(n=[1], kv=[1], H=1, d=64), dict(n=[1, 1, 1], kv=[1, 17, 128], H=8), dict(n=[0, 5, 0, 40, 0], kv=[0, 9, 33, 40, 7], H=3, d=64, page=32),
               dict(n=[300], kv=[500], H=5, page=128), dict(n=[3] * 70, kv=[50] * 70, H=2, d=64, tail=5), dict(n=[16, 256], kv=[16, 256], H=1, page=256)]


@pytest.mark.parametrize("case", CACHE_CASES, ids=lambda c: "B%d_H%d" % (len(c["n"]), c["H"]))
def test_append_bitexact(case):
    c = Case(seed=1, **case)
    want = c.appended()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV), dev_status=status)
    same_cache(got, want)
    assert int(status) == 0


@pytest.mark.parametrize("case", CACHE_CASES, ids=lambda c: "B%d_H%d" % (len(c["n"]), c["H"]))
def test_read_bitexact(case):
    c = Case(seed=2, **case)
    K, V = (torch.full_like(t, 7.0) for t in (c.K, c.V))
    want = c.read(c.cache(), K, V)
    got = vc.vc_cache_read(c.cache(DEV), *c.args(DEV), c.T, K=K.to(DEV), V=V.to(DEV))
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)     # rows behind the last sequence included: still 7


def test_append_extreme_rows():
    """Zero rows, tiny rows, the largest numbers, subnormals, NaN and infinities in single channels."""
    c = Case(n=[9], kv=[20], H=2, seed=3)
    c.K[0] = 0
    c.K[1] = 2.0 ** -101
    c.K[2, :, ::2] = 3e38
    c.K[3, 0, 5] = math.nan
    c.K[4, 1, 127] = -math.inf
    c.V[5] = -0.0
    c.V[6] = 2.0 ** -100
    c.V[7, :, 3] = math.inf
    c.V[8] *= 1e-40
    want = c.appended()
    got = vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV))
    same_cache(got, want)


@pytest.mark.parametrize("order", ["token", "joint", "strided"])
def test_cache_layouts(order):
    """Token-major pages, K and V as halves of one pool, and pages with gaps: same results."""
    c = Case(n=[5, 40], kv=[70, 41], H=3, G=2, d=64, page=32, seed=4)
    base = c.cache(DEV)
    if order == "token":
        cache = {k: base[k].transpose(1, 2).contiguous().transpose(1, 2) if k in ("K8", "V8") else base[k] for k in base}
    elif order == "joint":
        codes = torch.stack([base["K8"], base["V8"]], 1)
        scales = torch.stack([base["sk"], base["sv"]], 1)
        cache = dict(K8=codes[:, 0], V8=codes[:, 1], sk=scales[:, 0], sv=scales[:, 1])
    else:
        cache = {}
        for k in ("K8", "V8"):
            big = torch.full((c.pages, c.H + 1, c.page + 3, c.d + 16), 0x7F, dtype=torch.uint8, device=DEV)
            cache[k] = big[:, 1:, 2:2 + c.page, 16:]
            cache[k].copy_(base[k])
        for k in ("sk", "sv"):
            big = torch.full((c.pages, c.H + 2, c.page + 4), math.nan, device=DEV)
            cache[k] = big[:, :c.H, 4:]
            cache[k].copy_(base[k])
    vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), cache, *c.args(DEV))
    want = c.appended()
    same_cache(cache, want)
    K, V = vc.vc_cache_read(cache, *c.args(DEV), c.T)
    wk, wv = c.read(want, c.K, c.V)
    assert torch.equal(K.cpu(), wk) and torch.equal(V.cpu(), wv)
    c.check(attend(c, cache), want)


def test_strided_rows():
    """Q, K, V and O as views of packed [T, H, 3, d] tensors."""
    c = Case(n=[20, 3], kv=[50, 3], H=3, seed=5)
    packed = torch.stack([c.Q, c.K, c.V], 2).to(DEV)
    cache = c.cache(DEV)
    vc.vc_cache_append(packed[:, :, 1], packed[:, :, 2], cache, *c.args(DEV))
    want = c.appended()
    same_cache(cache, want)
    out = torch.full((c.T, 3, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got = vc.vc_attn_paged(packed[:, :, 0], cache, *c.args(DEV), O=out[:, :, 1])
    c.check(got, want)
    assert torch.all(out[:, :, 0] == 7.0)
    back = torch.full((c.T, 3, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    back2 = torch.full_like(back, 7.0)
    vc.vc_cache_read(cache, *c.args(DEV), c.T, K=back[:, :, 0], V=back2[:, :, 0])
    wk, wv = c.read(want, c.K, c.V)
    assert torch.equal(back[:, :, 0].cpu(), wk) and torch.equal(back2[:, :, 0].cpu(), wv)
    assert torch.all(back[:, :, 1] == 7.0) and torch.all(back2[:, :, 1] == 7.0)


# ---------------------------------------------------------------- attention

ATTN_CASES = [
    dict(n=[1], kv=[1], H=1, d=64), dict(n=[1], kv=[1]), dict(n=[1], kv=[219], H=2, d=64),
    dict(n=[1, 1, 1, 1], kv=[127, 128, 129, 1], H=8, G=4),
    dict(n=[1] * 9, kv=[2000, 1, 16, 17, 900, 128, 256, 257, 3], H=2, G=5, d=64),
    dict(n=[1, 0, 1], kv=[4000, 100, 700], H=1, G=8, page=128),
    dict(n=[1], kv=[600], H=1, G=20), dict(n=[1, 1], kv=[300, 20], H=1, G=70, d=64, page=64),
    dict(n=[3, 7, 1, 0, 5], kv=[300, 7, 40, 0, 129], H=2, G=3, d=64, page=32),
    dict(n=[9, 2], kv=[1000, 130], H=2, G=4, page=64),
    dict(n=[128], kv=[128]), dict(n=[256], kv=[256], d=64), dict(n=[130, 257, 40], kv=[130, 700, 41], H=2, page=32),
    dict(n=[200, 0, 1, 100], kv=[1000, 0, 500, 100], H=2, G=3, d=64, page=256),
    dict(n=[513], kv=[1200], H=1, G=2, page=128), dict(n=[33], kv=[2049], H=1, G=11, d=64),
]
MASKS = [dict(causal=1), dict(causal=0), dict(causal=1, window=1), dict(causal=1, window=130), dict(causal=0, window=70)]


@pytest.mark.parametrize("case", ATTN_CASES, ids=lambda c: "n%d_kv%d_H%d_G%d_d%d" % (max(c["n"]), max(c["kv"]), c.get("H", 2), c.get("G", 1), c.get("d", 128)))
@pytest.mark.parametrize("mask", MASKS, ids=lambda m: "c%d_w%d" % (m["causal"], m.get("window", 0)))
def test_attention(case, mask):
    c = Case(seed=6, **case)
    c.check(attend(c, **mask), c.cache(), **mask)


@pytest.mark.parametrize("max_q", [0, 1, 60, 5000])
def test_max_q_is_a_hint(max_q):
    c = Case(n=[1, 90, 0, 7], kv=[300, 400, 5, 7], H=2, G=3, seed=7)
    c.check(attend(c, max_q=max_q), c.cache())


@pytest.mark.parametrize("n,G", [(1, 4), (70, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_peaked_scores_and_scales(n, G, d):
    """Large scores (one key takes all), another softmax scale, and values of very different sizes."""
    c = Case(n=[n, n], kv=[700, 333], H=2, G=G, d=d, seed=8, qmul=6.0)
    g = torch.Generator().manual_seed(1)
    c.sv *= torch.exp2(torch.randint(-30, 30, c.sv.shape, generator=g).float())
    c.check(attend(c), c.cache())
    c.check(attend(c, softmax_scale=0.5), c.cache(), scale=0.5)


@pytest.mark.parametrize("n,G", [(1, 4), (70, 1)])
def test_zero_rows_of_the_cache(n, G):
    """Tokens whose keys or values are all zero (scale 0), some of them all that a row sees."""
    c = Case(n=[n, n, n], kv=[300, 200, 100], H=2, G=G, seed=9)
    zero = torch.rand(c.sv.shape, generator=torch.Generator().manual_seed(2)) < 0.5
    c.V8[zero], c.sv[zero] = 0, 0.0
    c.K8[zero.flip(0)], c.sk[zero.flip(0)] = 0, 0.0
    for p in range(0, 100, c.page):
        c.V8[c.table[2, p // c.page]], c.sv[c.table[2, p // c.page]] = 0, 0.0
    for b, f in ((0, 1e-6), (1, 1e6)):
        for p in range(0, c.kv[b], c.page):
            c.sv[c.table[b, p // c.page]] *= f
    got = attend(c)
    c.check(got, c.cache())
    assert torch.all(got[0][2 * n:] == 0)


@pytest.mark.parametrize("n,G", [(1, 4), (90, 1)])
def test_garbage_behind_the_last_token(n, G):
    """What lies in the pages behind kv_len (NaN codes, NaN and infinite scales) is never seen."""
    c = Case(n=[n, n], kv=[301, 99], H=2, G=G, page=64, seed=10)
    clean = c.cache()
    used = torch.zeros(c.sk.shape, dtype=torch.bool)
    for b in range(2):
        for p in range(c.kv[b]):
            used[c.table[b, p // c.page], :, p % c.page] = True
    for k in ("K8", "V8"):
        getattr(c, k)[~used] = 0x7F
    c.sk[~used], c.sv[~used] = math.nan, math.inf
    got = attend(c)
    c.check(got, clean)
    c.check(attend(c, causal=0), clean, causal=0)


@pytest.mark.parametrize("n,G", [(3, 2), (200, 1)])
def test_nan_token_spoils_only_rows_that_see_it(n, G):
    c = Case(n=[n], kv=[n + 100], H=2, G=G, seed=11)
    c.K[n // 2, 0, 3] = math.nan
    c.V[n - 1, 1, 3] = math.inf
    cache = vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV))
    O, lse = attend(c, cache)
    nan = torch.isnan(O.float()).all(-1).cpu()
    want = torch.zeros((n, 2 * G), dtype=torch.bool)
    want[n // 2:, :G] = True
    want[n - 1:, G:] = True
    assert torch.equal(nan, want) and torch.equal(torch.isnan(O.float()).any(-1).cpu(), want)
    clean = Case(n=[n], kv=[n + 100], H=2, G=G, seed=11)
    ref = clean.attend(clean.appended())
    off = (O.double().cpu() - ref[0]).abs()
    assert torch.all(off[~want] <= ref[1][~want])


@pytest.mark.parametrize("n", [[2, 40], [200, 150]])
def test_rows_without_keys(n):
    """kv_len below n: positions below 0 see nothing under a causal mask; kv_len 0 sees nothing at all."""
    c = Case(n=n, kv=[n[0], n[1]], H=2, G=2, seed=12)
    kv = torch.tensor([0, n[1] - 30], dtype=torch.int32)
    cache = c.cache(DEV)
    O = torch.full((c.T, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    O, lse = vc.vc_attn_paged(c.Q.to(DEV), cache, c.cu.to(DEV), kv.to(DEV), c.table.to(DEV), max_q=max(n), O=O)
    c.kv = kv.tolist()
    c.check((O, lse), c.cache())
    empty = n[0] + 30
    assert torch.all(O[:empty] == 0) and torch.all(lse[:empty] == -math.inf) and torch.all(torch.isfinite(lse[empty:]))


@pytest.mark.parametrize("n", [[1, 1], [150, 40]])
def test_rows_of_no_sequence_stay(n):
    c = Case(n=n, kv=[200, 60], H=2, tail=20, seed=13)
    O = torch.full((c.T, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.T, 2), 7.0, device=DEV)
    attend(c, O=O, lse=lse)
    c.check((O, lse), c.cache())
    assert torch.all(O[sum(n):] == 7.0) and torch.all(lse[sum(n):] == 7.0)


@pytest.mark.parametrize("n,G", [(1, 4), (90, 1)])
def test_shared_pages(n, G):
    """Two sequences whose prefixes lie in the same pages."""
    c = Case(n=[n, n], kv=[256, 230], H=2, G=G, seed=14)
    c.table[1, :4] = c.table[0, :4]
    c.check(attend(c), c.cache())


def test_no_rows():
    c = Case(n=[0, 0], kv=[30, 0], H=2, seed=15)
    cache, args = c.cache(DEV), c.args(DEV)
    vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), cache, *args)
    same_cache(cache, c.cache())
    O, lse = vc.vc_attn_paged(c.Q.to(DEV), cache, *args)
    K, V = vc.vc_cache_read(cache, *args, 0)
    assert O.shape == (0, 2, 128) and lse.shape == (0, 2) and K.shape == V.shape == (0, 2, 128)


def test_many_sequences():
    """More sequences than a block has threads, most with a single token, some with none."""
    n = [(b * 7) % 3 for b in range(1500)]
    c = Case(n=n, kv=[max(m, (b * 37) % 50) for b, m in enumerate(n)], H=1, G=2, d=64, seed=16)
    cache = vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV))
    want = c.appended()
    same_cache(cache, want)
    K, V = vc.vc_cache_read(cache, *c.args(DEV), c.T)
    wk, wv = c.read(want, c.K, c.V)
    assert torch.equal(K.cpu(), wk) and torch.equal(V.cpu(), wv)
    c.check(attend(c, cache), want)
    c.check(attend(c, cache, max_q=500), want)


@pytest.mark.parametrize("n", [1, 100])
def test_pages_beyond_two_to_the_31(n):
    """A pool of over 2^31 bytes of codes, with the sequence in its last pages."""
    c = Case(n=[n], kv=[150], H=1, d=128, page=16, seed=17)
    pages = (1 << 31) // (16 * 128) + 100
    cache = vc.alloc_cache(pages, 16, 1, 128, DEV)
    for k in cache:
        cache[k][-c.pages:] = getattr(c, k).to(DEV)
    table = torch.where(c.table >= 0, c.table + (pages - c.pages), c.table)
    vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), cache, c.cu.to(DEV), c.kv_len.to(DEV), table.to(DEV))
    want = c.appended()
    same_cache({k: v[-c.pages:] for k, v in cache.items()}, want)
    assert not any(bool(v[:-c.pages].any()) for v in cache.values())
    got = vc.vc_attn_paged(c.Q.to(DEV), cache, c.cu.to(DEV), c.kv_len.to(DEV), table.to(DEV), max_q=n)
    c.check(got, want)
    K, V = vc.vc_cache_read(cache, c.cu.to(DEV), c.kv_len.to(DEV), table.to(DEV), c.T)
    wk, wv = c.read(want, c.K, c.V)
    assert torch.equal(K.cpu(), wk) and torch.equal(V.cpu(), wv)


def test_pages_that_are_not_there():
    """Page numbers out of range: their tokens are unseen, unwritten, read as zeros, and reported."""
    for n, G in ((1, 2), (80, 1)):
        c = Case(n=[n, n], kv=[250, 300], H=2, G=G, seed=18)
        c.table[0, 2], c.table[0, 7], c.table[1, 5] = -1, c.pages, 2 ** 31 - 1
        c.table[1, (300 - 1) // 16] = -2 ** 31
        cache, args = c.cache(DEV), c.args(DEV)
        for i, call in enumerate((lambda s: vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), cache, *args, dev_status=s),
                                  lambda s: vc.vc_cache_read(cache, *args, c.T, dev_status=s),
                                  lambda s: vc.vc_attn_paged(c.Q.to(DEV), cache, *args, max_q=n, dev_status=s))):
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            out = call(status)
            assert int(status) == 1, i
            want = c.appended()
            if i == 0:
                same_cache(cache, want)
            elif i == 1:
                wk, wv = c.read(want, c.K, c.V)
                assert torch.equal(out[0].cpu(), wk) and torch.equal(out[1].cpu(), wv)
            else:
                c.check(out, want)


def test_broken_offsets_and_lengths_are_reported():
    """cu that decreases or leaves 0 .. T, kv_len out of range: reported, and nothing outside is touched."""
    c = Case(n=[4, 4, 4], kv=[20, 30, 40], H=2, seed=19)
    for cu, kv in (([0, 4, 2, 12], [20, 30, 40]), ([-3, 4, 8, 12], [20, 30, 40]), ([0, 4, 8, 2 ** 31 - 1], [20, 30, 40]),
                   ([0, 4, 8, 12], [20, -1, 40]), ([0, 4, 8, 12], [20, 30, 2 ** 31 - 1])):
        args = (torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(kv, dtype=torch.int32, device=DEV), c.table.to(DEV))
        for n in (4, 500):
            cache = c.cache(DEV)
            for call in (lambda s: vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), cache, *args, dev_status=s),
                         lambda s: vc.vc_cache_read(cache, *args, c.T, dev_status=s),
                         lambda s: vc.vc_attn_paged(c.Q.to(DEV), cache, *args, max_q=n, dev_status=s)):
                status = torch.zeros(1, dtype=torch.int32, device=DEV)
                call(status)
                assert int(status) == 1, (cu, kv)


# ---------------------------------------------------------------- as used: together, on streams, in graphs

@pytest.mark.parametrize("G,d", [(1, 128), (4, 64)])
def test_generation_in_chunks_matches_one_pass(G, d):
    """A sequence written and attended chunk by chunk, then token by token, gives what one causal pass gives,
    and reading it back gives the values attended to."""
    H, N = 2, 333
    whole = Case(n=[N], kv=[N], H=H, G=G, d=d, seed=20)
    want = whole.appended()
    O_ref, tol, _, _ = whole.attend(want)
    cache = whole.cache(DEV)
    outs, at = [], 0
    for n in [128, 100, 90, 7] + [1] * 8:
        cu, kv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, n], [at + n]))
        q, k, v = (t[at:at + n].to(DEV) for t in (whole.Q, whole.K, whole.V))
        vc.vc_cache_append(k, v, cache, cu, kv, whole.table.to(DEV))
        outs.append(vc.vc_attn_paged(q, cache, cu, kv, whole.table.to(DEV), max_q=n)[0])
        at += n
    assert at == N
    same_cache(cache, want)
    assert torch.all((torch.cat(outs).double().cpu() - O_ref).abs() <= tol)
    K, V = vc.vc_cache_read(cache, *whole.args(DEV), N)
    assert torch.equal(K.cpu(), whole.read(want, whole.K, whole.V)[0])


def test_same_call_same_bits_on_another_stream():
    for n, G in ((1, 4), (200, 1)):
        c = Case(n=[n] * 3, kv=[2000, 700, 300], H=2, G=G, seed=21)
        cache, args, Q = c.cache(DEV), c.args(DEV), c.Q.to(DEV)
        first = vc.vc_attn_paged(Q, cache, *args, max_q=n)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        given = vc.vc_attn_paged(Q, cache, *args, max_q=n, stream=side)
        with torch.cuda.stream(side):
            inside = [vc.vc_attn_paged(Q, cache, *args, max_q=n) for _ in range(3)]
        side.synchronize()
        for other in [given] + inside:
            assert same_bits(first[0], other[0]) and same_bits(first[1], other[1])


def test_captured_step_replayed_on_new_lengths():
    """append + attend in one graph, replayed with other tokens, lengths and page tables in the same buffers;
    two graphs captured in turn do not disturb each other."""
    for n, G in ((1, 4), (70, 1)):
        cases = [Case(n=[n, n], kv=kv, H=2, G=G, seed=22 + i, spare=0, cols=60) for i, kv in enumerate(([500, 400], [900, 70], [80, 800]))]
        pages = max(c.pages for c in cases)
        graphs = []
        for c in cases[:2]:
            buf = dict(Q=c.Q.to(DEV), K=c.K.to(DEV), V=c.V.to(DEV), cu=c.cu.to(DEV), kv=c.kv_len.to(DEV), table=c.table.to(DEV))
            cache = vc.alloc_cache(pages, 16, 2, 128, DEV)

            def step():
                vc.vc_cache_append(buf["K"], buf["V"], cache, buf["cu"], buf["kv"], buf["table"])
                return vc.vc_attn_paged(buf["Q"], cache, buf["cu"], buf["kv"], buf["table"], max_q=n)
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
            graphs.append((graph, out, buf, cache))
        for order in ((0, 1, 2, 0), (2, 1)):
            for which in order:
                c = cases[which]
                want = c.appended()
                for graph, out, buf, cache in graphs:
                    for k, t in (("Q", c.Q), ("K", c.K), ("V", c.V), ("kv", c.kv_len), ("table", c.table)):
                        buf[k].copy_(t)
                    for k, t in c.cache().items():
                        cache[k][:c.pages].copy_(t)
                    graph.replay()
                torch.cuda.synchronize()
                for _, out, _, _ in graphs:
                    c.check(out, want)


def test_scale_of_new_values_reaches_the_output():
    """quantize() of the definition and the kernel agree on what a token's value is: one key, one query."""
    c = Case(n=[1], kv=[1], H=4, seed=30)
    cache = vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV))
    O, lse = attend(c, cache)
    codes, scale = quantize(c.V)
    value = codes.view(torch.float8_e4m3fn).float() * scale[..., None]
    assert torch.all((O.float().cpu() - value).abs() <= 2.0 ** -8 * value.abs() + 2.0 ** -20 * value.abs())


@pytest.mark.parametrize("n,G", [(1, 4), (90, 1), (300, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_heavy_tokens_without_values(n, G, d):
    """Tokens whose values are all zero take nearly all of the weight: the others' share stays right as
    long as they have no more than 2^88 times the others' weights times value scales; beyond, it may
    vanish, and nothing overflows."""
    c = Case(n=[n, n], kv=[900, 400], H=2, G=G, d=d, seed=33)
    zero = torch.rand(c.sv.shape, generator=torch.Generator().manual_seed(3)) < 0.5
    c.V8[zero], c.sv[zero] = 0, 0.0
    keys = c.sk.clone()
    for times in (14.0, 120.0):
        c.sk = torch.where(zero, keys * times, keys)
        cache = c.cache()
        over = torch.zeros(c.T, 2 * G, dtype=torch.float64)   # log2 of that ratio
        for b in range(2):
            last = c.kv[b] - n + torch.arange(n)
            for h in range(2):
                (k, ks, _), (_, vs, _) = (c.sequence(cache, a, e, b, h) for a, e in (("K8", "sk"), ("V8", "sv")))
                unseen = torch.arange(c.kv[b]) > last[:, None]
                for j in range(G):
                    q = c.Q.double()[b * n:(b + 1) * n, h * G + j]
                    s = (q @ (k * ks[:, None]).T / math.sqrt(d) * LOG2E).masked_fill(unseen, -math.inf)
                    over[b * n:(b + 1) * n, h * G + j] = s[:, vs == 0].amax(-1) - (s + vs.log2())[:, vs > 0].amax(-1)
        O, lse = (t.double().cpu() for t in attend(c))
        O_ref, tol, lse_ref, told = c.attend(cache)
        assert torch.all((lse - lse_ref).abs() <= told)
        within = over <= 88
        assert torch.all((O - O_ref).abs()[within] <= tol[within])
        assert torch.isfinite(O).all() and torch.all(O[over > 120].abs() <= 1e-30)
        assert within.any() if times < 100 else (over > 120).any()


def test_calls_of_two_host_threads():
    """Two threads, each with its own stream, cache and outputs, at the same time."""
    import threading
    cases = [Case(n=[n] * 2, kv=[800, 300], H=2, G=G, seed=40 + n) for n, G in ((1, 4), (150, 1))]
    got, errors = [[], []], []

    def work(i):
        try:
            c, stream = cases[i], torch.cuda.Stream()
            with torch.cuda.stream(stream):
                cache, args, Q, K, V = c.cache(DEV), c.args(DEV), c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV)
                for _ in range(20):
                    vc.vc_cache_append(K, V, cache, *args)
                    got[i].append(vc.vc_attn_paged(Q, cache, *args, max_q=max(c.n)))
            stream.synchronize()
        except Exception as e:                              # carried to the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for c, outs in zip(cases, got):
        c.check(outs[0], c.appended())
        for O, lse in outs[1:]:
            assert same_bits(O, outs[0][0]) and same_bits(lse, outs[0][1])


@pytest.mark.parametrize("n,kv", [([3, 9], [2, 40]), ([200, 40], [150, 500])])
def test_windows_of_any_size(n, kv):
    """The largest window that a C int holds and larger ones see what no window sees, with rows before the
    first key in the same tile."""
    c = Case(n=n, kv=kv, H=2, G=2, seed=50)
    whole = attend(c)
    c.check(whole, c.cache())
    for window in (2 ** 31 - 1, 2 ** 31 - 50, 2 ** 32 + 3, 2 ** 40):
        got = attend(c, window=window)
        assert same_bits(got[0], whole[0]) and same_bits(got[1], whole[1]), window
    got = attend(c, max_q=2 ** 32 + 1)
    c.check(got, c.cache())


@pytest.mark.parametrize("n,G,d", [(1, 4, 128), (100, 1, 128), (300, 1, 64)])
def test_without_lse_and_with_given_outputs(n, G, d):
    """Strided O, a workspace kept by the caller, and the C entry without lse."""
    c = Case(n=[n, n], kv=[500, 310], H=2, G=G, d=d, seed=51)
    cache, args, Q = c.cache(DEV), c.args(DEV), c.Q.to(DEV)
    want = vc.vc_attn_paged(Q, cache, *args, max_q=n)
    c.check(want, c.cache())
    big = torch.full((c.T, 2 * G + 1, d + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    O = big[:, :2 * G, :d]
    ws = torch.empty(vc.attn_paged_workspace_bytes(cache, 2 * G, 2, c.T, n), dtype=torch.uint8, device=DEV)
    for _ in range(2):
        vc.vc_attn_paged(Q, cache, *args, max_q=n, O=O, workspace=ws)
    assert same_bits(O, want[0])
    assert torch.all(big[:, 2 * G] == 3.0) and torch.all(big[:, :, d:] == 3.0)
    O2 = torch.zeros_like(Q)
    shape, batch = vc.cache_shape_of(cache), vc._batch_of(*args, c.T, 0)
    rc = vc.lib().vc_attn_paged(Q.data_ptr(), 2 * G * d, d, 2 * G, shape, cache["K8"].data_ptr(), cache["sk"].data_ptr(),
                                cache["V8"].data_ptr(), cache["sv"].data_ptr(), batch, 0.0, 1, 0, n, O2.data_ptr(),
                                2 * G * d, d, None, ws.data_ptr(), ws.numel(), None,
                                torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and same_bits(O2, want[0])

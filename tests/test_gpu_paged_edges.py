"""GPU: the ends of what the paged cache's calls take, against the definitions in fp64 (paged_case.py)."""
import math

import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import LOG2E, Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TILES = [(1, 4), (3, 4), (5, 5), (90, 1), (150, 2)]    # (tokens, query heads a key head): tiles of 8, 16, 32, 128, 256 rows


def attend(c, cache=None, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw.setdefault("max_q", max(c.n))
    out = vc.vc_attn_paged(c.Q.to(DEV), cache or c.cache(DEV), *c.args(DEV), dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    return out


@pytest.mark.parametrize("n,G", [(1, 4), (200, 1)])
def test_calls_on_two_streams_at_once(n, G):
    """Calls on the current stream and, without a wait, on another one: each has its own workspace and outputs."""
    cases = [Case(n=[n] * 3, kv=[4000, 700, 300], H=2, G=G, seed=70 + i) for i in range(2)]
    data = [(c.Q.to(DEV), c.cache(DEV), *c.args(DEV)) for c in cases]
    want = [vc.vc_attn_paged(*d, max_q=n) for d in data]
    back = [vc.vc_cache_read(*d[1:], c.T) for c, d in zip(cases, data)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(30):
        here = [vc.vc_attn_paged(*data[0], max_q=n) for _ in range(3)]
        there = vc.vc_attn_paged(*data[1], max_q=n, stream=side)
        kv = vc.vc_cache_read(*data[1][1:], cases[1].T, stream=side)
        here.append(vc.vc_attn_paged(*data[0], max_q=n))
        torch.cuda.synchronize()
        for got, ref in [(x, want[0]) for x in here] + [(there, want[1]), (kv, back[1])]:
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("n,G", TILES)
@pytest.mark.parametrize("d", [64, 128])
def test_scale_zero_is_value_zero(n, G, d):
    """A value is code * scale: codes under a scale of 0 count in the sum of weights and nowhere else."""
    c = Case(n=[n, n], kv=[600, 333], H=2, G=G, d=d, seed=60)
    c.sv[torch.rand(c.sv.shape, generator=torch.Generator().manual_seed(4)) < 0.5] = 0.0
    for p in range(0, 333, c.page):
        c.sv[c.table[1, p // c.page], 1] = 0.0
    got = attend(c)
    c.check(got, c.cache())
    assert torch.all(got[0][n:, G:] == 0) and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("n,d", [(90, 64), (90, 128), (200, 64), (200, 128)])
def test_weights_before_a_large_rise(n, d):
    """A key whose product stays just below the bound of P sv, then one of 2^10.5 times its weight in the same
    unit of keys, with values on different channels."""
    B, L = 80, 384                                       # more items than CTAs: some lie whole in one
    c = Case(n=[n] * B, kv=[L] * B, H=2, d=d, page=128, seed=61, spare=0)
    c.Q[:] = 0
    c.Q[..., 0] = 1.0
    c.K8[:], c.V8[:], c.sv[:], c.sk[:] = 0, 0, 1.0, 0.0
    c.K8[..., 0] = 0x38                                   # 1.0
    c.V8[..., 2] = 0x38
    last = c.table[:, 2].long()                           # the third unit of each sequence
    for key, score, channel in ((5, 14.5, 0), (5 + 64, 25.0, 1)):
        c.sk[last, :, key] = score * math.log(2.0)        # scores in log2 units, 0 elsewhere
        c.V8[last, :, key] = 0
        c.V8[last, :, key, channel] = 0x38
    O, lse = attend(c, causal=0, softmax_scale=1.0)
    one = Case(n=[n], kv=[L], H=2, d=d, page=128, seed=61, spare=0)   # all sequences are the same
    one.Q, one.table = c.Q[:n], torch.arange(3, dtype=torch.int32)[None]
    for k in ("K8", "sk", "V8", "sv"):
        setattr(one, k, getattr(c, k)[c.table[0].long()])
    for b in range(B):
        one.check((O[b * n:(b + 1) * n], lse[b * n:(b + 1) * n]), one.cache(), causal=0, scale=1.0)


def sized(n, G, d, exponents, order):
    """Values times 2^e, down to what vc_cache_append still writes (2^-100): e mixed, or in the keys' order."""
    c = Case(n=[n, n], kv=[1700, 700], H=2, G=G, d=d, seed=62)
    e = torch.tensor(exponents, dtype=torch.float32)
    if order == "mixed":
        c.sv *= torch.exp2(e)[torch.randint(len(exponents), c.sv.shape, generator=torch.Generator().manual_seed(5))]
    else:
        for b in range(2):
            step = torch.arange(c.kv[b]) * len(exponents) // c.kv[b]
            for p in range(c.kv[b]):
                c.sv[c.table[b, p // c.page], :, p % c.page] *= 2.0 ** float(e[step[p]])
    return c


SIZES = [((-100,), "mixed"), ((-90,), "mixed"), ((-100, -60, 0, 100), "mixed"), ((-100, -30, 40, 100), "rising"), ((100, 40, -30, -100), "falling")]


@pytest.mark.parametrize("n,G", TILES[3:])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponents,order", SIZES, ids=str)
def test_values_of_any_size_many_rows(n, G, d, exponents, order):
    c = sized(n, G, d, exponents, order)
    for mask in (dict(), dict(causal=0, window=300)):
        c.check(attend(c, **mask), c.cache(), **mask)


@pytest.mark.parametrize("n,G", TILES[:3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponents,order", SIZES, ids=str)
def test_values_of_any_size_few_rows(n, G, d, exponents, order):
    c = sized(n, G, d, exponents, order)
    for mask in (dict(), dict(causal=0, window=300)):
        c.check(attend(c, **mask), c.cache(), **mask)


@pytest.mark.parametrize("n", [1, 90, 150])
def test_many_small_values_above_the_first(n):
    """Long sequences of values near 2^-100 whose weights lie a little above those of the first keys."""
    H, d, page, L = 304, 64, 256, 16384                   # more items than CTAs: some lie whole in one
    pages = L // page
    g = torch.Generator().manual_seed(6)
    V8 = (torch.randint(0x30, 0x40, (pages, page, d), generator=g) + 128 * torch.randint(2, (pages, page, d), generator=g)).to(torch.uint8)
    s = torch.full((L,), 7.4)
    s[:256] = 0.0                                         # log2 units
    cache = vc.alloc_cache(pages, page, H, d, DEV)
    cache["K8"][..., 0] = 0x38                            # 1.0
    cache["V8"].copy_(V8[:, None])
    cache["sk"].copy_((s * math.log(2.0)).view(pages, 1, page))
    cache["sv"].fill_(2.0 ** -108)
    Q = torch.zeros((n, H, d), dtype=torch.bfloat16, device=DEV)
    Q[..., 0] = 1.0
    cu, kv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, n], [L]))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    O, lse = vc.vc_attn_paged(Q, cache, cu, kv, table, softmax_scale=1.0, causal=0, max_q=n)
    sd = cache["sk"][:, 0].double().reshape(-1)
    p = torch.softmax(sd, 0)
    v = V8.to(DEV).view(torch.float8_e4m3fn).double().reshape(L, d) * 2.0 ** -108
    # P to fp16, O to bf16; the scores' products, scaling and exponential; sums of L terms
    want, rel = p @ v, 2.0 ** -11 + 3 * (2.0 ** -21 * 24 + 2 * (d + 16) * 2.0 ** -24 * 8) + (L + 64) * 2.0 ** -24
    tol = 2.0 ** -8 * want.abs() + rel * (p @ v.abs())
    assert torch.all((O.double() - want).abs() <= tol)
    assert torch.all((lse.double() - torch.logsumexp(sd, 0)).abs() <= rel)


@pytest.mark.parametrize("n,G", TILES)
@pytest.mark.parametrize("times", [20.0, 24.0])
def test_heavy_tokens_without_values_to_the_stated_end(n, G, times):
    """Tokens whose values are all zero with up to 2^110 times the others' weight times value scale."""
    c = Case(n=[n], kv=[900], H=1, G=G, d=64, seed=33)
    zero = torch.rand(c.sv.shape, generator=torch.Generator().manual_seed(3)) < 0.5
    c.V8[zero], c.sv[zero] = 0, 0.0
    c.sk = torch.where(zero, c.sk * times, c.sk)
    cache = c.cache()
    (k, ks, _), (_, vs, _) = (c.sequence(cache, a, e, 0, 0) for a, e in (("K8", "sk"), ("V8", "sv")))
    s = torch.einsum("tjd,kd->tjk", c.Q.double(), k * ks[:, None]) / math.sqrt(64) * LOG2E
    s.masked_fill_((torch.arange(900) > 900 - n + torch.arange(n)[:, None])[:, None], -math.inf)
    within = s[..., vs == 0].amax(-1) - (s + vs.log2())[..., vs > 0].amax(-1) <= 110
    O, lse = (t.double().cpu() for t in attend(c))
    want, tol, lse_want, lse_tol = c.attend(cache)
    assert within.any() and torch.isfinite(O).all()
    assert torch.all((O - want).abs()[within] <= tol[within]) and torch.all((lse - lse_want).abs() <= lse_tol)


@pytest.mark.parametrize("n,G", TILES)
def test_queries_that_are_not_finite(n, G):
    """They give NaN whatever the keys' signs, and only in their own rows; a row that sees no key stays empty."""
    c = Case(n=[n, n], kv=[300, n - 1], H=2, G=G, seed=63)
    c.K8[..., 7] = 0xB8                                   # -1.0: a score of -inf for an infinite channel 7
    c.Q[:n, 0, 7] = math.inf
    c.Q[n - 1, -1, 3] = math.nan
    c.Q[n, 0, 7] = math.inf                               # at position -1
    got = attend(c)
    c.check(got, c.cache())
    assert torch.isnan(got[0][:n, 0].float()).all() and torch.all(got[0][n] == 0)


@pytest.mark.parametrize("scale", [1e-60, 1e-46, 1e-30])
def test_small_softmax_scales(scale):
    """A scale that fp32 does not hold is not the default one."""
    c = Case(n=[2], kv=[200], H=2, seed=64)
    c.check(attend(c, softmax_scale=scale), c.cache(), scale=scale)


@pytest.mark.parametrize("n,G", TILES)
@pytest.mark.parametrize("d,skip", [(64, 1), (128, 0)])
def test_wait_timeout_and_recovery(n, G, d, skip):
    """The kernels' failure path: loaders that leave out a unit's keys.  The wait for them runs out and is
    recorded, every CTA ends, and the next call in the context is right."""
    c = Case(n=[n] * 40, kv=[1500] * 40, H=2, G=G, d=d, page=64, seed=66)
    Q, cache, args = c.Q.to(DEV), c.cache(DEV), c.args(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    vc.vc_debug_attn_paged_timeout(Q, cache, *args, status, skip, max_q=n)
    end.record()
    torch.cuda.synchronize()
    assert int(status) == 5
    # 2^16 attempts of 3.7 us, or twice that where something in flight never arrives
    assert start.elapsed_time(end) < 1000
    got = attend(c)
    one = Case(n=[n], kv=[1500], H=2, G=G, d=d, page=64, seed=66)
    one.Q, one.table, one.pages = c.Q[:n], c.table[:1], c.pages
    for k in ("K8", "sk", "V8", "sv"):
        setattr(one, k, getattr(c, k))
    one.check((got[0][:n], got[1][:n]), c.cache())


BROKEN = [([0, 4, 2, 12], [20, 30, 40]), ([-3, 4, 8, 12], [20, 30, 40]), ([5, 4, 3, 2], [20, 30, 40]), ([0, 4, 8, 2 ** 31 - 1], [20, 30, 40]),
          ([-2 ** 31, -1, 2 ** 31 - 1, 0], [20, 30, 40]), ([0, 4, 8, 12], [20, -1, 40]), ([0, 4, 8, 12], [20, 30, 2 ** 31 - 1]),
          ([0, 4, 8, 12], [-2 ** 31, 3, 1]), ([2, 4, 8, 11], [20, 30, 48])]


@pytest.mark.parametrize("cu,kv", BROKEN, ids=str)
@pytest.mark.parametrize("max_q", [1, 4, 500])
def test_broken_batches_touch_nothing_outside(cu, kv, max_q):
    """Offsets and lengths out of range, with guards around every buffer: nothing there is written, nor, as it
    would spread NaN, read; within them only the rows and slots that the clamped numbers name are written."""
    c = Case(n=[4, 4, 4], kv=[20, 30, 48], H=2, G=8, seed=19, cols=3)
    c.table[c.table < 0] = 0                              # what a length beyond the sequence's own finds
    guard = 64

    def guarded(t, fill):
        big = torch.full((t.shape[0] + 2 * guard, *t.shape[1:]), fill, dtype=t.dtype, device=DEV)
        inner = big[guard:-guard]
        inner.copy_(t)
        return inner, big

    nan = math.nan
    seven = torch.full((), 7.0)
    bufs = {"K8": guarded(c.K8, 0x7F), "V8": guarded(c.V8, 0x7F), "sk": guarded(c.sk, nan), "sv": guarded(c.sv, nan),
            "Q": guarded(c.Q, nan), "K": guarded(c.K, nan), "V": guarded(c.V, nan),
            "O": guarded(seven.to(torch.bfloat16).expand(c.T, 16, 128), 7.0), "lse": guarded(seven.expand(c.T, 16), 7.0),
            "K2": guarded(seven.to(torch.bfloat16).expand(c.T, 2, 128), 7.0), "V2": guarded(seven.to(torch.bfloat16).expand(c.T, 2, 128), 7.0)}
    cache = {k: bufs[k][0] for k in ("K8", "V8", "sk", "sv")}
    args = tuple(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, kv)) + (c.table.to(DEV),)
    before = {k: b[1].clone() for k, b in bufs.items()}
    rows, slots = torch.zeros(c.T, dtype=torch.bool), torch.zeros(c.pages, c.page, dtype=torch.bool)
    for b in range(3):
        first = min(max(cu[b], 0), c.T)
        n, length = min(max(cu[b + 1], first), c.T) - first, min(max(kv[b], 0), 3 * c.page)
        rows[first:first + n] = True
        for p in range(max(length - n, 0), length):
            slots[c.table[b, p // c.page], p % c.page] = True
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    vc.vc_attn_paged(bufs["Q"][0], cache, *args, max_q=max_q, O=bufs["O"][0], lse=bufs["lse"][0], dev_status=status)
    vc.vc_cache_read(cache, *args, c.T, K=bufs["K2"][0], V=bufs["V2"][0], dev_status=status)
    vc.vc_cache_append(bufs["K"][0], bufs["V"][0], cache, *args, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == (0 if kv[2] == 48 else 1)
    for k, (inner, big) in bufs.items():
        same = (big == before[k]) | (big != big) & (before[k] != before[k])
        assert same[:guard].all() and same[-guard:].all(), k
        assert not torch.isnan(inner.float()).any(), k
        same = same[guard:-guard].cpu()
        if k in ("K8", "V8", "sk", "sv"):
            assert same.transpose(1, 2)[~slots].all(), k
        else:
            assert same[~rows].all(), k


@pytest.mark.parametrize("n,G", TILES)
@pytest.mark.parametrize("d", [64, 128])
def test_items_of_many_parts(n, G, d):
    """One sequence over all CTAs: more parts of an item than a warp has lanes to join."""
    c = Case(n=[n], kv=[12000], H=1, G=G, d=d, page=64, seed=65)
    for mask in (dict(), dict(causal=0, window=9000)):
        c.check(attend(c, **mask), c.cache(), **mask)

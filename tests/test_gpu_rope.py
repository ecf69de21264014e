"""GPU: rotary positions (vc_rope, vc_cache_append_rope) against the formulas in fp64.

Bars.  The angle's fraction reaches sincospi within 2^-25 + 2^-31 half turns, which times pi is
below 2^-23.2; sincospi is within an ulp (2^-23 of 1 here, generously), the magnitude's product adds 2^-24:
cos and sin are within m 2^-21.  Two products and a sum in fp32 add 2 * 2^-24 of |x0 c| + |x1 s|.  So a
turned channel is within m (|x0| + |x1|) 2^-20.5 before it is rounded, to bf16 by half a step (2^-8 of the
value, or half the smallest step, 2^-134), or to E4M3 by half a step (2^-4, or 2^-10 of the scale)."""
import math

import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import E4M3, Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def turned(x, pos, rope, inverse=0):
    """fp64 [T, H, d] on the CPU and how far fp32 arithmetic may be off it."""
    x = x.double().cpu()
    turns, m = rope["turns"].cpu().tolist(), rope["magnitude"]
    half = len(turns)
    y, off = x.clone(), torch.zeros_like(x)
    for i, t in enumerate(turns):
        p, q = (i, i + half) if rope["layout"] == "halves" else (2 * i, 2 * i + 1)
        # whole numbers in Python: exact
        a = torch.tensor([2.0 * math.pi * (((t * int(k)) % 2 ** 64) / 2.0 ** 64) for k in pos], dtype=torch.float64)
        c, s = m * torch.cos(a)[:, None], m * torch.sin(a)[:, None] * (-1 if inverse else 1)
        y[..., p], y[..., q] = x[..., p] * c - x[..., q] * s, x[..., p] * s + x[..., q] * c
        off[..., p] = off[..., q] = m * (x[..., p].abs() + x[..., q].abs()) * 2.0 ** -20.5
    return y, off


def check(got, x, pos, rope, inverse=0):
    y, off = turned(x, pos, rope, inverse)
    got = got.double().cpu()
    rot = 2 * rope["turns"].numel()
    assert torch.equal(got[..., rot:], x.double().cpu()[..., rot:])
    assert torch.all((got - y).abs() <= off + 2.0 ** -8 * y.abs() + 2.0 ** -134)


def rows(T, H, d, seed):
    return torch.randn((T, H, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def some_positions(T, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 1 << 22, (T,), generator=g)
    ends = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, 1 << 20])[:T]
    pos[:len(ends)] = ends
    return pos.to(torch.int32)


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 80), (128, 96), (128, 128)])
@pytest.mark.parametrize("T,H", [(1, 1), (37, 1), (300, 3), (9, 40)])
def test_rope(layout, d, rot, T, H):
    rope = vc.make_rope(rot, layout=layout, device=DEV)
    X, pos = rows(T, H, d, 1), some_positions(T, 2)
    for inverse in (0, 1):
        check(vc.vc_rope(X, rope, pos=pos.to(DEV), inverse=inverse), X, pos.tolist(), rope, inverse)


@pytest.mark.parametrize("T,H,d,rot,layout", [(3001, 40, 128, 96, "halves"), (5003, 24, 64, 64, "pairs"), (60001, 1, 128, 32, "pairs"), (30011, 3, 64, 16, "halves"),
                                              (20011, 7, 128, 64, "halves")])
def test_many_rows(T, H, d, rot, layout):
    """Several rows a group of lanes, tokens that end anywhere among them."""
    rope = vc.make_rope(rot, layout=layout, device=DEV)
    X, pos = rows(T, H, d, 30), some_positions(T, 31)
    check(vc.vc_rope(X, rope, pos=pos.to(DEV)), X, pos.tolist(), rope)
    in_place = X.clone()
    vc.vc_rope(in_place, rope, pos=pos.to(DEV), out=in_place, inverse=1)
    check(in_place, X, pos.tolist(), rope, 1)


@pytest.mark.parametrize("kw", [dict(scaling="positions", factor=4.0), dict(scaling="base", factor=8.0, base=500000.0),
                                dict(scaling="ramp", factor=16.0), dict(scaling="ramp", factor=2.0, magnitude=0.75, original=8192)], ids=str)
def test_scaled_contexts(kw):
    rope = vc.make_rope(64, layout="pairs", device=DEV, **kw)
    X, pos = rows(50, 4, 128, 3), some_positions(50, 4)
    check(vc.vc_rope(X, rope, pos=pos.to(DEV)), X, pos.tolist(), rope)


def test_given_turns_of_any_size():
    """Turns that are not of a base: whole numbers of any size, sign bit and all."""
    g = torch.Generator().manual_seed(5)
    turns = torch.randint(-2 ** 63, 2 ** 63 - 1, (32,), generator=g)
    turns[0], turns[1], turns[2] = 0, -1, 2 ** 62
    rope = dict(turns=turns.to(DEV), layout="halves", magnitude=3.0)
    X, pos = rows(40, 2, 64, 6), some_positions(40, 7)
    check(vc.vc_rope(X, rope, pos=pos.to(DEV)), X, pos.tolist(), rope)


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_strides_and_in_place(layout):
    rope = vc.make_rope(96, layout=layout, device=DEV)
    packed = rows(60, 9, 128, 8).view(60, 3, 3, 128)
    X, pos = packed[:, 1], some_positions(60, 9).to(DEV)
    want = vc.vc_rope(X.contiguous(), rope, pos=pos)
    big = torch.full((60, 4, 136), 5.0, dtype=torch.bfloat16, device=DEV)
    out = vc.vc_rope(X, rope, pos=pos, out=big[:, :3, :128])
    assert torch.equal(out, want) and torch.all(big[:, 3] == 5.0) and torch.all(big[:, :, 128:] == 5.0)
    before = packed.clone()
    assert vc.vc_rope(X, rope, pos=pos, out=X) is X
    assert torch.equal(packed[:, 1], want) and torch.equal(packed[:, 0], before[:, 0]) and torch.equal(packed[:, 2], before[:, 2])


def test_positions_of_a_batch():
    """Those of the tokens in the cache; rows of no sequence stay, with given positions too."""
    c = Case(n=[3, 0, 70, 1], kv=[3, 9, 100, 5000], H=2, d=64, tail=4, seed=10)
    rope = vc.make_rope(64, device=DEV)
    X = c.Q.to(DEV)
    pos = torch.zeros(c.T, dtype=torch.int32)
    for r, _, p in c.places():
        pos[r] = p
    cu, kv, _ = c.args(DEV)
    for given in (None, pos.to(DEV)):
        out = torch.full_like(X, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        vc.vc_rope(X, rope, pos=given, cu=cu, kv_len=kv, out=out, dev_status=status)
        n = sum(c.n)
        check(out[:n], X[:n], pos[:n].tolist(), rope)
        assert torch.all(out[n:] == 7.0) and int(status) == 0
    for bad_cu, bad_kv in (([0, 3, 2, 73, 74], c.kv), ([0, 3, 3, 73, 99], c.kv), (c.cu.tolist(), [3, -9, 100, 5000])):
        status.zero_()
        vc.vc_rope(X, rope, cu=torch.tensor(bad_cu, dtype=torch.int32, device=DEV), kv_len=torch.tensor(bad_kv, dtype=torch.int32, device=DEV),
                   dev_status=status)
        assert int(status) == 1


def test_there_and_back():
    """The transposed map takes the first back, and is the gradient: the sums x . R^T g and (R x) . g agree, and so do
    differences of (R x) . g along single channels."""
    rope = vc.make_rope(128, device=DEV)
    X, g, pos = rows(200, 5, 128, 11), rows(200, 5, 128, 12), some_positions(200, 13)
    y = vc.vc_rope(X, rope, pos=pos.to(DEV))
    back = vc.vc_rope(y, rope, pos=pos.to(DEV), inverse=1)
    # two roundings to bf16, of both channels of a pair
    pair = (X.double().abs() + X.double().abs().roll(64, -1)) * 1.01
    assert torch.all((back.double() - X.double()).abs() <= 2.0 ** -8 * 2 * pair + 2.0 ** -8 * X.double().abs())
    dx = vc.vc_rope(g, rope, pos=pos.to(DEV), inverse=1)
    ref, _ = turned(X, pos.tolist(), rope)
    lhs = (ref * g.double().cpu()).sum(-1)
    bar = 2.0 ** -8 * (X.double().abs() * dx.double().abs()).sum(-1).cpu() + 1e-3
    assert torch.all((lhs - (X.double() * dx.double()).sum(-1).cpu()).abs() <= bar)
    for ch in (0, 5, 64, 127):
        e = X.double().cpu()
        step = torch.zeros_like(e)
        step[..., ch] = 1.0
        up, _ = turned(e + step, pos.tolist(), rope)
        down, _ = turned(e - step, pos.tolist(), rope)
        slope = ((up - down) / 2 * g.double().cpu()).sum(-1)
        want = dx.double().cpu()[..., ch]
        assert torch.all((slope - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * g.double().abs().cpu().amax(-1))


def test_rows_that_are_not_finite_spoil_only_themselves():
    rope = vc.make_rope(64, device=DEV)
    X, pos = rows(20, 4, 64, 14), some_positions(20, 15).to(DEV)
    want = vc.vc_rope(X, rope, pos=pos)
    Y = X.clone()
    Y[3, 1, 5], Y[7, 0, 40] = math.nan, math.inf
    got = vc.vc_rope(Y, rope, pos=pos)
    touched = torch.zeros_like(X, dtype=torch.bool)
    touched[3, 1, [5, 37]] = touched[7, 0, [8, 40]] = True
    assert torch.equal(got[~touched], want[~touched]) and torch.isnan(got[3, 1, [5, 37]]).all() and not torch.isfinite(got[7, 0, [8, 40]]).any()


def test_no_rows():
    rope = vc.make_rope(64, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert vc.vc_rope(rows(0, 4, 64, 0), rope, pos=none).shape == (0, 4, 64)
    c = Case(n=[0], kv=[5], H=2)
    out = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV), vc.make_rope(128, device=DEV))
    assert out.shape == (0, 2, 128)


# ---------------------------------------------------------------- with the cache

APPEND_CASES = [dict(n=[1], kv=[1], H=1, d=64), dict(n=[1] * 5, kv=[1, 17, 128, 5000, 16], H=8, G=4), dict(n=[0, 5, 0, 40, 0], kv=[0, 9, 33, 40, 7], H=3, G=2, d=64, page=32),
                dict(n=[300], kv=[500], H=5, page=128), dict(n=[3] * 70, kv=[50] * 70, H=2, d=64, tail=5), dict(n=[16, 256], kv=[16, 256], H=1, G=16, page=256),
                dict(n=[1500, 0, 703], kv=[1600, 9, 703], H=8, G=5, page=64), dict(n=[9000], kv=[9001], H=2, G=3, d=64, page=128, tail=3)]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "B%d_H%d" % (len(c["n"]), c["H"]))
@pytest.mark.parametrize("layout,rot", [("halves", 64), ("pairs", 48)])
def test_append(case, layout, rot):
    c = Case(seed=16, **case)
    rope = vc.make_rope(rot, layout=layout, scaling="ramp", factor=4.0, device=DEV)
    args, (K, V) = c.args(DEV), (c.K.to(DEV), c.V.to(DEV))
    cache, plain = c.cache(DEV), c.cache(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((c.T, c.H * c.G, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    assert vc.vc_cache_append_rope(c.Q.to(DEV), K, V, cache, *args, rope, out=out, dev_status=status) is out
    vc.vc_cache_append(K, V, plain, *args)
    assert int(status) == 0 and torch.equal(cache["V8"], plain["V8"]) and torch.equal(cache["sv"], plain["sv"])
    n, pos = sum(c.n), [p for _, _, p in c.places()]
    check(out[:n], c.Q[:n], pos, rope)
    assert torch.all(out[n:] == 7.0)
    # the keys, and everything else in the cache as it was
    y, off = turned(c.K[:n], pos, rope)
    got, untouched = {k: v.cpu() for k, v in cache.items()}, torch.ones(c.pages, c.page, dtype=torch.bool)
    for r, b, p in c.places():
        pg, at = c.page_of(b, p), p % c.page
        untouched[pg, at] = False
        scale = got["sk"][pg, :, at].double()
        amax = y[r].abs().amax(-1)
        assert torch.all((scale * 448 - amax).abs() <= off[r].amax(-1) + 2.0 ** -22 * amax)
        value = E4M3[got["K8"][pg, :, at].long()] * scale[:, None]
        bar = off[r] * 2 + (2.0 ** -4 + 2.0 ** -21) * y[r].abs() + 2.0 ** -10 * scale[:, None]
        assert torch.all((value - y[r]).abs() <= bar)
    before = c.cache()
    for k in ("K8", "sk"):
        assert torch.equal(got[k].transpose(1, 2)[untouched], before[k].transpose(1, 2)[untouched])
    # keys alone; and at position 0 of magnitude 1 nothing turns: bit for bit vc_cache_append
    again = c.cache(DEV)
    assert vc.vc_cache_append_rope(None, K, V, again, *args, rope) is None
    assert all(torch.equal(again[k], cache[k]) for k in again)
    still = c.cache(DEV)
    vc.vc_cache_append_rope(None, K, V, still, *args, dict(rope, magnitude=1.0), pos=torch.zeros(c.T, dtype=torch.int32, device=DEV))
    assert all(torch.equal(still[k], plain[k]) for k in still)


def test_append_at_other_positions():
    """pos turns, the batch places."""
    c = Case(n=[40, 3], kv=[90, 3], H=2, G=2, seed=17)
    rope, pos = vc.make_rope(128, device=DEV), some_positions(43, 18)
    cache = c.cache(DEV)
    out = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), cache, *c.args(DEV), rope, pos=pos.to(DEV))
    check(out, c.Q, pos.tolist(), rope)
    want = c.cache(DEV)
    vc.vc_cache_append_rope(None, c.K.to(DEV), c.V.to(DEV), want, *c.args(DEV), rope, pos=pos.to(DEV))
    assert all(torch.equal(want[k], cache[k]) for k in want)
    K, _ = vc.vc_cache_read(cache, *c.args(DEV), 43)
    y, off = turned(c.K, pos.tolist(), rope)
    amax = y.abs().amax(-1, keepdim=True)
    assert torch.all((K.double().cpu() - y).abs() <= (2.0 ** -4 + 2.0 ** -7) * y.abs() + 2.0 ** -10 * amax / 448 + 3 * off)


def test_append_extreme_rows():
    """Zeros, tiny rows, rows that leave fp32 when turned, NaN and infinities: as vc_cache_append writes such rows."""
    c = Case(n=[8], kv=[20], H=2, seed=19)
    c.K[0], c.K[1] = 0, 2.0 ** -102
    c.K[2] = 3.3e38                       # cos + sin > 1: beyond fp32
    c.K[3, 0, 5], c.K[4, 1, 127] = math.nan, -math.inf
    rope = vc.make_rope(128, device=DEV)
    pos = torch.full((8,), 1, dtype=torch.int32, device=DEV)
    cache = vc.vc_cache_append(c.K.to(DEV), c.V.to(DEV), c.cache(DEV), *c.args(DEV))
    vc.vc_cache_append_rope(None, c.K.to(DEV), c.V.to(DEV), cache, *c.args(DEV), rope, pos=pos)
    sk = torch.stack([cache["sk"][c.page_of(0, p), :, p % 16] for p in range(12, 20)]).cpu()
    K8 = torch.stack([cache["K8"][c.page_of(0, p), :, p % 16] for p in range(12, 20)]).cpu()
    assert torch.all(sk[:2] == 0) and torch.isnan(sk[2]).all() and torch.isnan(sk[3, 0]) and torch.isnan(sk[4, 1])
    assert torch.isfinite(sk[3, 1]) and torch.isfinite(sk[4, 0]) and not K8[:3].any() and not K8[3, 0].any() and torch.isfinite(sk[5:]).all()


def test_append_where_a_page_is_not_there():
    c = Case(n=[40, 30], kv=[40, 20], H=2, G=2, seed=20)     # the second begins 10 positions below 0
    c.table[0, 1] = -1
    rope, status = vc.make_rope(64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    cache, before = c.cache(DEV), c.cache()
    out = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), cache, *c.args(DEV), rope, dev_status=status)
    assert int(status) == 1
    check(out, c.Q, [p for _, _, p in c.places()], rope)
    slots = torch.zeros(c.pages, c.page, dtype=torch.bool)
    for _, b, p in c.places():
        if p >= 0 and c.page_of(b, p) is not None:
            slots[c.page_of(b, p), p % c.page] = True
    for k in before:
        same = (cache[k].cpu() == before[k]).transpose(1, 2)
        assert same[~slots].all() and not same[slots].all()


@pytest.mark.parametrize("H,G,d", [(8, 5, 128), (1, 1, 64)])
def test_captured_steps_on_another_stream(H, G, d):
    """Two graphs of the step, replayed with other tokens and lengths, beside the same call on another stream."""
    rope = vc.make_rope(d, device=DEV)
    cases = [Case(n=[1, 3], kv=kv, H=H, G=G, d=d, seed=21 + i, spare=0, cols=60) for i, kv in enumerate(([500, 400], [900, 70]))]
    pages = max(c.pages for c in cases)
    buf = [t.to(DEV) for t in (cases[0].Q, cases[0].K, cases[0].V, *cases[0].args("cpu"))]
    cache = vc.alloc_cache(pages, 16, H, d, DEV)
    graph = torch.cuda.CUDAGraph()
    vc.vc_cache_append_rope(*buf[:3], cache, *buf[3:], rope)
    with torch.cuda.graph(graph):
        out = vc.vc_cache_append_rope(*buf[:3], cache, *buf[3:], rope)
    side = torch.cuda.Stream()
    for c in (cases[1], cases[0], cases[1]):
        for t, new in zip(buf, (c.Q, c.K, c.V, *c.args("cpu"))):
            t.copy_(new)
        for k in cache:
            cache[k][:c.pages].copy_(getattr(c, k))
        torch.cuda.synchronize()
        graph.replay()
        other = c.cache(DEV)
        side.wait_stream(torch.cuda.current_stream())
        got = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), other, *c.args(DEV), rope, stream=side)
        torch.cuda.synchronize()
        check(out, c.Q, [p for _, _, p in c.places()], rope)
        assert torch.equal(got, out) and all(torch.equal(other[k], cache[k][:c.pages]) for k in other)


@pytest.mark.parametrize("n", [1, 60])
def test_step_then_attention(n):
    """Turned queries over turned keys depend on the distance of their positions alone: a step of the whole sequence
    moved by 1,000,003 positions gives the same scores, within what the turned rows' rounding allows."""
    c = Case(n=[n], kv=[n], H=2, G=2, seed=25)
    rope = vc.make_rope(128, device=DEV)
    outs = []
    for shift in (0, 1000003):
        cache = c.cache(DEV)
        pos = (torch.arange(n, dtype=torch.int32) + shift).to(DEV)
        Q = vc.vc_cache_append_rope(c.Q.to(DEV), c.K.to(DEV), c.V.to(DEV), cache, *c.args(DEV), rope, pos=pos)
        O, lse = vc.vc_attn_paged(Q, cache, *c.args(DEV), max_q=n)
        one = Case(n=[n], kv=[n], H=2, G=2, seed=25)
        one.Q = Q.cpu()
        for k, v in cache.items():
            setattr(one, k, v.cpu())
        one.check((O, lse), one.cache())
        outs.append(lse.double())
    # scores of |q| |k| / sqrt(d): keys within half a step of E4M3 a channel, queries of bf16, both times
    norms = (c.Q.double().view(n, 2, 2, 128).norm(dim=-1) * c.K.double().norm(dim=-1).amax(0)[:, None]).amax(-1).amax(-1) / math.sqrt(128)
    assert torch.all((outs[0] - outs[1]).abs().amax(-1).cpu() <= 2 * (2.0 ** -4 + 2.0 ** -8) * norms + 1e-4)

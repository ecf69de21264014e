"""CPU: what the rotary and page calls refuse before any launch, the angles of make_rope, and the page calls' meaning."""
import ctypes
import math

import pytest
import torch

from bit_fp8_attention_means_gb300 import build, vc
from paged_case import Case
from pool_model import Model, rng_of, walk

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
ODD, TWO = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    build.build()
    return vc.lib()


def cache(**kw):
    s = vc.VcCacheShape(10, 16, 2, 128, 2 * 16 * 128, 16 * 128, 128, 32, 16)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def batch(**kw):
    b = vc.VcBatch(0x10000, 0x10000, 0x10000, 3, 7, 4, 4)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def spec(**kw):
    s = vc.VcRopeSpec(0x10000, 64, 0, 1.0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD_SPECS = [dict(turns=None), dict(turns=0x10004), dict(rot=0), dict(rot=8), dict(rot=40), dict(rot=144), dict(rot=-16), dict(layout=2), dict(layout=-1),
             dict(magnitude=0.0), dict(magnitude=-1.0), dict(magnitude=math.nan), dict(magnitude=math.inf)]


def test_rope_refusals(L):
    def call(X=FAKE, s=(256, 128), T=7, H=2, d=128, rope=spec(), pos=FAKE, cu=FAKE, kv=FAKE, B=3, inverse=0, out=FAKE, o=(256, 128)):
        return L.vc_rope(X, *s, T, H, d, rope, pos, cu, kv, B, inverse, out, *o, None, None)
    for bad in BAD_SPECS:
        assert call(rope=spec(**bad)) == 1, bad
    for bad in (dict(X=None), dict(X=ODD), dict(out=None), dict(out=ODD), dict(s=(0, 128)), dict(s=(256, 4)), dict(o=(-8, 128)), dict(o=(256, 0)), dict(T=-1), dict(H=0),
                dict(d=0), dict(inverse=2), dict(cu=None), dict(kv=None), dict(pos=None, cu=None, kv=None), dict(B=0), dict(pos=TWO)):
        assert call(**bad) == 1, bad
    for bad in (dict(d=96), dict(T=1 << 30, H=2)):
        assert call(**bad) == 2, bad
    assert call(T=0, X=None, out=None, pos=None, cu=None, kv=None) == 0


def test_append_rope_refusals(L):
    def call(Q=FAKE, q=(512, 128), Hq=4, K=FAKE, V=FAKE, s=(256, 128), c=cache(), codes=(FAKE,) * 4, b=batch(), rope=spec(), pos=None, out=FAKE, o=(512, 128)):
        return L.vc_cache_append_rope(Q, *q, Hq, K, V, *s, c, *codes, b, rope, pos, out, *o, None, None)
    for bad in BAD_SPECS:
        assert call(rope=spec(**bad)) == 1, bad
    assert call(rope=spec(rot=80), c=cache(d=64)) == 1
    for bad in (dict(Q=None), dict(Q=ODD), dict(out=None), dict(out=ODD), dict(q=(0, 128)), dict(o=(512, 4)), dict(Hq=-1), dict(K=None), dict(V=ODD), dict(s=(100, 128)),
                dict(codes=(None, FAKE, FAKE, FAKE)), dict(codes=(FAKE, FAKE, ODD, FAKE)), dict(b=batch(B=0)), dict(b=batch(cu=None)), dict(b=batch(s_table=3)), dict(pos=TWO),
                dict(c=cache(pages=0)), dict(c=cache(s_tok=8))):
        assert call(**bad) == 1, bad
    for bad in (dict(c=cache(d=96)), dict(c=cache(page_size=48)), dict(b=batch(T=1 << 28)), dict(b=batch(cols=1 << 26, s_table=1 << 26))):
        assert call(**bad) == 2, bad
    assert call(b=batch(T=0, cu=None), codes=(None,) * 4, Q=None, K=None) == 0


def pool(**kw):
    p = vc.VcPool(0x10000, 0x10000)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


SHAPES = [(dict(pages=0), 1), (dict(page_size=8), 2), (dict(d=96), 2), (dict(s_tok=8), 1), (dict(pages=(1 << 30) + 1), 2)]
POOLS = [dict(refs=None), dict(free_pages=None), dict(refs=0x10002), dict(free_pages=0x10001)]


def test_reserve_refusals(L):
    def call(c=cache(), codes=(FAKE,) * 4, p=pool(), b=batch(), ws=FAKE, nbytes=1 << 20):
        return L.vc_pages_reserve(c, *codes, p, b, ws, nbytes, None, None)
    for kw, code in SHAPES:
        assert call(c=cache(**kw)) == code, kw
    for kw in POOLS:
        assert call(p=pool(**kw)) == 1, kw
    for kw, code in ((dict(B=0), 1), (dict(T=-1), 1), (dict(cols=0), 1), (dict(cu=None), 1), (dict(table=None), 1), (dict(s_table=3), 1), (dict(cols=1 << 26, s_table=1 << 26), 2)):
        assert call(b=batch(**kw)) == code, kw
    assert call(codes=(FAKE, None, FAKE, FAKE)) == 1 and call(c=cache(H=1 << 20)) == 2
    need = L.vc_pages_reserve_workspace(cache(), 3, 7)
    assert need >= 4 * 7 and call(ws=None) == 3 and call(nbytes=need - 1) == 3 and call(ws=ctypes.c_void_p(0x10080)) == 3
    assert L.vc_pages_reserve_workspace(cache(d=96), 3, 7) == 0 and call(b=batch(T=0)) == 0


def test_fork_and_trim_refusals(L):
    apart = ctypes.c_void_p(0x20000)

    def fork(c=cache(), p=pool(), table=FAKE, s=4, B=3, cols=4, kv=FAKE, parents=FAKE, lens=None, N=2, new=apart, s_new=4, new_cols=4, new_len=apart):
        return L.vc_pages_fork(c, p, table, s, B, cols, kv, parents, lens, N, new, s_new, new_cols, new_len, None, None)

    def trim(c=cache(), p=pool(), table=FAKE, s=4, B=3, cols=4, kv=FAKE, lens=FAKE):
        return L.vc_pages_trim(c, p, table, s, B, cols, kv, lens, None, None)
    for call in (fork, trim):
        for kw, code in SHAPES:
            assert call(c=cache(**kw)) == code, kw
        for kw in POOLS:
            assert call(p=pool(**kw)) == 1, kw
        for kw in (dict(table=None), dict(table=TWO), dict(s=3), dict(B=0), dict(cols=0), dict(kv=None), dict(kv=TWO), dict(lens=TWO)):
            assert call(**kw) == 1, kw
        assert call(cols=1 << 26, s=1 << 26) == 2
    assert trim(lens=None) == 1
    for kw in (dict(parents=None), dict(new=None), dict(new=TWO), dict(N=-1), dict(s_new=3), dict(new_cols=0), dict(new_len=None), dict(new_len=FAKE), dict(new=FAKE),
               dict(new=ctypes.c_void_p(0x10000 + 4 * 11)), dict(new=ctypes.c_void_p(0x10000 - 4 * 7)), dict(new_len=ctypes.c_void_p(0x10000 - 4)),
               dict(parents=apart), dict(parents=ctypes.c_void_p(0x20004))):
        assert fork(**kw) == 1, kw
    assert fork(new_cols=1 << 26, s_new=1 << 26) == 2 and fork(N=0, new=None) == 0


def test_compact_and_copy_refusals(L):
    def compact(c=cache(), codes=(FAKE,) * 4, p=pool(), table=FAKE, s=4, B=3, cols=4, used=FAKE, ws=FAKE, nbytes=1 << 20):
        return L.vc_pages_compact(c, *codes, p, table, s, B, cols, used, ws, nbytes, None, None)

    def copy(c=cache(), codes=(FAKE,) * 4, t=cache(), to_codes=(FAKE,) * 4, pages=FAKE, to=FAKE, N=3):
        return L.vc_cache_copy(c, *codes, t, *to_codes, pages, to, N, None, None)
    for kw, code in SHAPES:
        assert compact(c=cache(**kw)) == code, kw
    for kw in POOLS:
        assert compact(p=pool(**kw)) == 1, kw
    for kw in (dict(table=None), dict(s=3), dict(B=0), dict(cols=0), dict(used=TWO), dict(codes=(ODD, FAKE, FAKE, FAKE))):
        assert compact(**kw) == 1, kw
    need = L.vc_pages_compact_workspace(cache())
    assert need >= 4 * 10 and compact(ws=None) == 3 and compact(nbytes=need - 1) == 3 and compact(c=cache(H=1 << 20)) == 2
    for kw in (dict(c=cache(pages=0)), dict(t=cache(s_page=-16)), dict(t=cache(page_size=32)), dict(t=cache(H=3)), dict(t=cache(d=64)), dict(N=-1), dict(pages=None), dict(to=None),
               dict(pages=TWO), dict(codes=(FAKE, FAKE, FAKE, None)), dict(to_codes=(FAKE, ODD, FAKE, FAKE))):
        assert copy(**kw) == 1, kw
    assert copy(c=cache(d=96), t=cache(d=96)) == 2 and copy(c=cache(H=1 << 20), t=cache(H=1 << 20)) == 2 and copy(N=0, pages=None) == 0


def test_binding_refusals(L):
    c = Case(n=[2], kv=[5], H=2)
    data, args, rope = c.cache(), c.args("cpu"), vc.make_rope(64, device="cpu")
    pos, p = torch.zeros(2, dtype=torch.int32), vc.alloc_pool(c.pages, "cpu")
    for bad in (c.Q.float(), c.Q[0], c.Q.transpose(0, 2)):
        with pytest.raises(ValueError):
            vc.vc_rope(bad, rope, pos=pos)
    for kw in (dict(), dict(pos=pos.long()), dict(pos=pos[:1]), dict(cu=args[0]), dict(cu=args[0][:1], kv_len=args[1])):
        with pytest.raises(ValueError):
            vc.vc_rope(c.Q, rope, **kw)
    for bad in (dict(rope, turns=rope["turns"].int()), dict(rope, turns=rope["turns"][::2]), dict(rope, layout="quarters")):
        with pytest.raises(ValueError):
            vc.vc_rope(c.Q, bad, pos=pos)
        with pytest.raises(ValueError):
            vc.vc_cache_append_rope(c.Q, c.K, c.V, data, *args, bad)
    for Q, K, kw in ((c.Q[:1], c.K, {}), (c.Q.float(), c.K, {}), (c.Q, c.K[:, :1], {}), (None, c.K, dict(out=c.Q)), (c.Q, c.K, dict(pos=pos.float()))):
        with pytest.raises(ValueError):
            vc.vc_cache_append_rope(Q, K, c.V, data, *args, rope, **kw)
    other = torch.full((1, 3), -1, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    calls = [lambda p: vc.vc_pages_reserve(data, p, *args, 2), lambda p: vc.vc_pages_fork(data, p, args[2], args[1], lens, other, lens.clone()),
             lambda p: vc.vc_pages_trim(data, p, args[2], args[1], lens), lambda p: vc.vc_pages_compact(data, p, args[2])]
    for call in calls:
        for bad in (dict(p, refs=p["refs"][1:]), dict(p, refs=p["refs"].long()), dict(p, free=p["free"].float()), dict(p, free=p["free"].repeat(2))):
            with pytest.raises(ValueError):
                call(bad)
        with pytest.raises(ValueError, match="CUDA"):
            call(p)
    for bad in (lambda: vc.vc_pages_trim(data, p, args[2][0], args[1], lens), lambda: vc.vc_pages_trim(data, p, args[2].long(), args[1], lens),
                lambda: vc.vc_pages_trim(data, p, args[2], args[1], lens.repeat(2)), lambda: vc.vc_pages_fork(data, p, args[2], args[1], lens.repeat(2), other, lens),
                lambda: vc.vc_cache_copy(data, data, lens, lens.repeat(2)), lambda: vc.vc_cache_copy(data, data, lens.long(), lens)):
        with pytest.raises(ValueError):
            bad()
    for call in (lambda: vc.vc_rope(c.Q, rope, pos=pos), lambda: vc.vc_cache_append_rope(c.Q, c.K, c.V, data, *args, rope), lambda: vc.vc_cache_copy(data, data, lens, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for kw in (dict(rot=24), dict(rot=0), dict(rot=64, layout="x"), dict(rot=64, scaling="x"), dict(rot=64, base=0.0), dict(rot=64, fast=1.0)):
        with pytest.raises(ValueError):
            vc.make_rope(device="cpu", **kw)


def radians(rope):
    return [2 * math.pi * (t % 2 ** 64) / 2.0 ** 64 for t in rope["turns"].tolist()]


def test_angles():
    def near(x, y):
        return all(abs(a - b) <= 1e-13 * abs(b) + 1e-17 for a, b in zip(x, y))
    w = [10000.0 ** (-i / 32.0) for i in range(32)]
    assert near(radians(vc.make_rope(64, device="cpu")), w)
    assert near(radians(vc.make_rope(64, scaling="positions", factor=4.0, device="cpu")), [x / 4 for x in w])
    based = radians(vc.make_rope(64, scaling="base", factor=4.0, device="cpu"))
    assert near(based[:1], [1.0]) and near(based[-1:], [w[-1] / 4])
    ramp = vc.make_rope(64, scaling="ramp", factor=8.0, device="cpu")
    turns = [4096 * x / (2 * math.pi) for x in w]
    keep = [min(max((t - 1) / 31, 0), 1) for t in turns]
    assert near(radians(ramp), [x * k + x / 8 * (1 - k) for x, k in zip(w, keep)])
    assert 0 in keep and 1 in keep and any(0 < k < 1 for k in keep)
    assert ramp["magnitude"] == 0.1 * math.log(8.0) + 1 and vc.make_rope(64, scaling="ramp", factor=8.0, magnitude=2, device="cpu")["magnitude"] == 2.0
    assert vc.make_rope(64, device="cpu")["magnitude"] == 1.0


def test_new_pools():
    for pages in (1, 31, 32, 33, 64, 100):
        p = vc.alloc_pool(pages, "cpu")
        m = Model(pages, 16, 1, 1, H=1)
        assert p["refs"].tolist() == m.refs and p["free"].tolist() == m.bits()


def test_model_walks_stay_consistent():
    """The tests' own model: counts are names after any walk, and a refused reservation changes no count."""
    refused = 0
    for seed in range(6):
        rng = rng_of(seed)
        m = Model(rng.choice([9, 14, 33]), 16, 6, 8, H=1, seed=seed)
        for op, arg in walk(m, rng, 60):
            if op == "reserve":
                m.kv = [k + n for k, n in zip(m.kv, arg)]
                refs = list(m.refs)
                if not m.reserve(arg):
                    refused += 1
                    assert m.refs == refs and m.consistent()
                    m.trim([k - n for k, n in zip(m.kv, arg)])
            elif op == "trim":
                m.trim(arg)
            elif op == "compact":
                used = m.compact()
                assert all(r > 0 for r in m.refs[:used]) and not any(m.refs[used:])
            else:
                parents, rows, lens = arg
                m.trim([0 if r in rows else -1 for r in range(6)])
                m.fork(parents, rows, lens)
            assert m.consistent()
    assert refused


def test_shared_prefix_refusals(L):
    def call(c=cache(), b=batch(), Q=FAKE, O=FAKE, Hq=4, q=(512, 128), o=(512, 128), groups=FAKE, prefix=FAKE, N=2, scale=0.0, causal=1, max_q=0, max_rows=0, lse=FAKE, ws=FAKE,
             ws_bytes=1 << 40, codes=(FAKE,) * 4):
        return L.vc_attn_paged_shared(Q, *q, Hq, c, *codes, b, groups, prefix, N, scale, causal, max_q, max_rows, O, *o, lse, ws, ws_bytes, None, None)
    for bad in (dict(groups=None), dict(prefix=None), dict(groups=TWO), dict(prefix=TWO), dict(N=-1), dict(max_rows=-1), dict(max_q=-1), dict(Q=None), dict(Q=ODD), dict(O=ODD),
                dict(Hq=3), dict(q=(0, 128)), dict(o=(512, 4)), dict(scale=math.nan), dict(scale=3.4e38), dict(causal=2), dict(lse=TWO), dict(codes=(FAKE, FAKE, None, FAKE)),
                dict(c=cache(pages=0)), dict(b=batch(B=0)), dict(b=batch(cu=None)), dict(b=batch(s_table=3))):
        assert call(**bad) == 1, bad
    for bad in (dict(c=cache(d=96)), dict(b=batch(T=1 << 28)), dict(b=batch(cols=1 << 26, s_table=1 << 26))):
        assert call(**bad) == 2, bad
    for N in (0, 2):
        need = L.vc_attn_paged_shared_workspace(cache(), 4, 3, 7, N, 0, 0)
        assert need > 0 and call(N=N, ws=None) == 3 and call(N=N, ws_bytes=need - 1) == 3 and call(N=N, ws=ctypes.c_void_p(0x10080)) == 3
    assert L.vc_attn_paged_shared_workspace(cache(), 3, 3, 7, 2, 0, 0) == 0 and L.vc_attn_paged_shared_workspace(cache(), 4, 3, 7, -1, 0, 0) == 0
    assert call(b=batch(T=0, cu=None), groups=None, Q=None, codes=(None,) * 4) == 0
    c = Case(n=[2], kv=[5], H=2)
    groups, prefix = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    for bad in ((groups[:1], prefix), (groups.long(), prefix), (groups, prefix.float()), (groups, prefix.repeat(2))):
        with pytest.raises(ValueError):
            vc.vc_attn_paged_shared(c.Q, c.cache(), *c.args("cpu"), *bad)
    with pytest.raises(ValueError, match="CUDA"):
        vc.vc_attn_paged_shared(c.Q, c.cache(), *c.args("cpu"), groups, prefix)

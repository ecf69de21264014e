"""CPU: calls that read what other blocks of the same launch write are refused before any launch."""
import ctypes

import pytest

from bit_fp8_attention_means_gb300 import build, vc
from test_rope_pages_host import batch, cache, pool

PAST = 4  # VC_ERR_CUDA: the arguments were taken, and there is no GPU here


@pytest.fixture(scope="module")
def L():
    build.build()
    return vc.lib()


def at(words):
    return ctypes.c_void_p(0x100000 + 4 * words)


@pytest.fixture(autouse=True)
def without_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")


def test_fork(L):
    """table 3 x 4 of row stride 6 at word 0 (16 words), kv_len [3] at 100, parents [2] at 200, lens [2] at 300, new_table
    2 x 5 of row stride 7 at 400 (12 words), new_len [2] at 500."""
    def call(table=0, kv=100, parents=200, lens=300, new=400, new_len=500):
        return L.vc_pages_fork(cache(), pool(), at(table), 6, 3, 4, at(kv), at(parents), None if lens is None else at(lens), 2, at(new), 7, 5,
                               at(new_len), None, None)
    for good in ({}, dict(lens=None), dict(lens=500), dict(new=16), dict(table=412), dict(new_len=103), dict(new_len=98), dict(new_len=202), dict(new_len=198),
                 dict(new_len=302), dict(new_len=298), dict(new_len=412), dict(new_len=398), dict(lens=412), dict(lens=398), dict(parents=412), dict(kv=397),
                 dict(parents=300), dict(lens=100), dict(kv=0), dict(new_len=16), dict(new_len=-2)):
        assert call(**good) == PAST, good
    for bad in (dict(new=15), dict(table=411), dict(new_len=102), dict(new_len=99), dict(new_len=201), dict(new_len=199), dict(new_len=301), dict(new_len=299),
                dict(new_len=411), dict(new_len=399), dict(lens=411), dict(lens=399), dict(parents=411), dict(parents=399), dict(kv=398), dict(kv=411), dict(new_len=15),
                dict(new_len=-1), dict(new_len=5), dict(new_len=100), dict(new_len=400), dict(new=300), dict(lens=499), dict(lens=501),
                dict(parents=500, lens=500), dict(kv=500, lens=500)):
        assert call(**bad) == 1, bad


def test_trim(L):
    """table 3 x 4 of row stride 6 at word 0 (16 words), kv_len [3] at 100, lens [3] at 200."""
    def call(table=0, kv=100, lens=200):
        return L.vc_pages_trim(cache(), pool(), at(table), 6, 3, 4, at(kv), at(lens), None, None)
    for good in ({}, dict(lens=100), dict(lens=103), dict(lens=97), dict(lens=16), dict(lens=-3), dict(kv=16), dict(kv=-3)):
        assert call(**good) == PAST, good
    for bad in (dict(lens=101), dict(lens=98), dict(lens=15), dict(lens=-2), dict(lens=7), dict(kv=15), dict(kv=-2)):
        assert call(**bad) == 1, bad


def test_reserve_and_compact(L):
    """table 3 x 4 at word 0 (12 words); cu [4], kv_len [3] and used [1] beside it and within it."""
    codes = [ctypes.c_void_p(0x200000)] * 4

    def reserve(cu=100, kv=200):
        b = batch(cu=at(cu).value, kv_len=at(kv).value, table=at(0).value)
        return L.vc_pages_reserve(cache(), *codes, pool(), b, ctypes.c_void_p(0x300000), 1 << 20, None, None)

    def compact(used):
        return L.vc_pages_compact(cache(), *codes, pool(), at(0), 4, 3, 4, used, ctypes.c_void_p(0x300000), 1 << 20, None, None)
    for good in ({}, dict(cu=12), dict(cu=-4), dict(kv=12), dict(kv=-3), dict(cu=200)):
        assert reserve(**good) == PAST, good
    for bad in (dict(cu=11), dict(cu=-3), dict(kv=11), dict(kv=-2), dict(kv=4)):
        assert reserve(**bad) == 1, bad
    assert [compact(x) for x in (None, at(12), at(-1))] == [PAST] * 3 and [compact(x) for x in (at(0), at(11))] == [1, 1]


def rows_of(at, s_n, s_h, T, H, d):
    return [range(a, a + d) for a in (at + t * s_n + h * s_h for t in range(T) for h in range(H))]


def meet(a, b):
    return any(x.start < y.stop and y.start < x.stop for x in a for y in b)


def test_rows_turned_into_others_place(L):
    """vc_rope and vc_cache_append_rope into rows that hold what is still to be read: against every pair of rows.
    Offsets of heads of 64 channels, in units of 8 elements."""
    rope = vc.VcRopeSpec(0x10000, 64, 0, 1.0)
    base, d, seen = 0x400000, 64, set()

    def element(x):
        return ctypes.c_void_p(base + 16 * x)

    def turn(x, s, out, o, T, H):
        return L.vc_rope(element(x), 8 * s[0], 8 * s[1], T, H, d, rope, at(0), None, None, 0, 0, element(out), 8 * o[0], 8 * o[1], None, None)

    for T, H, s in ((3, 2, (48, 8)), (3, 2, (8, 24)), (1, 3, (16, 8)), (4, 1, (24, 8)), (2, 3, (25, 9)), (5, 2, (16, 40))):
        x = rows_of(0, *s, T, H, 8)
        for out in range(-120, 121):
            want = 1 if out and meet(x, rows_of(out, *s, T, H, 8)) else PAST
            seen.add((out == 0, want))
            assert turn(0, s, out, s, T, H) == want, (T, H, s, out)
    assert seen == {(True, PAST), (False, 1), (False, PAST)}
    # a dimension of one row or head has any stride; X itself with other strides is not X itself
    assert turn(0, (48, 8), 0, (99, 8), 1, 3) == turn(0, (48, 8), 0, (48, 77), 3, 1) == PAST
    assert turn(0, (48, 8), 0, (56, 8), 3, 3) == turn(0, (48, 8), 0, (48, 16), 3, 3) == 1
    # queries, keys and values as heads of one tensor: in place, into a part of it, and into what keys or values hold
    code = [ctypes.c_void_p(0x200000)] * 4

    def append(out, Hq=3, q=0, k=24, v=40, o=(64, 8)):
        b = batch(T=3)
        return L.vc_cache_append_rope(element(q), 512, 64, Hq, element(k), element(v), 512, 64, cache(d=64, s_page=2048, s_head=1024, s_tok=64), *code, b, rope, None,
                                      element(out), 8 * o[0], 8 * o[1], None, None)
    q, k, v = (rows_of(x, 64, 8, 3, H, 8) for x, H in ((0, 3), (24, 2), (40, 2)))
    for out in range(-200, 201):
        o = rows_of(out, 64, 8, 3, 3, 8)
        assert append(out) == (1 if meet(o, k) or meet(o, v) or (out and meet(o, q)) else PAST), out
    assert append(500, o=(24, 8)) == PAST and append(0, o=(24, 8)) == append(24, Hq=1, o=(8, 8)) == 1

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

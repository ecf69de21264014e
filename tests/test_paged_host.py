"""CPU: what the paged cache's entry points refuse before any launch, and the tests' own definitions."""
import ctypes
import math

import pytest
import torch

from bit_fp8_attention_means_gb300 import build, vc
from paged_case import E4M3, Case, encode, quantize

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    build.build()
    return vc.lib()


def _cache(**kw):
    s = vc.VcCacheShape(10, 16, 2, 128, 2 * 16 * 128, 16 * 128, 128, 32, 16)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _batch(**kw):
    b = vc.VcBatch(0x10000, 0x10000, 0x10000, 3, 7, 4, 4)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


BAD_SHAPES = [(dict(pages=0), 1), (dict(H=0), 1), (dict(d=0), 1), (dict(page_size=-16), 1), (dict(d=96), 2), (dict(d=256), 2),
              (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=8192), 2), (dict(s_tok=0), 1),
              (dict(s_tok=8), 1), (dict(s_page=-4096), 1), (dict(s_head=24), 1), (dict(t_page=0), 1), (dict(t_head=6), 1),
              (dict(s_page=1 << 40), 1), (dict(s_head=1 << 41), 1), (dict(s_tok=1 << 40), 1)]
BAD_BATCHES = [(dict(B=0), 1), (dict(T=-1), 1), (dict(cols=0), 1), (dict(cu=None), 1), (dict(kv_len=None), 1),
               (dict(table=None), 1), (dict(s_table=3), 1), (dict(cols=1 << 27, s_table=1 << 27), 2), (dict(T=1 << 30), 2),
               (dict(cols=1 << 26, s_table=1 << 26), 2)]


def _append(L, cache, batch, K=FAKE, V=FAKE, s_n=256, s_h=128, codes=(FAKE,) * 4):
    return L.vc_cache_append(K, V, s_n, s_h, cache, *codes, batch, None, None)


def _read(L, cache, batch, K=FAKE, V=FAKE, s_n=256, s_h=128, codes=(FAKE,) * 4):
    return L.vc_cache_read(cache, *codes, batch, K, V, s_n, s_h, None, None)


def _attn(L, cache, batch, Q=FAKE, O=FAKE, Hq=4, q=(512, 128), o=(512, 128), scale=0.0, causal=1, window=0, max_q=0,
          lse=FAKE, ws=FAKE, ws_bytes=1 << 40, codes=(FAKE,) * 4):
    return L.vc_attn_paged(Q, *q, Hq, cache, *codes, batch, scale, causal, window, max_q, O, *o, lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("call", [_append, _read, _attn])
def test_shared_refusals(L, call):
    for kw, code in BAD_SHAPES:
        assert call(L, _cache(**kw), _batch()) == code, kw
    for kw, code in BAD_BATCHES:
        assert call(L, _cache(), _batch(**kw)) == code, kw
    for i in range(4):
        for bad in (None, ODD):
            codes = [FAKE] * 4
            codes[i] = bad
            assert call(L, _cache(), _batch(), codes=codes) == 1, i
    # a call without rows has nothing to do, whatever its pointers are
    assert call(L, _cache(), _batch(T=0, cu=None), codes=(None,) * 4) == 0


@pytest.mark.parametrize("call", [_append, _read])
def test_row_refusals(L, call):
    for kw in (dict(K=None), dict(V=None), dict(K=ODD), dict(V=ODD), dict(s_n=0), dict(s_n=100), dict(s_h=-128), dict(s_h=4)):
        assert call(L, _cache(), _batch(), **kw) == 1, kw


def test_attention_refusals(L):
    for kw in (dict(Q=None), dict(O=None), dict(Q=ODD), dict(O=ODD), dict(Hq=0), dict(Hq=3), dict(q=(0, 128)), dict(q=(512, 4)),
               dict(o=(-8, 128)), dict(o=(512, 0)), dict(scale=math.nan), dict(scale=math.inf), dict(causal=2), dict(causal=-1),
               dict(window=-1), dict(max_q=-1), dict(lse=ctypes.c_void_p(0x10002))):
        assert _attn(L, _cache(), _batch(), **kw) == 1, kw
    assert _attn(L, _cache(), _batch(T=1 << 28), Hq=16) == 2
    assert _attn(L, _cache(), _batch(T=1 << 28), Hq=4) == 2
    need = L.vc_attn_paged_workspace(_cache(), 4, 3, 7, 0)
    if need:
        assert _attn(L, _cache(), _batch(), ws=None) == 3
        assert _attn(L, _cache(), _batch(), ws=ctypes.c_void_p(0x10080)) == 3
        assert _attn(L, _cache(), _batch(), ws_bytes=need - 1) == 3
    assert L.vc_attn_paged_workspace(_cache(d=96), 4, 3, 7, 0) == 0
    assert L.vc_attn_paged_workspace(_cache(), 3, 3, 7, 0) == 0


def test_binding_refusals(L):
    c = Case(n=[2], kv=[5], H=2)
    cache, args = c.cache(), c.args("cpu")
    bf = torch.bfloat16
    for bad in (c.K.float(), c.K[:, :1], c.K[..., :64], c.K[0], c.K.transpose(0, 2)):
        with pytest.raises(ValueError):
            vc.vc_cache_append(bad, c.V, cache, *args)
    with pytest.raises(ValueError, match="CUDA"):       # tensors on the CPU: nothing runs on the host
        vc.vc_cache_append(c.K, c.V, cache, *args)
    with pytest.raises(ValueError, match="CUDA"):
        vc.vc_cache_read(cache, *args, 2)
    with pytest.raises(ValueError, match="CUDA"):
        vc.vc_attn_paged(c.Q, cache, *args)
    for name, i, bad in (("cu", 0, args[0].long()), ("cu", 0, args[0][:1]), ("kv_len", 1, args[1].float()), ("table", 2, args[2][0])):
        a = list(args)
        a[i] = bad
        with pytest.raises(ValueError):
            vc.vc_attn_paged(c.Q, cache, *a)
    for k, bad in (("K8", cache["K8"].to(torch.int8)), ("sv", cache["sv"].double()), ("V8", cache["V8"][:1]), ("sk", cache["sk"][:, :1])):
        with pytest.raises(ValueError):
            vc.vc_cache_read({**cache, k: bad}, *args, 2)
    with pytest.raises(ValueError):
        vc.vc_attn_paged(c.Q, cache, *args, dev_status=torch.zeros(1))
    assert vc.cache_shape_of(cache).s_head == 16 * 128 and bf == c.Q.dtype


def test_encode_is_the_nearest_value():
    """The tests' encoder against every midpoint and its neighbours."""
    pos = E4M3[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    assert torch.equal(encode(pos), torch.arange(127, dtype=torch.uint8))
    even = torch.where(torch.arange(126) % 2 == 0, torch.arange(126), torch.arange(126) + 1).to(torch.uint8)
    assert torch.equal(encode(mid), even)
    assert torch.equal(encode(mid * (1 + 1e-9)), torch.arange(1, 127, dtype=torch.uint8))
    assert torch.equal(encode(-mid * (1 - 1e-9)), torch.arange(126, dtype=torch.uint8) + 128)


def test_definition_of_attention():
    """Case.attend against torch's softmax on the dequantized keys, for a case with every mask."""
    c = Case(n=[3, 2], kv=[40, 2], H=2, G=2, d=64, seed=1)
    cache = c.appended()
    for causal, window in ((1, 0), (0, 0), (1, 5), (0, 7)):
        O, _, lse, _ = c.attend(cache, causal, window)
        for r, b, p in c.places():
            for hq in range(4):
                kc, ks, _ = c.sequence(cache, "K8", "sk", b, hq // 2)
                vc_, vs, _ = c.sequence(cache, "V8", "sv", b, hq // 2)
                hi = p if causal else c.kv[b] - 1
                lo = max(0, hi - window + 1) if window else 0
                s = (kc * ks[:, None])[lo:hi + 1] @ c.Q[r, hq].double() / 8.0
                assert torch.allclose(O[r, hq], torch.softmax(s, 0) @ (vc_ * vs[:, None])[lo:hi + 1], atol=1e-12)
                assert abs(float(torch.logsumexp(s, 0) - lse[r, hq])) < 1e-12


def test_quantize_definition():
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[1, 0], x[2, 5] = 2.0, -1.0, 2.0 ** -101, math.inf
    codes, scale = quantize(x)
    assert codes[0, 0] == 0x7E and codes[0, 1] == 0x80 | 0x76 and scale[0] == torch.tensor(2.0) / 448.0
    assert scale[1] == 0 and not codes[1].any() and math.isnan(scale[2]) and not codes[2].any()

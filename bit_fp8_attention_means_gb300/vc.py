"""Thin ctypes binding over libvc_gb300.so (the C ABI in include/vc.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
fallback: if the library has not been built, every call raises.
"""
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvc_gb300.so")
BLOCK = 128

STATUS = {0: "VC_OK", 1: "VC_ERR_INVALID_ARG", 2: "VC_ERR_UNSUPPORTED", 3: "VC_ERR_WORKSPACE",
          4: "VC_ERR_CUDA", 5: "VC_ERR_TIMEOUT"}


class VcError(RuntimeError):
    def __init__(self, code, where):
        super().__init__("%s failed: %s" % (where, STATUS.get(code, code)))
        self.code = code


class VcShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("s_b", ctypes.c_int64), ("s_n", ctypes.c_int64), ("s_h", ctypes.c_int64)]


class VcCacheShape(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("H", ctypes.c_int32), ("d", ctypes.c_int32),
                ("s_page", ctypes.c_int64), ("s_head", ctypes.c_int64), ("s_tok", ctypes.c_int64),
                ("t_page", ctypes.c_int64), ("t_head", ctypes.c_int64)]


class VcBatch(ctypes.Structure):
    _fields_ = [("cu", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("cols", ctypes.c_int32), ("s_table", ctypes.c_int64)]


_lib = None
_vp = ctypes.c_void_p


def lib():
    """Load the CUDA library; raises if it was not built (no silent fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libvc_gb300.so is missing: build it with `python -c \"import __graft_entry__ as g; "
                               "g.build()\"` (nvcc, sm_103a)")
        L = ctypes.CDLL(LIB_PATH)
        L.vc_status_string.restype = ctypes.c_char_p
        L.vc_status_string.argtypes = [ctypes.c_int]
        L.vc_version.restype = ctypes.c_int
        L.vc_cluster_workspace.restype = ctypes.c_size_t
        L.vc_cluster_workspace.argtypes = [VcShape, ctypes.c_int]
        L.vc_cluster.restype = ctypes.c_int
        L.vc_cluster.argtypes = [_vp, VcShape, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp,
                                 ctypes.c_size_t, _vp, _vp]
        L.vc_cluster_ex.restype = ctypes.c_int
        L.vc_cluster_ex.argtypes = [_vp, VcShape, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp,
                                    _vp, _vp, ctypes.c_size_t, _vp, _vp]
        L.vc_quantize_workspace.restype = ctypes.c_size_t
        L.vc_quantize_workspace.argtypes = [VcShape]
        L.vc_quantize.restype = ctypes.c_int
        L.vc_quantize.argtypes = [_vp, _vp, _vp, VcShape, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, ctypes.c_size_t, _vp]
        L.vc_quantize_ex.restype = ctypes.c_int
        L.vc_quantize_ex.argtypes = [_vp, _vp, _vp, VcShape, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _vp, _vp,
                                     _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.vc_quantize_v4.restype = ctypes.c_int
        L.vc_quantize_v4.argtypes = L.vc_quantize.argtypes
        L.vc_quantize_staged_workspace.restype = ctypes.c_size_t
        L.vc_quantize_staged_workspace.argtypes = [VcShape]
        L.vc_quantize_staged.restype = ctypes.c_int
        L.vc_quantize_staged.argtypes = L.vc_quantize_ex.argtypes
        L.vc_attn_fwd.restype = ctypes.c_int
        L.vc_attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, VcShape, ctypes.c_float, ctypes.c_int,
                                  ctypes.c_int, _vp, _vp, _vp]
        L.vc_attn_fwd_hybrid.restype = ctypes.c_int
        L.vc_attn_fwd_hybrid.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, VcShape, ctypes.c_float,
                                         ctypes.c_float, ctypes.c_int, _vp, _vp, _vp]
        L.vc_attn_fwd_debug.restype = ctypes.c_int
        L.vc_attn_fwd_debug.argtypes = L.vc_attn_fwd.argtypes + [ctypes.c_int, ctypes.c_int, _vp, _vp,
                                                                 ctypes.c_float]
        L.vc_cache_append.restype = ctypes.c_int
        L.vc_cache_append.argtypes = [_vp, _vp, ctypes.c_int64, ctypes.c_int64, VcCacheShape, _vp, _vp, _vp, _vp,
                                      VcBatch, _vp, _vp]
        L.vc_cache_read.restype = ctypes.c_int
        L.vc_cache_read.argtypes = [VcCacheShape, _vp, _vp, _vp, _vp, VcBatch, _vp, _vp, ctypes.c_int64,
                                    ctypes.c_int64, _vp, _vp]
        L.vc_attn_paged_workspace.restype = ctypes.c_size_t
        L.vc_attn_paged_workspace.argtypes = [VcCacheShape, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.vc_attn_paged.restype = ctypes.c_int
        L.vc_attn_paged.argtypes = [_vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, VcCacheShape, _vp, _vp, _vp,
                                    _vp, VcBatch, ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp,
                                    ctypes.c_int64, ctypes.c_int64, _vp, _vp, ctypes.c_size_t, _vp, _vp]
        L.vc_debug_attn_paged_timeout.restype = ctypes.c_int
        L.vc_debug_attn_paged_timeout.argtypes = [_vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, VcCacheShape, _vp,
                                                  _vp, _vp, _vp, VcBatch, ctypes.c_int, _vp, ctypes.c_int64,
                                                  ctypes.c_int64, _vp, ctypes.c_size_t, _vp, _vp, ctypes.c_int]
        L.vc_debug_e4m3_encode.restype = ctypes.c_int
        L.vc_debug_e4m3_encode.argtypes = [_vp, ctypes.c_int64, _vp, _vp]
        L.vc_debug_wait_timeout.restype = ctypes.c_int
        L.vc_debug_wait_timeout.argtypes = [_vp, ctypes.c_uint32, _vp]
        L.vc_debug_attn_timeout.restype = ctypes.c_int
        L.vc_debug_attn_timeout.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, VcShape, ctypes.c_int, _vp, _vp, _vp,
                                            ctypes.c_int, ctypes.c_uint32]
        _lib = L
    return _lib


def _check(code, where):
    if code != 0:
        raise VcError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(stream, call, *args, **kw):
    """call(*args, **kw) with `stream` as the current one, for an entry point that makes outputs or a workspace.

    They come from the memory of `stream` then.  From that of the caller's stream they could be
    what its kernels, still under way, read or write: `stream` does not wait for those.  The
    caller's stream is to use the outputs, so their memory is kept until it has."""
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(caller)
    return out


def _is_other(stream):
    """Whether a call's `stream` is another than the current one."""
    return stream is not None and stream != torch.cuda.current_stream(stream.device)


def nblk_of(N):
    return (N + BLOCK - 1) // BLOCK


def shape_of(X: torch.Tensor) -> VcShape:
    """[B, N, H, d] bf16 tensor with unit channel stride -> vc_shape."""
    if X.dim() != 4 or X.stride(3) != 1:
        raise ValueError("expected [B, N, H, d] with unit channel stride")
    B, N, H, d = X.shape
    return VcShape(B, H, N, d, X.stride(0), X.stride(1), X.stride(2))


def _empty(shape, dtype, device, fill=None):
    t = torch.empty(shape, dtype=dtype, device=device)
    if fill is not None:
        t.fill_(fill)
    return t


def quantize_workspace_bytes(shape: VcShape) -> int:
    return lib().vc_quantize_workspace(shape)


def cluster_workspace_bytes(shape: VcShape, k: int) -> int:
    return lib().vc_cluster_workspace(shape, k)


def _workspace(nbytes, device):
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def vc_cluster(V, k, iters, warm_start=False, centroids=None, labels=None, perm=None, workspace=None,
               dev_status=None, stream=None, block_fill=0):
    """Grouping step. Returns (centroids fp32 [B,H,k,d], labels int32 [B,H,N], perm int32 [B,H,N]).

    block_fill=1 calls vc_cluster_ex: perm keeps whole 128-token blocks per
    cluster and chains the clusters' leftovers by centroid distance."""
    if _is_other(stream):
        return _on_stream(stream, vc_cluster, V, k, iters, warm_start, centroids, labels, perm, workspace, dev_status,
                          block_fill=block_fill)
    s = shape_of(V)
    dev = V.device
    if centroids is None:
        if warm_start:
            raise ValueError("warm start needs centroids")
        centroids = _empty((s.B, s.H, k, s.d), torch.float32, dev)
    if labels is None:
        labels = _empty((s.B, s.H, s.N), torch.int32, dev)
    if perm is None:
        perm = _empty((s.B, s.H, s.N), torch.int32, dev)
    need = lib().vc_cluster_workspace(s, k)
    if workspace is None:
        workspace = _workspace(need, dev)
    if block_fill:
        rc = lib().vc_cluster_ex(_ptr(V), s, k, iters, int(bool(warm_start)), int(block_fill), _ptr(centroids),
                                 _ptr(labels), _ptr(perm), _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                 _stream(stream))
        _check(rc, "vc_cluster_ex")
        return centroids, labels, perm
    rc = lib().vc_cluster(_ptr(V), s, k, iters, int(bool(warm_start)), _ptr(centroids), _ptr(labels), _ptr(perm),
                          _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    _check(rc, "vc_cluster")
    return centroids, labels, perm


def alloc_quantized(shape: VcShape, device, vsmooth=1):
    nb = nblk_of(shape.N)
    npad = nb * BLOCK
    B, H, d = shape.B, shape.H, shape.d
    return dict(
        Q8=_empty((B, H, npad, d), torch.uint8, device), sq=_empty((B, H, nb), torch.float32, device),
        K8=_empty((B, H, npad, d), torch.uint8, device), sk=_empty((B, H, nb), torch.float32, device),
        V8T=_empty((B, H, d, npad), torch.uint8, device), sv=_empty((B, H, d), torch.float32, device),
        mu=_empty((B, H, nb, d), torch.int16, device) if vsmooth else None)


def _check_qkv(Q, K, V):
    s = shape_of(Q)
    if shape_of(K).N != s.N or shape_of(V).N != s.N:
        raise ValueError("Q, K, V shapes differ")
    if (K.stride(), V.stride()) != (Q.stride(), Q.stride()):
        raise ValueError("Q, K, V must share strides")
    return s


def _check_rope(rope, s: VcShape):
    if rope is None:
        return
    if rope.dtype != torch.float32 or tuple(rope.shape) != (s.N, s.d // 2, 2) or not rope.is_contiguous():
        raise ValueError("rope must be a contiguous fp32 [N, d/2, 2] (cos, sin) table")


def _quantize_call(fn, name, Q, K, V, perm, vsmooth, rope, hadamard, out, workspace, need, stream):
    s = _check_qkv(Q, K, V)
    _check_rope(rope, s)
    dev = Q.device
    if out is None:
        out = alloc_quantized(s, dev, vsmooth)
    if workspace is None:
        workspace = _workspace(need(s), dev)
    args = [_ptr(Q), _ptr(K), _ptr(V), s, _ptr(perm), int(vsmooth), _ptr(rope), int(hadamard),
             _ptr(out["Q8"]), _ptr(out["sq"]), _ptr(out["K8"]), _ptr(out["sk"]), _ptr(out["V8T"]), _ptr(out["sv"]),
             _ptr(out["mu"]) if vsmooth else None, _ptr(workspace), workspace.numel(), _stream(stream)]
    _check(fn(*args), name)
    return out


def vc_quantize(Q, K, V, perm=None, vsmooth=1, out=None, workspace=None, stream=None, vbits=8):
    """Fused quantizer. Returns a dict with Q8, sq, K8, sk, V8T, sv, mu (mu is bf16 bits as int16).
    vbits=4 calls vc_quantize_v4: the V residual in 4 bits (E2M1 with a power-of-two
    scale per 32 tokens of a channel), stored as E4M3 bytes for vc_attn_fwd."""
    if _is_other(stream):
        return _on_stream(stream, vc_quantize, Q, K, V, perm, vsmooth, out, workspace, vbits=vbits)
    L = lib()
    s = _check_qkv(Q, K, V)
    dev = Q.device
    if out is None:
        out = alloc_quantized(s, dev, vsmooth)
    if workspace is None:
        workspace = _workspace(L.vc_quantize_workspace(s), dev)
    if vbits not in (4, 8):
        raise ValueError("vbits must be 4 or 8")
    fn, name = (L.vc_quantize_v4, "vc_quantize_v4") if vbits == 4 else (L.vc_quantize, "vc_quantize")
    rc = fn(_ptr(Q), _ptr(K), _ptr(V), s, _ptr(perm), int(vsmooth), _ptr(out["Q8"]),
            _ptr(out["sq"]), _ptr(out["K8"]), _ptr(out["sk"]), _ptr(out["V8T"]), _ptr(out["sv"]),
            _ptr(out["mu"]) if vsmooth else None, _ptr(workspace), workspace.numel(),
            _stream(stream))
    _check(rc, name)
    return out


def vc_quantize_ex(Q, K, V, perm=None, vsmooth=1, rope=None, hadamard=0, out=None, workspace=None, stream=None):
    """vc_quantize with the rotary transform (``rope``: fp32 [N, d/2, 2] (cos, sin)
    table on the device) and/or the Hadamard rotation of Q and K fused in."""
    if _is_other(stream):
        return _on_stream(stream, vc_quantize_ex, Q, K, V, perm, vsmooth, rope, hadamard, out, workspace)
    L = lib()
    return _quantize_call(L.vc_quantize_ex, "vc_quantize_ex", Q, K, V, perm, vsmooth, rope, hadamard, out,
                          workspace, L.vc_quantize_workspace, stream)


def vc_quantize_staged(Q, K, V, perm=None, vsmooth=1, rope=None, hadamard=0, out=None, workspace=None,
                       stream=None):
    """The same computation as vc_quantize_ex as the unfused chain of kernels
    (intermediates in device memory); bit-identical outputs."""
    if _is_other(stream):
        return _on_stream(stream, vc_quantize_staged, Q, K, V, perm, vsmooth, rope, hadamard, out, workspace)
    L = lib()
    return _quantize_call(L.vc_quantize_staged, "vc_quantize_staged", Q, K, V, perm, vsmooth, rope, hadamard, out,
                          workspace, L.vc_quantize_staged_workspace, stream)


def quantize_staged_workspace_bytes(shape: VcShape) -> int:
    return lib().vc_quantize_staged_workspace(shape)


def vc_attn_fwd(qz, shape: VcShape, softmax_scale=0.0, expcast=1, vsmooth=1, O=None, dev_status=None,
                stream=None, debug=None, exact_margin=None):
    """FP8 attention on vc_quantize outputs. O is bf16 [B,N,H,d] laid out with `shape`'s strides.

    exact_margin (float) selects the hybrid bytes (vc_attn_fwd_hybrid):
    exp-then-cast on the key tiles within that many log2 units of a row's
    running maximum, ExpCast elsewhere; expcast is then ignored.
    expcast: 0 exp-then-cast, 1 ExpCast, 3 range-adaptive ExpCast (a beta per
    pair of codes of the octave).
    debug=(bh, qtile) additionally returns the fp32 scores and probability bytes
    of that one query tile: (O, S_dump [128, Npad], P_dump [128, Npad]).
    """
    if _is_other(stream):
        return _on_stream(stream, vc_attn_fwd, qz, shape, softmax_scale, expcast, vsmooth, O, dev_status, debug=debug,
                          exact_margin=exact_margin)
    dev = qz["Q8"].device
    if O is None:
        O = torch.empty((shape.B, shape.N, shape.H, shape.d), dtype=torch.bfloat16, device=dev)
        if (O.stride(0), O.stride(1), O.stride(2)) != (shape.s_b, shape.s_n, shape.s_h):
            O = torch.empty_strided((shape.B, shape.N, shape.H, shape.d), (shape.s_b, shape.s_n, shape.s_h, 1),
                                    dtype=torch.bfloat16, device=dev)
    ops = [_ptr(qz["Q8"]), _ptr(qz["sq"]), _ptr(qz["K8"]), _ptr(qz["sk"]), _ptr(qz["V8T"]), _ptr(qz["sv"]),
           _ptr(qz["mu"]) if vsmooth else None, shape, float(softmax_scale)]
    tail = [_ptr(O), _ptr(dev_status), _stream(stream)]
    if exact_margin is not None:
        expcast = 2
    if debug is None:
        if exact_margin is not None:
            _check(lib().vc_attn_fwd_hybrid(*ops, float(exact_margin), int(vsmooth), *tail), "vc_attn_fwd_hybrid")
        else:
            _check(lib().vc_attn_fwd(*ops, int(expcast), int(vsmooth), *tail), "vc_attn_fwd")
        return O
    npad = nblk_of(shape.N) * BLOCK
    S = torch.zeros((BLOCK, npad), dtype=torch.float32, device=dev)
    P = torch.zeros((BLOCK, npad), dtype=torch.uint8, device=dev)
    _check(lib().vc_attn_fwd_debug(*ops, int(expcast), int(vsmooth), *tail, int(debug[0]), int(debug[1]), _ptr(S),
                                   _ptr(P), float(exact_margin or 0.0)), "vc_attn_fwd_debug")
    return O, S, P


# ------------------------------------------------------------ paged cache

_U8, _F32, _I32, _BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16
_LEAST_FP32 = 2.0 ** -149


def alloc_cache(pages, page_size, H, d, device):
    """A page pool for vc_cache_append, vc_cache_read and vc_attn_paged: dict of K8, V8 (E4M3 bytes
    [pages, H, page_size, d]) and their scales sk, sv (fp32 [pages, H, page_size]), zeroed.

    Any tensors of these shapes and types do, in any order of the first three
    dimensions of K8 and V8 (as views, e.g. one half of a joint pool): the
    channels and the scales' tokens have to be contiguous, the strides of K8
    and V8 equal, and those of sk and sv too."""
    c = {}
    for code, scale in (("K8", "sk"), ("V8", "sv")):
        c[code] = _empty((pages, H, page_size, d), torch.uint8, device, 0)
        c[scale] = _empty((pages, H, page_size), torch.float32, device, 0)
    return c


def _cache_parts(cache):
    """Checks a dict of K8, sk, V8, sv (see alloc_cache): its vc_cache_shape, the four pointers, the device's index."""
    K8, V8, sk, sv = cache["K8"], cache["V8"], cache["sk"], cache["sv"]
    shape, k, t = K8.shape, K8.stride(), sk.stride()
    if len(shape) != 4 or K8.dtype is not _U8 or V8.dtype is not _U8 or V8.shape != shape:
        raise ValueError("K8 and V8 must be uint8 [pages, H, page_size, d]")
    pages, H, page, d = shape
    if sk.dtype is not _F32 or sv.dtype is not _F32 or sk.shape != (pages, H, page) or sv.shape != (pages, H, page):
        raise ValueError("sk and sv must be fp32 [pages, H, page_size]")
    v, u = V8.stride(), sv.stride()
    if pages < 2 or H < 2:  # a dimension of one element may have any stride: it gets a legal one
        k, v = _plain_strides(shape, k, d), _plain_strides(shape, v, d)
        t, u = _plain_strides(shape[:3], t, page), _plain_strides(shape[:3], u, page)
    if v != k or u != t:
        raise ValueError("K8 and V8, and sk and sv, must share strides")
    if (k[3] != 1 or t[2] != 1) and min(shape) > 0:
        raise ValueError("channels and the scales' tokens must be contiguous")
    dev = K8.get_device()
    if V8.get_device() != dev or sk.get_device() != dev or sv.get_device() != dev:
        raise ValueError("the cache's tensors are on different devices")
    return (VcCacheShape(pages, page, H, d, k[0], k[1], k[2], t[0], t[1]),
            (K8.data_ptr(), sk.data_ptr(), V8.data_ptr(), sv.data_ptr()), dev)


def _plain_strides(shape, strides, unit):
    """`strides`, with `unit` in the place of an outer dimension's of one element."""
    return tuple(s if n > 1 or i >= 2 else unit for i, (n, s) in enumerate(zip(shape, strides)))


def cache_shape_of(cache) -> VcCacheShape:
    """The vc_cache_shape of a dict of K8, sk, V8, sv (see alloc_cache)."""
    return _cache_parts(cache)[0]


def _batch_of(cu, kv_len, table, T, dev) -> VcBatch:
    c = table.shape
    if cu.dtype is not _I32 or kv_len.dtype is not _I32 or table.dtype is not _I32 or len(c) != 2 or \
            cu.dim() != 1 or kv_len.dim() != 1:
        raise ValueError("cu [B+1], kv_len [B] and table [B, cols] must be int32")
    B, cols = c
    if cu.numel() != B + 1 or kv_len.numel() != B:
        raise ValueError("cu, kv_len and table disagree on the number of sequences")
    s = table.stride()
    if cu.stride(0) != 1 or (B > 1 and kv_len.stride(0) != 1) or (s[1] != 1 and cols > 1):
        raise ValueError("cu, kv_len and the rows of table must be contiguous")
    if cu.get_device() != dev or kv_len.get_device() != dev or table.get_device() != dev:
        raise ValueError("cu, kv_len or table is not on the cache's device")
    return VcBatch(cu.data_ptr(), kv_len.data_ptr(), table.data_ptr(), B, T, cols, s[0] if B > 1 else max(cols, 1))


def _rows(name, t, H, d, dev):
    """Checks a bf16 [T, H, d] tensor with contiguous channels: its row and head strides."""
    shape, s = t.shape, t.stride()
    if t.dtype is not _BF16 or len(shape) != 3 or shape[1] != H or shape[2] != d:
        raise ValueError("%s must be bf16 [T, %d, %d]" % (name, H, d))
    if s[2] != 1:
        raise ValueError("%s must have contiguous channels" % name)
    if t.get_device() != dev:
        raise ValueError("%s is not on the cache's device" % name)
    return s[0] if shape[0] > 1 else H * d, s[1] if H > 1 else d


def _status_ptr(dev_status, dev):
    if dev_status is None:
        return None
    if dev_status.dtype != torch.int32 or dev_status.numel() < 1 or dev_status.get_device() != dev:
        raise ValueError("dev_status must be int32 on the cache's device")
    return dev_status.data_ptr()


def _on_device(dev, stream, fn, args, where):
    """Calls fn(*args, stream) with device `dev` current."""
    here = torch._C._cuda_getDevice()
    if here != dev:
        torch.cuda.set_device(dev)
    try:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream), where)
    finally:
        if here != dev:
            torch.cuda.set_device(here)


def _check_stream(stream, dev):
    if stream is not None and stream.device.index != dev:
        raise ValueError("stream is not on the cache's device")


def _int32(x):
    """The number itself or the nearest that a C int holds: ctypes would drop the upper bits."""
    return x if -1 <= x <= 0x7FFFFFFF else max(-1, min(x, 0x7FFFFFFF))


def _need_cuda(dev):
    if dev < 0:
        raise ValueError("the cache must be on a CUDA device")


def vc_cache_append(K, V, cache, cu, kv_len, table, dev_status=None, stream=None):
    """Quantizes new keys and values (bf16 [T, H, d]) into the pages of `cache` (see alloc_cache).

    cu int32 [B+1], kv_len int32 [B], table int32 [B, cols]: sequence b has
    rows cu[b] .. cu[b+1]-1 of the call and kv_len[b] tokens in the cache with
    these included; position p lies in page table[b, p // page_size].
    stream: where this and the other calls run, if not the current one.  It has to have waited for
    what is handed in; what a call makes itself, its workspace too, is of that stream's memory."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    strides = _rows("K", K, s.H, s.d, dev)
    if V.shape != K.shape or _rows("V", V, s.H, s.d, dev) != strides:
        raise ValueError("K and V must share shape and strides")
    batch = _batch_of(cu, kv_len, table, K.shape[0], dev)
    status = _status_ptr(dev_status, dev)
    _need_cuda(dev)
    _check_stream(stream, dev)
    _on_device(dev, stream, L.vc_cache_append, (K.data_ptr(), V.data_ptr(), *strides, s, K8, sk, V8, sv, batch, status),
               "vc_cache_append")
    return cache


def vc_cache_read(cache, cu, kv_len, table, T, K=None, V=None, dev_status=None, stream=None):
    """Reads cached tokens back as bf16 [T, H, d] (K, V): the rows that vc_cache_append would write.
    Rows of no sequence stay as they are in K and V given, and hold anything in new ones."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    batch = _batch_of(cu, kv_len, table, T, dev)
    status = _status_ptr(dev_status, dev)
    _need_cuda(dev)
    _check_stream(stream, dev)
    if _is_other(stream):
        return _on_stream(stream, vc_cache_read, cache, cu, kv_len, table, T, K, V, dev_status)
    if K is None:
        K = torch.empty((T, s.H, s.d), dtype=_BF16, device=dev)  # half the time of new_empty
    if V is None:
        V = torch.empty_like(K) if K.is_contiguous() else K.new_empty_strided(K.shape, K.stride())
    strides = _rows("K", K, s.H, s.d, dev)
    if K.shape[0] != T or V.shape != K.shape or _rows("V", V, s.H, s.d, dev) != strides:
        raise ValueError("K and V must have T rows and share strides")
    _on_device(dev, stream, L.vc_cache_read, (s, K8, sk, V8, sv, batch, K.data_ptr(), V.data_ptr(), *strides, status),
               "vc_cache_read")
    return K, V


@functools.lru_cache(maxsize=256)
def _attn_paged_bytes(page_size, H, d, Hq, B, T, max_q):
    """vc_attn_paged_workspace, which depends on these numbers alone."""
    s = VcCacheShape(1, page_size, H, d, H * page_size * d, page_size * d, d, H * page_size, page_size)
    return lib().vc_attn_paged_workspace(s, Hq, B, T, max_q)


def attn_paged_workspace_bytes(cache, Hq, B, T, max_q=0) -> int:
    return lib().vc_attn_paged_workspace(cache_shape_of(cache), Hq, B, T, _int32(max_q))


def vc_attn_paged(Q, cache, cu, kv_len, table, softmax_scale=0.0, causal=1, window=0, max_q=0, O=None, lse=None,
                  workspace=None, dev_status=None, stream=None):
    """Attention of the call's queries (bf16 [T, Hq, d]) over the paged cache, their own keys included:
    append them first.  Returns (O bf16 [T, Hq, d], lse fp32 [T, Hq]).

    cu, kv_len, table as in vc_cache_append.  causal=0: a row sees all of its
    sequence's keys; window > 0: only the last `window` of those it would see.
    max_q: the longest chunk among the sequences, if known (it chooses the
    kernel, nothing else).  Rows of no sequence stay as they are in O and lse."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    shape = Q.shape
    if len(shape) != 3:
        raise ValueError("Q must be bf16 [T, Hq, %d]" % s.d)
    T, Hq, d = shape
    q_strides = _rows("Q", Q, Hq, s.d, dev)
    batch = _batch_of(cu, kv_len, table, T, dev)
    status = _status_ptr(dev_status, dev)
    _need_cuda(dev)
    _check_stream(stream, dev)
    if _is_other(stream):
        return _on_stream(stream, vc_attn_paged, Q, cache, cu, kv_len, table, softmax_scale, causal, window, max_q, O,
                          lse, workspace, dev_status)
    window, max_q = _int32(window), _int32(max_q)
    if 0 < softmax_scale < _LEAST_FP32:  # as fp32 it would be 0, the default
        softmax_scale = _LEAST_FP32
    if O is None:
        O = torch.empty(shape, dtype=_BF16, device=dev)
        o_strides = (Hq * d, d)
    else:
        o_strides = _rows("O", O, Hq, d, dev)
        if O.shape != shape:
            raise ValueError("O must have Q's shape")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=_F32, device=dev)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (T, Hq) or not lse.is_contiguous() or \
            lse.get_device() != dev:
        raise ValueError("lse must be contiguous fp32 [T, Hq] on the cache's device")
    if workspace is None:
        workspace = torch.empty(max(_attn_paged_bytes(s.page_size, s.H, d, Hq, batch.B, T, max_q), 256), dtype=_U8,
                                device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    _on_device(dev, stream, L.vc_attn_paged,
               (Q.data_ptr(), *q_strides, Hq, s, K8, sk, V8, sv, batch, softmax_scale, causal, window, max_q,
                O.data_ptr(), *o_strides, lse.data_ptr(), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), status), "vc_attn_paged")
    return O, lse


def vc_debug_e4m3_encode(x: torch.Tensor, out=None, stream=None):
    if _is_other(stream):
        return _on_stream(stream, vc_debug_e4m3_encode, x, out)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(lib().vc_debug_e4m3_encode(_ptr(x), x.numel(), _ptr(out), _stream(stream)), "vc_debug_e4m3_encode")
    return out


def vc_debug_wait_timeout(dev_status: torch.Tensor, timeout_us: int, stream=None):
    _check(lib().vc_debug_wait_timeout(_ptr(dev_status), int(timeout_us), _stream(stream)), "vc_debug_wait_timeout")


def vc_debug_attn_timeout(qz, shape: VcShape, dev_status: torch.Tensor, skip_k_tile: int, timeout_us: int,
                          vsmooth=1, O=None, stream=None):
    """vc_attn_fwd whose K loader never delivers key tile `skip_k_tile`, every
    device wait bounded by timeout_us: the kernel must record VC_ERR_TIMEOUT in
    dev_status and return.  Returns O (unspecified contents)."""
    if _is_other(stream):
        return _on_stream(stream, vc_debug_attn_timeout, qz, shape, dev_status, skip_k_tile, timeout_us, vsmooth, O)
    if O is None:
        O = torch.empty((shape.B, shape.N, shape.H, shape.d), dtype=torch.bfloat16, device=qz["Q8"].device)
    _check(lib().vc_debug_attn_timeout(_ptr(qz["Q8"]), _ptr(qz["sq"]), _ptr(qz["K8"]), _ptr(qz["sk"]),
                                       _ptr(qz["V8T"]), _ptr(qz["sv"]), _ptr(qz["mu"]) if vsmooth else None, shape,
                                       int(vsmooth), _ptr(O), _ptr(dev_status), _stream(stream), int(skip_k_tile),
                                       int(timeout_us)), "vc_debug_attn_timeout")
    return O


def vc_debug_attn_paged_timeout(Q, cache, cu, kv_len, table, dev_status, skip_unit, max_q=0, stream=None):
    """vc_attn_paged whose loaders leave out the keys of each CTA's unit `skip_unit`: it must record
    VC_ERR_TIMEOUT in dev_status, after about a quarter of a second, and return.  Returns O (unspecified)."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    T, Hq, d = Q.shape
    strides, batch = _rows("Q", Q, Hq, s.d, dev), _batch_of(cu, kv_len, table, T, dev)
    status = _status_ptr(dev_status, dev)
    _need_cuda(dev)
    _check_stream(stream, dev)
    if _is_other(stream):
        return _on_stream(stream, vc_debug_attn_paged_timeout, Q, cache, cu, kv_len, table, dev_status, skip_unit,
                          max_q)
    O = torch.empty((T, Hq, d), dtype=_BF16, device=dev)
    ws = _workspace(L.vc_attn_paged_workspace(s, Hq, batch.B, T, max_q), O.device)
    _on_device(dev, stream, lambda *args: L.vc_debug_attn_paged_timeout(*args, skip_unit),
               (Q.data_ptr(), *strides, Hq, s, K8, sk, V8, sv, batch, max_q, O.data_ptr(), Hq * d, d, ws.data_ptr(),
                ws.numel(), status), "vc_debug_attn_paged_timeout")
    return O

"""Thin ctypes binding over libvc_gb300.so (the C ABI in include/vc.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
fallback: if the library has not been built, every call raises.
"""
import ctypes
import functools
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvc_gb300.so")
BLOCK = 128

STATUS = {0: "VC_OK", 1: "VC_ERR_INVALID_ARG", 2: "VC_ERR_UNSUPPORTED", 3: "VC_ERR_WORKSPACE",
          4: "VC_ERR_CUDA", 5: "VC_ERR_TIMEOUT", 6: "VC_ERR_PAGES"}


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


class VcRopeSpec(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("magnitude", ctypes.c_float)]


class VcPool(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("free_pages", ctypes.c_void_p)]


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
        i32, i64 = ctypes.c_int, ctypes.c_int64
        L.vc_rope.restype = i32
        L.vc_rope.argtypes = [_vp, i64, i64, i32, i32, i32, VcRopeSpec, _vp, _vp, _vp, i32, i32, _vp, i64, i64, _vp, _vp]
        L.vc_cache_append_rope.restype = i32
        L.vc_cache_append_rope.argtypes = [_vp, i64, i64, i32, _vp, _vp, i64, i64, VcCacheShape, _vp, _vp, _vp, _vp, VcBatch,
                                           VcRopeSpec, _vp, _vp, i64, i64, _vp, _vp]
        L.vc_pages_reserve_workspace.restype = ctypes.c_size_t
        L.vc_pages_reserve_workspace.argtypes = [VcCacheShape, i32, i32]
        L.vc_pages_reserve.restype = i32
        L.vc_pages_reserve.argtypes = [VcCacheShape, _vp, _vp, _vp, _vp, VcPool, VcBatch, _vp, ctypes.c_size_t, _vp, _vp]
        L.vc_pages_fork.restype = i32
        L.vc_pages_fork.argtypes = [VcCacheShape, VcPool, _vp, i64, i32, i32, _vp, _vp, _vp, i32, _vp, i64, i32, _vp, _vp, _vp]
        L.vc_pages_trim.restype = i32
        L.vc_pages_trim.argtypes = [VcCacheShape, VcPool, _vp, i64, i32, i32, _vp, _vp, _vp, _vp]
        L.vc_pages_compact_workspace.restype = ctypes.c_size_t
        L.vc_pages_compact_workspace.argtypes = [VcCacheShape]
        L.vc_pages_compact.restype = i32
        L.vc_pages_compact.argtypes = [VcCacheShape, _vp, _vp, _vp, _vp, VcPool, _vp, i64, i32, i32, _vp, _vp,
                                       ctypes.c_size_t, _vp, _vp]
        L.vc_cache_copy.restype = i32
        L.vc_cache_copy.argtypes = [VcCacheShape, _vp, _vp, _vp, _vp, VcCacheShape, _vp, _vp, _vp, _vp, _vp, _vp, i32, _vp, _vp]
        L.vc_attn_paged_shared_workspace.restype = ctypes.c_size_t
        L.vc_attn_paged_shared_workspace.argtypes = [VcCacheShape, i32, i32, i32, i32, i32, i32]
        L.vc_attn_paged_shared.restype = i32
        L.vc_attn_paged_shared.argtypes = [_vp, i64, i64, i32, VcCacheShape, _vp, _vp, _vp, _vp, VcBatch, _vp, _vp, i32,
                                           ctypes.c_float, i32, i32, i32, _vp, i64, i64, _vp, _vp, ctypes.c_size_t, _vp, _vp]
        L.vc_debug_attn_paged_shared_timeout.restype = i32
        L.vc_debug_attn_paged_shared_timeout.argtypes = [_vp, i64, i64, i32, VcCacheShape, _vp, _vp, _vp, _vp, VcBatch, _vp, _vp, i32,
                                                         i32, i32, _vp, i64, i64, _vp, _vp, ctypes.c_size_t, _vp, _vp, i32, i32]
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


@functools.lru_cache(maxsize=256)
def _cache_shape(shape, sk_shape, k, t):
    """The vc_cache_shape of K8 (and V8) and sk (and sv) of these shapes and strides, which depends on them alone."""
    if len(shape) != 4:
        raise ValueError("K8 and V8 must be uint8 [pages, H, page_size, d]")
    pages, H, page, d = shape
    if sk_shape != (pages, H, page):
        raise ValueError("sk and sv must be fp32 [pages, H, page_size]")
    if pages < 2 or H < 2:  # a dimension of one element may have any stride: it gets a legal one
        k, t = _plain_strides(shape, k, d), _plain_strides(shape[:3], t, page)
    if (k[3] != 1 or t[2] != 1) and min(shape) > 0:
        raise ValueError("channels and the scales' tokens must be contiguous")
    return VcCacheShape(pages, page, H, d, k[0], k[1], k[2], t[0], t[1])


def _cache_parts(cache):
    """Checks a dict of K8, sk, V8, sv (see alloc_cache): its vc_cache_shape (not to be changed), the four pointers,
    the device's index."""
    K8, V8, sk, sv = cache["K8"], cache["V8"], cache["sk"], cache["sv"]
    if K8.dtype is not _U8 or V8.dtype is not _U8 or V8.shape != K8.shape:
        raise ValueError("K8 and V8 must be uint8 [pages, H, page_size, d]")
    if sk.dtype is not _F32 or sv.dtype is not _F32 or sv.shape != sk.shape:
        raise ValueError("sk and sv must be fp32 [pages, H, page_size]")
    shape, scales, k, t = K8.shape, sk.shape, K8.stride(), sk.stride()
    s = _cache_shape(shape, scales, k, t)
    v, u = V8.stride(), sv.stride()
    if v != k or u != t:  # they may differ where a dimension has one element
        page, d = shape[2:]
        if _plain_strides(shape, v, d) != _plain_strides(shape, k, d) or \
                _plain_strides(scales, u, page) != _plain_strides(scales, t, page):
            raise ValueError("K8 and V8, and sk and sv, must share strides")
    dev = K8.get_device()
    if V8.get_device() != dev or sk.get_device() != dev or sv.get_device() != dev:
        raise ValueError("the cache's tensors are on different devices")
    return s, (K8.data_ptr(), sk.data_ptr(), V8.data_ptr(), sv.data_ptr()), dev


def _plain_strides(shape, strides, unit):
    """`strides`, with `unit` in the place of an outer dimension's of one element."""
    return tuple(s if n > 1 or i >= 2 else unit for i, (n, s) in enumerate(zip(shape, strides)))


def cache_shape_of(cache) -> VcCacheShape:
    """The vc_cache_shape of a dict of K8, sk, V8, sv (see alloc_cache)."""
    return VcCacheShape.from_buffer_copy(_cache_parts(cache)[0])


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
        code = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    finally:
        if here != dev:
            torch.cuda.set_device(here)
    if code:
        raise VcError(code, where)


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


@functools.lru_cache(maxsize=256)
def _attn_shared_bytes(page_size, H, d, Hq, B, T, N, max_q, max_rows):
    """vc_attn_paged_shared_workspace, which depends on these numbers alone."""
    s = VcCacheShape(1, page_size, H, d, H * page_size * d, page_size * d, d, H * page_size, page_size)
    return lib().vc_attn_paged_shared_workspace(s, Hq, B, T, N, max_q, max_rows)


def attn_paged_shared_workspace_bytes(cache, Hq, B, T, N, max_q=0, max_rows=0) -> int:
    return lib().vc_attn_paged_shared_workspace(cache_shape_of(cache), Hq, B, T, N, _int32(max_q), _int32(max_rows))


def vc_attn_paged_shared(Q, cache, cu, kv_len, table, groups, prefix, softmax_scale=0.0, causal=1, max_q=0, max_rows=0,
                         O=None, lse=None, workspace=None, dev_status=None, stream=None):
    """vc_attn_paged (without a window) for sequences that begin alike, as forks do: groups int32 [N+1] are offsets of
    N runs of sequences, prefix int32 [N] how many tokens a run's sequences have in common, in the same pages but for
    the page that the prefix ends in.  Each prefix is read once for all rows of its run.  Returns (O, lse).

    A prefix holds none of the call's tokens; 0 and runs of one sequence are fine, as are sequences of no run, and
    sequences without tokens in the call, which may have ended.
    max_q: the longest chunk among the sequences, max_rows: the most tokens of this call in one run, if known (they
    choose kernels, nothing else)."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    shape = Q.shape
    if len(shape) != 3:
        raise ValueError("Q must be bf16 [T, Hq, %d]" % s.d)
    T, Hq, d = shape
    q_strides = _rows("Q", Q, Hq, s.d, dev)
    batch = _batch_of(cu, kv_len, table, T, dev)
    N = prefix.numel()
    runs = _int32_vector("groups", groups, N + 1, dev), _int32_vector("prefix", prefix, N, dev)
    status = _status_ptr(dev_status, dev)
    _check_place(stream, dev)
    if stream is not None and _is_other(stream):
        return _on_stream(stream, vc_attn_paged_shared, Q, cache, cu, kv_len, table, groups, prefix, softmax_scale, causal,
                          max_q, max_rows, O, lse, workspace, dev_status)
    max_q, max_rows = _int32(max_q), _int32(max_rows)
    if 0 < softmax_scale < _LEAST_FP32:  # as fp32 it would be 0, the default
        softmax_scale = _LEAST_FP32
    if O is None:
        o_strides = (Hq * d, d)
        O = _new_rows(Q, q_strides == o_strides, dev)
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
        workspace = torch.empty(max(_attn_shared_bytes(s.page_size, s.H, d, Hq, batch.B, T, N, max_q, max_rows), 256),
                                dtype=_U8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    _on_device(dev, stream, L.vc_attn_paged_shared,
               (Q.data_ptr(), *q_strides, Hq, s, K8, sk, V8, sv, batch, *runs, N, softmax_scale, causal, max_q, max_rows,
                O.data_ptr(), *o_strides, lse.data_ptr(), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), status), "vc_attn_paged_shared")
    return O, lse


def _new_rows(x, contiguous, dev):
    """A new contiguous tensor of x's shape and type (half the time of the general call where x is contiguous itself)."""
    return torch.empty_like(x) if contiguous else torch.empty(x.shape, dtype=_BF16, device=dev)


def _check_place(stream, dev):
    _need_cuda(dev)
    if stream is not None:
        _check_stream(stream, dev)


# ------------------------------------------------------------ rotary positions

_LAYOUTS = {"halves": 0, "pairs": 1}


def make_rope(rot, base=10000.0, layout="halves", scaling="none", factor=1.0, original=4096, slow=1.0, fast=32.0,
              magnitude=None, device="cuda"):
    """The angles of vc_rope and vc_cache_append_rope: a dict of turns (int64 [rot/2], turns a position as 64-bit
    fractions), layout and magnitude.

    rot: turned channels of a head (a multiple of 16).  layout "halves": pair i is channels (i, i + rot/2),
    "pairs": (2i, 2i + 1).  Pair i turns by w_i = base^(-2i/rot) radians a position, computed in fp64;
    scaling, for contexts `factor` times as long as the `original` ones:
      "positions"  w_i / factor;
      "base"       base times factor^(rot / (rot - 2)), so that the slowest pair turns 1/factor as fast;
      "ramp"       pairs that turn `fast` times or more over the original positions stay, those that turn `slow`
                   times or less are divided by factor, linear in the turns between, and magnitude is
                   0.1 ln factor + 1 unless it is given (1 for the others).
    A dict with other turns, made by hand, does as well."""
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'halves' or 'pairs'")
    if rot < 16 or rot % 16:
        raise ValueError("rot must be a multiple of 16")
    if not (base > 0 and factor > 0 and original > 0 and fast > slow):
        raise ValueError("base, factor and original must be positive, fast above slow")
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2.0))
    w = base ** (torch.arange(rot // 2, dtype=torch.float64) * (-2.0 / rot))
    if scaling == "positions":
        w = w / factor
    elif scaling == "ramp":
        keep = ((original * w / (2.0 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        w = w * keep + w / factor * (1.0 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0 if magnitude is None else magnitude
    elif scaling not in ("none", "base"):
        raise ValueError("scaling must be 'none', 'positions', 'base' or 'ramp'")
    turns = torch.round(torch.remainder(w / (2.0 * math.pi), 1.0) * 2.0 ** 62).to(torch.int64) << 2
    return dict(turns=turns.to(device), layout=layout, magnitude=1.0 if magnitude is None else float(magnitude))


def _rope_spec(rope, dev):
    turns = rope["turns"]
    if turns.dtype is not torch.int64 or turns.dim() != 1 or not turns.is_contiguous() or turns.numel() < 1:
        raise ValueError("rope's turns must be contiguous int64 [rot/2]")
    if turns.get_device() != dev:
        raise ValueError("rope's turns are not on the rows' device")
    if rope["layout"] not in _LAYOUTS:
        raise ValueError("rope's layout must be 'halves' or 'pairs'")
    return VcRopeSpec(turns.data_ptr(), 2 * turns.shape[0], _LAYOUTS[rope["layout"]], rope["magnitude"])


def _int32_vector(name, t, n, dev):
    """Checks an int32 vector of n elements: its pointer."""
    if t.dtype is not _I32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous int32 [%d]" % (name, n))
    if t.get_device() != dev:
        raise ValueError("%s is not on the other tensors' device" % name)
    return t.data_ptr()


def vc_rope(X, rope, pos=None, cu=None, kv_len=None, inverse=0, out=None, dev_status=None, stream=None):
    """X (bf16 [T, H, d]) turned by its rows' positions, for a `rope` of make_rope: pos int32 [T], or those of a
    batch (cu, kv_len as in vc_cache_append; rows of no sequence stay as they are in `out`).
    inverse=1: the transposed map, as for the gradient.  out: X itself to turn it in place."""
    L = lib()
    if X.dim() != 3:
        raise ValueError("X must be bf16 [T, H, d]")
    T, H, d = X.shape
    dev = X.get_device()
    strides = _rows("X", X, H, d, dev)
    spec = _rope_spec(rope, dev)
    if pos is None and cu is None:
        raise ValueError("vc_rope needs pos, or cu and kv_len")
    if (cu is None) != (kv_len is None):
        raise ValueError("cu and kv_len belong together")
    at = None if pos is None else _int32_vector("pos", pos, T, dev)
    B = 0 if cu is None else kv_len.numel()
    batch = (None, None) if cu is None else (_int32_vector("cu", cu, B + 1, dev), _int32_vector("kv_len", kv_len, B, dev))
    status = _status_ptr(dev_status, dev)
    _check_place(stream, dev)
    if stream is not None and _is_other(stream):
        return _on_stream(stream, vc_rope, X, rope, pos, cu, kv_len, inverse, out, dev_status)
    if out is None:
        o_strides = (H * d, d)
        out = _new_rows(X, strides == o_strides, dev)
    else:
        o_strides = _rows("out", out, H, d, dev)
        if out.shape[0] != T:
            raise ValueError("out must have X's shape")
    _on_device(dev, stream, L.vc_rope, (X.data_ptr(), *strides, T, H, d, spec, at, *batch, B, inverse, out.data_ptr(),
                                        *o_strides, status), "vc_rope")
    return out


def vc_cache_append_rope(Q, K, V, cache, cu, kv_len, table, rope, pos=None, out=None, dev_status=None, stream=None):
    """What comes before a step's attention, in one launch: returns Q (bf16 [T, Hq, d], or None) turned as by
    vc_rope, and quantizes the turned K and V (bf16 [T, H, d]) into the pages of `cache` as vc_cache_append does.
    pos int32 [T]: other positions to turn by than the tokens' places in the cache.  out: where the turned
    queries go (Q itself: in place)."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    strides = _rows("K", K, s.H, s.d, dev)
    if V.shape != K.shape or _rows("V", V, s.H, s.d, dev) != strides:
        raise ValueError("K and V must share shape and strides")
    T = K.shape[0]
    Hq, q_strides, o_strides = 0, (0, 0), (0, 0)
    if Q is not None:
        if Q.dim() != 3 or Q.shape[0] != T:
            raise ValueError("Q must be bf16 [%d, Hq, %d]" % (T, s.d))
        Hq = Q.shape[1]
        q_strides = _rows("Q", Q, Hq, s.d, dev)
    elif out is not None:
        raise ValueError("out without Q")
    batch = _batch_of(cu, kv_len, table, T, dev)
    spec = _rope_spec(rope, dev)
    at = None if pos is None else _int32_vector("pos", pos, T, dev)
    status = _status_ptr(dev_status, dev)
    _check_place(stream, dev)
    if stream is not None and _is_other(stream):
        return _on_stream(stream, vc_cache_append_rope, Q, K, V, cache, cu, kv_len, table, rope, pos, out, dev_status)
    if out is not None:
        o_strides = _rows("out", out, Hq, s.d, dev)
        if out.shape[0] != T:
            raise ValueError("out must have Q's shape")
    elif Q is not None:
        o_strides = (Hq * s.d, s.d)
        out = _new_rows(Q, q_strides == o_strides, dev)
    _on_device(dev, stream, L.vc_cache_append_rope,
               (None if Q is None else Q.data_ptr(), *q_strides, Hq, K.data_ptr(), V.data_ptr(), *strides, s, K8, sk, V8, sv,
                batch, spec, at, None if out is None else out.data_ptr(), *o_strides, status), "vc_cache_append_rope")
    return out


# ------------------------------------------------------------ pages of a cache


def alloc_pool(pages, device):
    """The state of a cache's pages, all free: dict of refs (int32 [pages], table entries that name a page) and free
    (int32 words, a bit for each page that none names).  Tables of the pool begin as -1."""
    bits = torch.full((-(-pages // 32),), -1, dtype=_I32, device=device)
    if pages % 32:
        bits[-1] = (1 << pages % 32) - 1
    return dict(refs=torch.zeros(pages, dtype=_I32, device=device), free=bits)


@functools.lru_cache(maxsize=256)
def _pages_shape(shape):
    """A vc_cache_shape for calls that look at the pages' number and size alone, for K8 of this shape."""
    if len(shape) != 4:
        raise ValueError("K8 and V8 must be uint8 [pages, H, page_size, d]")
    pages, H, page, d = shape
    return VcCacheShape(pages, page, H, d, H * page * d, page * d, d, H * page, page)


def _pages_of(cache):
    """The pages of a cache: what _pages_shape says, the device's index."""
    K8 = cache["K8"]
    return _pages_shape(K8.shape), K8.get_device()


def _pool_of(pool, pages, dev) -> VcPool:
    return VcPool(_int32_vector("refs", pool["refs"], pages, dev), _int32_vector("free", pool["free"], -(-pages // 32), dev))


def _table_of(name, table, dev):
    """Checks an int32 [rows, cols] table: its pointer and what the C calls take beside it (stride, rows, cols)."""
    shape = table.shape
    if table.dtype is not _I32 or len(shape) != 2:
        raise ValueError("%s must be int32 [rows, cols]" % name)
    if table.get_device() != dev:
        raise ValueError("%s is not on the cache's device" % name)
    (rows, cols), (s, one) = shape, table.stride()
    if one != 1 and cols > 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    return table.data_ptr(), s if rows > 1 else max(cols, 1), rows, cols


def pages_reserve_workspace_bytes(cache, B, T) -> int:
    return lib().vc_pages_reserve_workspace(cache_shape_of(cache), B, T)


def pages_compact_workspace_bytes(cache) -> int:
    return lib().vc_pages_compact_workspace(cache_shape_of(cache))


def _given_workspace(workspace, nbytes, dev):
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=_U8, device=dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    return workspace


def _launch_side(stream, call):
    """call(), which returns nothing to the caller but may make a workspace, with `stream` as the current one."""
    with torch.cuda.stream(stream):
        call()


@functools.lru_cache(maxsize=256)
def _reserve_bytes(page_size, B, T):
    """vc_pages_reserve_workspace, which depends on these numbers alone."""
    return max(lib().vc_pages_reserve_workspace(VcCacheShape(1, page_size, 1, 64, page_size * 64, page_size * 64, 64, page_size,
                                                             page_size), B, T), 256)


def vc_pages_reserve(cache, pool, cu, kv_len, table, T, workspace=None, dev_status=None, stream=None):
    """Pages of their own for the tokens of a call (cu, kv_len, table as that call gets them, T rows in all): entries of
    -1 in `table` get the lowest free pages of `pool` (see alloc_pool), pages that others name too are replaced by a
    copy.  With too few free pages nothing is taken and dev_status becomes 6 (VC_ERR_PAGES)."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    batch = _batch_of(cu, kv_len, table, T, dev)
    p = _pool_of(pool, s.pages, dev)
    status = _status_ptr(dev_status, dev)
    _check_place(stream, dev)
    if stream is not None and _is_other(stream):
        return _launch_side(stream, lambda: vc_pages_reserve(cache, pool, cu, kv_len, table, T, workspace, dev_status))
    workspace = _given_workspace(workspace, _reserve_bytes(s.page_size, batch.B, T), dev)
    _on_device(dev, stream, L.vc_pages_reserve, (s, K8, sk, V8, sv, p, batch, workspace.data_ptr(),
                                                 workspace.numel() * workspace.element_size(), status), "vc_pages_reserve")


def vc_pages_fork(cache, pool, table, kv_len, parents, new_table, new_len, lens=None, dev_status=None, stream=None):
    """Rows of new_table (int32 [N, cols]) and new_len (int32 [N]) become sequences that name the pages of the first
    lens[i] tokens (all of them without lens) of sequence parents[i] of `table`; parents[i] = -1: an empty one.
    Nothing is copied before vc_pages_reserve.  What the rows held is not given back: vc_pages_trim does that."""
    L = lib()
    s, dev = _pages_of(cache)
    p = _pool_of(pool, s.pages, dev)
    at, s_table, B, cols = _table_of("table", table, dev)
    to, s_new, N, new_cols = _table_of("new_table", new_table, dev)
    args = (s, p, at, s_table, B, cols, _int32_vector("kv_len", kv_len, B, dev), _int32_vector("parents", parents, N, dev),
            None if lens is None else _int32_vector("lens", lens, N, dev), N, to, s_new, new_cols,
            _int32_vector("new_len", new_len, N, dev), _status_ptr(dev_status, dev))
    _check_place(stream, dev)
    _on_device(dev, stream, L.vc_pages_fork, args, "vc_pages_fork")


def vc_pages_trim(cache, pool, table, kv_len, lens, dev_status=None, stream=None):
    """Each sequence keeps the pages of its first lens[b] tokens (int32 [B]; 0 ends it, a negative one leaves it
    alone): its other entries of `table` become -1, kv_len at most lens."""
    L = lib()
    s, dev = _pages_of(cache)
    p = _pool_of(pool, s.pages, dev)
    at, s_table, B, cols = _table_of("table", table, dev)
    args = (s, p, at, s_table, B, cols, _int32_vector("kv_len", kv_len, B, dev), _int32_vector("lens", lens, B, dev),
            _status_ptr(dev_status, dev))
    _check_place(stream, dev)
    _on_device(dev, stream, L.vc_pages_trim, args, "vc_pages_trim")


def vc_pages_compact(cache, pool, table, used=None, workspace=None, dev_status=None, stream=None):
    """Moves the pages in use to the lowest numbers and renames them in `table`, which has to hold all entries of the
    pool.  Returns how many are in use (int32 [1] on the device): the pages from there on are free."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    p = _pool_of(pool, s.pages, dev)
    at, s_table, B, cols = _table_of("table", table, dev)
    status = _status_ptr(dev_status, dev)
    _check_place(stream, dev)
    if stream is not None and _is_other(stream):
        return _on_stream(stream, vc_pages_compact, cache, pool, table, used, workspace, dev_status)
    if used is None:
        used = torch.empty(1, dtype=_I32, device=dev)
    out = _int32_vector("used", used, 1, dev)
    workspace = _given_workspace(workspace, L.vc_pages_compact_workspace(s), dev)
    _on_device(dev, stream, L.vc_pages_compact,
               (s, K8, sk, V8, sv, p, at, s_table, B, cols, out, workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), status), "vc_pages_compact")
    return used


def vc_cache_copy(source, target, from_pages, to_pages, dev_status=None, stream=None):
    """Copies whole pages: from_pages[i] of `source` to to_pages[i] of `target` (int32 [N]; a -1 leaves the pair out),
    caches of one page size, heads and channels, or one cache."""
    L = lib()
    s, parts, dev = _cache_parts(source)
    t, to_parts, to_dev = _cache_parts(target)
    if to_dev != dev:
        raise ValueError("the caches are on different devices")
    N = from_pages.numel()
    args = (s, *parts, t, *to_parts, _int32_vector("from_pages", from_pages, N, dev), _int32_vector("to_pages", to_pages, N, dev), N,
            _status_ptr(dev_status, dev))
    _check_place(stream, dev)
    _on_device(dev, stream, L.vc_cache_copy, args, "vc_cache_copy")
    return target


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
    _check_place(stream, dev)
    if stream is not None and _is_other(stream):
        return _on_stream(stream, vc_debug_attn_paged_timeout, Q, cache, cu, kv_len, table, dev_status, skip_unit,
                          max_q)
    O = torch.empty((T, Hq, d), dtype=_BF16, device=dev)
    ws = _workspace(L.vc_attn_paged_workspace(s, Hq, batch.B, T, max_q), O.device)
    _on_device(dev, stream, lambda *args: L.vc_debug_attn_paged_timeout(*args, skip_unit),
               (Q.data_ptr(), *strides, Hq, s, K8, sk, V8, sv, batch, max_q, O.data_ptr(), Hq * d, d, ws.data_ptr(),
                ws.numel(), status), "vc_debug_attn_paged_timeout")
    return O


def vc_debug_attn_paged_shared_timeout(Q, cache, cu, kv_len, table, groups, prefix, dev_status, skip_pass, skip_unit, max_q=0,
                                       max_rows=0, workspace=None):
    """vc_attn_paged_shared whose pass `skip_pass` leaves out the keys of each CTA's unit `skip_unit`: as
    vc_debug_attn_paged_timeout.  Returns (O, lse): NaN in the rows of all sequences if a wait ran out."""
    L = lib()
    s, (K8, sk, V8, sv), dev = _cache_parts(cache)
    T, Hq, d = Q.shape
    strides, batch = _rows("Q", Q, Hq, s.d, dev), _batch_of(cu, kv_len, table, T, dev)
    N = prefix.numel()
    runs = _int32_vector("groups", groups, N + 1, dev), _int32_vector("prefix", prefix, N, dev)
    status = _status_ptr(dev_status, dev)
    _need_cuda(dev)
    O, lse = torch.empty((T, Hq, d), dtype=_BF16, device=dev), torch.empty((T, Hq), dtype=_F32, device=dev)
    workspace = _given_workspace(workspace, L.vc_attn_paged_shared_workspace(s, Hq, batch.B, T, N, max_q, max_rows), dev)
    _on_device(dev, None, lambda *args: L.vc_debug_attn_paged_shared_timeout(*args, skip_pass, skip_unit),
               (Q.data_ptr(), *strides, Hq, s, K8, sk, V8, sv, batch, *runs, N, max_q, max_rows, O.data_ptr(), Hq * d, d,
                lse.data_ptr(), workspace.data_ptr(), workspace.numel(), status), "vc_debug_attn_paged_shared_timeout")
    return O, lse

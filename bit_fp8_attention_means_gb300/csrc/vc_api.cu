// vc_api.cu -- the extern "C" entry points declared in include/vc.h.
// Argument checks happen here, on the host, before anything is enqueued.
#include <cstdint>
#include <mutex>
#include <vector>

#include "vc.h"
#include "vc_internal.h"

namespace vc {

vc_status cuda_status(cudaError_t e) { return e == cudaSuccess ? VC_OK : VC_ERR_CUDA; }

vc_status check_shape(const vc_shape& s) {
    if (s.B < 1 || s.H < 1 || s.N < 1 || s.d < 1) return VC_ERR_INVALID_ARG;
    if (s.d != 64 && s.d != 128) return VC_ERR_UNSUPPORTED;
    if (s.N > (1 << 24)) return VC_ERR_UNSUPPORTED;
    if (s.s_b <= 0 || s.s_n <= 0 || s.s_h <= 0) return VC_ERR_INVALID_ARG;
    if ((s.s_b % 8) || (s.s_n % 8) || (s.s_h % 8)) return VC_ERR_INVALID_ARG;
    // TMA row coordinates are 32-bit
    if ((int64_t)s.B * s.H * npad_of(s.N) >= (int64_t(1) << 31)) return VC_ERR_UNSUPPORTED;
    return VC_OK;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

namespace {
using CtxGetCurrentFn = CUresult (*)(CUcontext*);

CtxGetCurrentFn ctx_get_current_fn() {
    static CtxGetCurrentFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<CtxGetCurrentFn>(ptr);
        return static_cast<CtxGetCurrentFn>(nullptr);
    }();
    return fn;
}

CtxAttrCache g_smem_attr;
}  // namespace

vc_status current_ctx(CtxKey* out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return VC_ERR_CUDA;
    CUcontext ctx = nullptr;
    CtxGetCurrentFn fn = ctx_get_current_fn();
    if (fn && fn(&ctx) != CUDA_SUCCESS) ctx = nullptr;
    out->device = dev;
    out->ctx = ctx;
    return VC_OK;
}

vc_status ensure_smem_attr(const void* kern, int bytes) {
    CtxKey key;
    vc_status st = current_ctx(&key);
    if (st != VC_OK) return st;
    return g_smem_attr.ensure(key, kern, bytes, [&](CtxKey* k) -> vc_status {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return cuda_status(e);
        // a context created by this call's own runtime initialisation is known only now
        if (!k->ctx) current_ctx(k);
        return VC_OK;
    });
}

vc_status quantize_args(const void* Q, const void* K, const void* V, const vc_shape& shape, int vsmooth,
                        const float* rope, int hadamard, const uint8_t* Q8, const float* sq, const uint8_t* K8,
                        const float* sk, const uint8_t* V8T, const float* sv, const void* mu) {
    vc_status st = check_shape(shape);
    if (st != VC_OK) return st;
    if ((vsmooth != 0 && vsmooth != 1) || (hadamard != 0 && hadamard != 1)) return VC_ERR_INVALID_ARG;
    if (!Q || !K || !V || !Q8 || !sq || !K8 || !sk || !V8T || !sv || (vsmooth && !mu)) return VC_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(Q8) || !aligned16(K8) || !aligned16(V8T) ||
        !aligned16(rope))
        return VC_ERR_INVALID_ARG;
    return VC_OK;
}

}  // namespace vc

using namespace vc;

extern "C" {

const char* vc_status_string(vc_status s) {
    switch (s) {
        case VC_OK: return "VC_OK";
        case VC_ERR_INVALID_ARG: return "VC_ERR_INVALID_ARG";
        case VC_ERR_UNSUPPORTED: return "VC_ERR_UNSUPPORTED";
        case VC_ERR_WORKSPACE: return "VC_ERR_WORKSPACE";
        case VC_ERR_CUDA: return "VC_ERR_CUDA";
        case VC_ERR_TIMEOUT: return "VC_ERR_TIMEOUT";
        case VC_ERR_PAGES: return "VC_ERR_PAGES";
    }
    return "VC_ERR_UNKNOWN";
}

int vc_version(void) { return 101; }

size_t vc_cluster_workspace(vc_shape shape, int k) {
    if (check_shape(shape) != VC_OK || k < 1) return 0;
    return cluster_workspace(shape, k);
}

vc_status vc_cluster(const void* V, vc_shape shape, int k, int iters, int warm_start, float* centroids,
                     int32_t* labels, int32_t* perm, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                     vc_stream_t stream) {
    return vc_cluster_ex(V, shape, k, iters, warm_start, 0, centroids, labels, perm, workspace, workspace_bytes,
                         dev_status, stream);
}

vc_status vc_cluster_ex(const void* V, vc_shape shape, int k, int iters, int warm_start, int block_fill,
                        float* centroids, int32_t* labels, int32_t* perm, void* workspace, size_t workspace_bytes,
                        int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_shape(shape);
    if (st != VC_OK) return st;
    if (!V || !centroids || !labels || !perm) return VC_ERR_INVALID_ARG;
    if (!aligned16(V) || !aligned16(centroids)) return VC_ERR_INVALID_ARG;
    if (iters < 1 || (warm_start != 0 && warm_start != 1) || (block_fill != 0 && block_fill != 1))
        return VC_ERR_INVALID_ARG;
    if (k < 1 || k > 1024) return VC_ERR_UNSUPPORTED;
    if (k > shape.N) return VC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < cluster_workspace(shape, k) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return VC_ERR_WORKSPACE;
    return launch_cluster(static_cast<const uint16_t*>(V), shape, k, iters, warm_start, block_fill, centroids, labels,
                          perm, workspace, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

size_t vc_quantize_workspace(vc_shape shape) {
    if (check_shape(shape) != VC_OK) return 0;
    return quantize_workspace(shape);
}

static bool workspace_ok(const void* ws, size_t bytes, size_t need) {
    return ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

vc_status vc_quantize(const void* Q, const void* K, const void* V, vc_shape shape, const int32_t* perm, int vsmooth,
                      uint8_t* Q8, float* sq, uint8_t* K8, float* sk, uint8_t* V8T, float* sv, void* mu,
                      void* workspace, size_t workspace_bytes, vc_stream_t stream) {
    return vc_quantize_ex(Q, K, V, shape, perm, vsmooth, nullptr, 0, Q8, sq, K8, sk, V8T, sv, mu, workspace,
                          workspace_bytes, stream);
}

vc_status vc_quantize_ex(const void* Q, const void* K, const void* V, vc_shape shape, const int32_t* perm,
                         int vsmooth, const float* rope, int hadamard, uint8_t* Q8, float* sq, uint8_t* K8,
                         float* sk, uint8_t* V8T, float* sv, void* mu, void* workspace, size_t workspace_bytes,
                         vc_stream_t stream) {
    vc_status st = quantize_args(Q, K, V, shape, vsmooth, rope, hadamard, Q8, sq, K8, sk, V8T, sv, mu);
    if (st != VC_OK) return st;
    if (!workspace_ok(workspace, workspace_bytes, quantize_workspace(shape))) return VC_ERR_WORKSPACE;
    Preproc pp;
    pp.rope = rope;
    pp.hadamard = hadamard;
    return launch_quantize(static_cast<const uint16_t*>(Q), static_cast<const uint16_t*>(K),
                           static_cast<const uint16_t*>(V), shape, perm, vsmooth, pp, Q8, sq, K8, sk, V8T, sv,
                           static_cast<uint16_t*>(mu), workspace, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_quantize_v4(const void* Q, const void* K, const void* V, vc_shape shape, const int32_t* perm,
                         int vsmooth, uint8_t* Q8, float* sq, uint8_t* K8, float* sk, uint8_t* V8T, float* sv,
                         void* mu, void* workspace, size_t workspace_bytes, vc_stream_t stream) {
    vc_status st = quantize_args(Q, K, V, shape, vsmooth, nullptr, 0, Q8, sq, K8, sk, V8T, sv, mu);
    if (st != VC_OK) return st;
    if (!workspace_ok(workspace, workspace_bytes, quantize_workspace(shape))) return VC_ERR_WORKSPACE;
    Preproc pp;
    pp.v4 = 1;
    return launch_quantize(static_cast<const uint16_t*>(Q), static_cast<const uint16_t*>(K),
                           static_cast<const uint16_t*>(V), shape, perm, vsmooth, pp, Q8, sq, K8, sk, V8T, sv,
                           static_cast<uint16_t*>(mu), workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t vc_quantize_staged_workspace(vc_shape shape) {
    if (check_shape(shape) != VC_OK) return 0;
    return quantize_staged_workspace(shape);
}

vc_status vc_quantize_staged(const void* Q, const void* K, const void* V, vc_shape shape, const int32_t* perm,
                             int vsmooth, const float* rope, int hadamard, uint8_t* Q8, float* sq, uint8_t* K8,
                             float* sk, uint8_t* V8T, float* sv, void* mu, void* workspace, size_t workspace_bytes,
                             vc_stream_t stream) {
    vc_status st = quantize_args(Q, K, V, shape, vsmooth, rope, hadamard, Q8, sq, K8, sk, V8T, sv, mu);
    if (st != VC_OK) return st;
    if (!workspace_ok(workspace, workspace_bytes, quantize_staged_workspace(shape))) return VC_ERR_WORKSPACE;
    Preproc pp;
    pp.rope = rope;
    pp.hadamard = hadamard;
    return launch_quantize_staged(static_cast<const uint16_t*>(Q), static_cast<const uint16_t*>(K),
                                  static_cast<const uint16_t*>(V), shape, perm, vsmooth, pp, Q8, sq, K8, sk, V8T,
                                  sv, static_cast<uint16_t*>(mu), workspace, reinterpret_cast<cudaStream_t>(stream));
}

static vc_status attn_common(const uint8_t* Q8, const float* sq, const uint8_t* K8, const float* sk,
                             const uint8_t* V8T, const float* sv, const void* mu, const vc_shape& shape,
                             int expcast, int vsmooth, void* O) {
    vc_status st = check_shape(shape);
    if (st != VC_OK) return st;
    if ((expcast < 0 || expcast > 3) || (vsmooth != 0 && vsmooth != 1)) return VC_ERR_INVALID_ARG;
    if (!Q8 || !sq || !K8 || !sk || !V8T || !sv || !O || (vsmooth && !mu)) return VC_ERR_INVALID_ARG;
    if (!aligned16(Q8) || !aligned16(K8) || !aligned16(V8T) || !aligned16(O)) return VC_ERR_INVALID_ARG;
    return VC_OK;
}

vc_status vc_attn_fwd(const uint8_t* Q8, const float* sq, const uint8_t* K8, const float* sk, const uint8_t* V8T,
                      const float* sv, const void* mu, vc_shape shape, float softmax_scale, int expcast, int vsmooth,
                      void* O, int32_t* dev_status, vc_stream_t stream) {
    if (expcast == 2) return VC_ERR_INVALID_ARG;  // the hybrid has its own entry point
    vc_status st = attn_common(Q8, sq, K8, sk, V8T, sv, mu, shape, expcast, vsmooth, O);
    if (st != VC_OK) return st;
    return launch_attn(Q8, sq, K8, sk, V8T, sv, static_cast<const uint16_t*>(mu), shape, softmax_scale, expcast, 0.f,
                       vsmooth, static_cast<uint16_t*>(O), dev_status, reinterpret_cast<cudaStream_t>(stream),
                       nullptr);
}

vc_status vc_attn_fwd_hybrid(const uint8_t* Q8, const float* sq, const uint8_t* K8, const float* sk,
                             const uint8_t* V8T, const float* sv, const void* mu, vc_shape shape,
                             float softmax_scale, float exact_margin, int vsmooth, void* O, int32_t* dev_status,
                             vc_stream_t stream) {
    if (exact_margin != exact_margin) return VC_ERR_INVALID_ARG;  // NaN
    vc_status st = attn_common(Q8, sq, K8, sk, V8T, sv, mu, shape, 2, vsmooth, O);
    if (st != VC_OK) return st;
    return launch_attn(Q8, sq, K8, sk, V8T, sv, static_cast<const uint16_t*>(mu), shape, softmax_scale, 2,
                       exact_margin, vsmooth, static_cast<uint16_t*>(O), dev_status,
                       reinterpret_cast<cudaStream_t>(stream), nullptr);
}

// ------------------------------------------------------------ paged cache

static bool row_strides_ok(int64_t s_n, int64_t s_h) { return s_n > 0 && s_h > 0 && s_n % 8 == 0 && s_h % 8 == 0; }

static vc_status check_cache_shape(const vc_cache_shape& c) {
    if (c.pages < 1 || c.page_size < 1 || c.H < 1 || c.d < 1) return VC_ERR_INVALID_ARG;
    if (c.s_page <= 0 || c.s_head <= 0 || c.s_tok <= 0 || c.s_page % 16 || c.s_head % 16 || c.s_tok % 16)
        return VC_ERR_INVALID_ARG;
    if (c.s_page >> 40 || c.s_head >> 40 || c.s_tok >> 40) return VC_ERR_INVALID_ARG;  // what a tensor map holds
    if (c.t_page <= 0 || c.t_head <= 0 || c.t_page % 4 || c.t_head % 4) return VC_ERR_INVALID_ARG;
    if (c.d != 64 && c.d != 128) return VC_ERR_UNSUPPORTED;
    if (c.page_size < 16 || c.page_size > 4096 || (c.page_size & (c.page_size - 1))) return VC_ERR_UNSUPPORTED;
    return VC_OK;
}

// Checks what the three cache entry points share and fills the kernels' view.
// Called for T > 0 only: without rows the pointers may be null.
static vc_status cache_view(const vc_cache_shape& c, const uint8_t* K8, const float* sk, const uint8_t* V8,
                            const float* sv, const vc_batch& b, int32_t* dev_status, CacheView* out) {
    if (!K8 || !sk || !V8 || !sv || !b.cu || !b.kv_len || !b.table) return VC_ERR_INVALID_ARG;
    if (!aligned16(K8) || !aligned16(V8) || !aligned16(sk) || !aligned16(sv)) return VC_ERR_INVALID_ARG;
    if (b.s_table < b.cols) return VC_ERR_INVALID_ARG;
    // positions and rows are 32-bit, with room for a unit of keys and a tile of rows past the end
    if ((int64_t)b.cols * c.page_size >= (int64_t(1) << 30) || (int64_t)b.T * c.H >= (int64_t(1) << 31))
        return VC_ERR_UNSUPPORTED;
    out->K8 = const_cast<uint8_t*>(K8);
    out->sk = const_cast<float*>(sk);
    out->V8 = const_cast<uint8_t*>(V8);
    out->sv = const_cast<float*>(sv);
    out->s_page = c.s_page;
    out->s_head = c.s_head;
    out->s_tok = c.s_tok;
    out->t_page = c.t_page;
    out->t_head = c.t_head;
    out->cu = b.cu;
    out->kv_len = b.kv_len;
    out->table = b.table;
    out->s_table = b.s_table;
    out->pages = c.pages;
    out->page_log2 = __builtin_ctz((unsigned)c.page_size);
    out->H = c.H;
    out->B = b.B;
    out->T = b.T;
    out->cols = b.cols;
    out->dev_status = dev_status;
    return VC_OK;
}

static vc_status check_batch_sizes(const vc_batch& b) {
    return (b.B < 1 || b.T < 0 || b.cols < 1) ? VC_ERR_INVALID_ARG : VC_OK;
}

vc_status vc_cache_append(const void* K, const void* V, int64_t s_n, int64_t s_h, vc_cache_shape cache, uint8_t* K8,
                          float* sk, uint8_t* V8, float* sv, vc_batch batch, int32_t* dev_status,
                          vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    if ((st = check_batch_sizes(batch)) != VC_OK) return st;
    if (!row_strides_ok(s_n, s_h)) return VC_ERR_INVALID_ARG;
    if (batch.T == 0) return VC_OK;
    if (!K || !V || !aligned16(K) || !aligned16(V)) return VC_ERR_INVALID_ARG;
    CacheView v;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, &v)) != VC_OK) return st;
    return launch_cache_append(static_cast<const uint16_t*>(K), static_cast<const uint16_t*>(V), s_n, s_h, cache.d, v,
                               reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_cache_read(vc_cache_shape cache, const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv,
                        vc_batch batch, void* K, void* V, int64_t s_n, int64_t s_h, int32_t* dev_status,
                        vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    if ((st = check_batch_sizes(batch)) != VC_OK) return st;
    if (!row_strides_ok(s_n, s_h)) return VC_ERR_INVALID_ARG;
    if (batch.T == 0) return VC_OK;
    if (!K || !V || !aligned16(K) || !aligned16(V)) return VC_ERR_INVALID_ARG;
    CacheView v;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, &v)) != VC_OK) return st;
    return launch_cache_read(v, cache.d, static_cast<uint16_t*>(K), static_cast<uint16_t*>(V), s_n, s_h,
                             reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------ rotary positions

static vc_status check_rope(const vc_rope_spec& r, int d) {
    if (d < 1) return VC_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return VC_ERR_UNSUPPORTED;
    if (r.rot < 16 || r.rot > d || r.rot % 16 || (r.layout != 0 && r.layout != 1)) return VC_ERR_INVALID_ARG;
    if (!(r.magnitude > 0.f) || !__builtin_isfinite(r.magnitude)) return VC_ERR_INVALID_ARG;
    return VC_OK;
}

// Rows (token, head) of d channels of bf16.
struct RowsAt {
    const void* at;
    int64_t s_n, s_h;
    int T, H, d;
};
// Whether a row of `a` and one of `b` (as many tokens) share memory.  Exact where both have the same strides, as
// heads of one tensor do; with others, known only where both begin at the same place or lie apart.
static bool rows_meet(RowsAt a, RowsAt b) {
    if (a.T == 1) a.s_n = b.s_n;  // one token or head: any stride
    if (a.H == 1) a.s_h = b.s_h;
    if (b.H == 1) b.s_h = a.s_h;
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at)) / 2;
    auto size = [](const RowsAt& r) { return (r.T - 1) * r.s_n + (r.H - 1) * r.s_h + r.d; };
    if (off >= size(a) || -off >= size(b)) return false;
    if (a.s_n != b.s_n || a.s_h != b.s_h) return off == 0;
    // some t in -(T-1) .. T-1 and h in -(a.H-1) .. b.H-1 with |off + t s_n + h s_h| < d: the shorter range step by
    // step, of the other one the number nearest to it
    struct Range {
        int64_t lo, hi, step;
    } t{1 - (int64_t)a.T, (int64_t)a.T - 1, a.s_n}, h{1 - (int64_t)a.H, (int64_t)b.H - 1, a.s_h};
    const Range &some = t.hi - t.lo < h.hi - h.lo ? t : h, &other = &some == &t ? h : t;
    for (int64_t i = some.lo; i <= some.hi; ++i) {
        const int64_t at = off + i * some.step, near = -at / other.step;
        for (int64_t n = near - 1; n <= near + 1; ++n) {
            const int64_t k = n < other.lo ? other.lo : n > other.hi ? other.hi : n, x = at + k * other.step;
            if (x < a.d && -x < a.d) return true;
        }
    }
    return false;
}
// Whether rows may be turned into `out`: in place, or apart from what is read.
static bool place_ok(const RowsAt& x, const RowsAt& out) {
    const bool same = x.at == out.at && (x.T == 1 || x.s_n == out.s_n) && (x.H == 1 || x.s_h == out.s_h);
    return same || !rows_meet(x, out);
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static vc_status rope_rows(const vc_rope_spec& r, const int32_t* pos, int inverse, RopeRows* a) {
    if (!r.turns || (reinterpret_cast<uintptr_t>(r.turns) & 7u) || !aligned4(pos)) return VC_ERR_INVALID_ARG;
    *a = RopeRows{};
    a->turns = r.turns;
    a->pos = pos;
    a->rot = r.rot;
    a->pairs = r.layout;
    a->magnitude = r.magnitude;
    a->sign = inverse ? -r.magnitude : r.magnitude;
    return VC_OK;
}

vc_status vc_rope(const void* X, int64_t s_n, int64_t s_h, int T, int H, int d, vc_rope_spec rope, const int32_t* pos,
                  const int32_t* cu, const int32_t* kv_len, int B, int inverse, void* out, int64_t o_sn, int64_t o_sh,
                  int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_rope(rope, d);
    if (st != VC_OK) return st;
    if (T < 0 || H < 1 || (inverse != 0 && inverse != 1)) return VC_ERR_INVALID_ARG;
    if (!row_strides_ok(s_n, s_h) || !row_strides_ok(o_sn, o_sh)) return VC_ERR_INVALID_ARG;
    if ((int64_t)T * H >= (int64_t(1) << 31)) return VC_ERR_UNSUPPORTED;
    if (T == 0) return VC_OK;
    if (!X || !out || !aligned16(X) || !aligned16(out) || (!cu) != (!kv_len) || (!pos && !cu) || (cu && B < 1))
        return VC_ERR_INVALID_ARG;
    if (!place_ok(RowsAt{X, s_n, s_h, T, H, d}, RowsAt{out, o_sn, o_sh, T, H, d})) return VC_ERR_INVALID_ARG;
    RopeRows a;
    if ((st = rope_rows(rope, pos, inverse, &a)) != VC_OK) return st;
    a.Q = static_cast<const uint16_t*>(X);
    a.q_sn = s_n;
    a.q_sh = s_h;
    a.out = static_cast<uint16_t*>(out);
    a.o_sn = o_sn;
    a.o_sh = o_sh;
    a.Hq = H;
    CacheView v{};  // no cache: sequences of up to 2^30 - 1 tokens
    v.cu = cu;
    v.kv_len = kv_len;
    v.cols = (1 << 30) - 1;
    v.B = B;
    v.T = T;
    v.dev_status = dev_status;
    return launch_rope(a, v, d, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_cache_append_rope(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, const void* K, const void* V,
                               int64_t s_n, int64_t s_h, vc_cache_shape cache, uint8_t* K8, float* sk, uint8_t* V8,
                               float* sv, vc_batch batch, vc_rope_spec rope, const int32_t* pos, void* Q_out,
                               int64_t o_sn, int64_t o_sh, int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    if ((st = check_batch_sizes(batch)) != VC_OK) return st;
    if ((st = check_rope(rope, cache.d)) != VC_OK) return st;
    if (Hq < 0 || !row_strides_ok(s_n, s_h)) return VC_ERR_INVALID_ARG;
    if (Hq && (!row_strides_ok(q_sn, q_sh) || !row_strides_ok(o_sn, o_sh))) return VC_ERR_INVALID_ARG;
    if ((int64_t)batch.T * ((int64_t)Hq + 2 * (int64_t)cache.H) >= (int64_t(1) << 31)) return VC_ERR_UNSUPPORTED;
    if (batch.T == 0) return VC_OK;
    if (!K || !V || !aligned16(K) || !aligned16(V)) return VC_ERR_INVALID_ARG;
    if (Hq && (!Q || !Q_out || !aligned16(Q) || !aligned16(Q_out))) return VC_ERR_INVALID_ARG;
    RopeRows a;
    if ((st = rope_rows(rope, pos, 0, &a)) != VC_OK) return st;
    CacheView v;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, &v)) != VC_OK) return st;
    if (Hq) {
        const RowsAt o{Q_out, o_sn, o_sh, batch.T, Hq, cache.d};
        if (!place_ok(RowsAt{Q, q_sn, q_sh, batch.T, Hq, cache.d}, o) || rows_meet(RowsAt{K, s_n, s_h, batch.T, cache.H, cache.d}, o) ||
            rows_meet(RowsAt{V, s_n, s_h, batch.T, cache.H, cache.d}, o))
            return VC_ERR_INVALID_ARG;
    }
    a.Q = static_cast<const uint16_t*>(Q);
    a.K = static_cast<const uint16_t*>(K);
    a.V = static_cast<const uint16_t*>(V);
    a.out = static_cast<uint16_t*>(Q_out);
    a.q_sn = q_sn;
    a.q_sh = q_sh;
    a.k_sn = s_n;
    a.k_sh = s_h;
    a.o_sn = o_sn;
    a.o_sh = o_sh;
    a.Hq = Hq;
    return launch_append_rope(a, v, cache.d, reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------ pages of a cache

static vc_status check_pool(const vc_cache_shape& c, const vc_pool& p, Pool* out) {
    if (!p.refs || !p.free_pages || !aligned4(p.refs) || !aligned4(p.free_pages)) return VC_ERR_INVALID_ARG;
    if (c.pages > (1 << 30)) return VC_ERR_UNSUPPORTED;
    out->refs = p.refs;
    out->free = p.free_pages;
    return VC_OK;
}

// Pieces of a page are counted in 32 bits.
static vc_status check_page_bytes(const vc_cache_shape& c) {
    return (int64_t)c.H * c.page_size * c.d >= (int64_t(1) << 31) ? VC_ERR_UNSUPPORTED : VC_OK;
}

static vc_status check_table(const vc_cache_shape& c, const int32_t* table, int64_t s_table, int rows, int cols) {
    if (!table || !aligned4(table) || rows < 1 || cols < 1 || s_table < cols) return VC_ERR_INVALID_ARG;
    if ((int64_t)cols * c.page_size >= (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
    return VC_OK;
}

// Memory of a call: what its blocks read must not be what other blocks write.
struct Words {
    const int32_t* at;
    int64_t n;
};
static Words table_words(const int32_t* table, int64_t s_table, int rows, int cols) {
    return Words{table, (rows - 1) * s_table + cols};  // from the first to the last row
}
static bool overlap(const Words& a, const Words& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.at && b.at && x < y + (uint64_t)b.n * 4 && y < x + (uint64_t)a.n * 4;
}

size_t vc_pages_reserve_workspace(vc_cache_shape cache, int B, int T) {
    if (check_cache_shape(cache) != VC_OK || B < 1 || T < 1) return 0;
    return pages_reserve_workspace(B, T, __builtin_ctz((unsigned)cache.page_size));
}

vc_status vc_pages_reserve(vc_cache_shape cache, uint8_t* K8, float* sk, uint8_t* V8, float* sv, vc_pool pool,
                           vc_batch batch, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                           vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    if ((st = check_batch_sizes(batch)) != VC_OK) return st;
    Pool p;
    if ((st = check_pool(cache, pool, &p)) != VC_OK || (st = check_page_bytes(cache)) != VC_OK) return st;
    if (batch.T == 0) return VC_OK;
    CacheView v;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, &v)) != VC_OK) return st;
    if (!workspace_ok(workspace, workspace_bytes, pages_reserve_workspace(v.B, v.T, v.page_log2))) return VC_ERR_WORKSPACE;
    const Words rows = table_words(batch.table, batch.s_table, v.B, v.cols);
    if (overlap(rows, Words{v.cu, v.B + 1}) || overlap(rows, Words{v.kv_len, v.B})) return VC_ERR_INVALID_ARG;
    return launch_pages_reserve(v, cache.d, p, workspace, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_pages_fork(vc_cache_shape cache, vc_pool pool, const int32_t* table, int64_t s_table, int B, int cols,
                        const int32_t* kv_len, const int32_t* parents, const int32_t* lens, int N, int32_t* new_table,
                        int64_t s_new, int new_cols, int32_t* new_len, int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    Pool p;
    if ((st = check_pool(cache, pool, &p)) != VC_OK) return st;
    if (N < 0) return VC_ERR_INVALID_ARG;
    if (N == 0) return VC_OK;
    if ((st = check_table(cache, table, s_table, B, cols)) != VC_OK) return st;
    if ((st = check_table(cache, new_table, s_new, N, new_cols)) != VC_OK) return st;
    if (!kv_len || !parents || !new_len || !aligned4(kv_len) || !aligned4(parents) || !aligned4(lens) || !aligned4(new_len))
        return VC_ERR_INVALID_ARG;
    const Words rows = table_words(new_table, s_new, N, new_cols), lengths{new_len, N};
    if (overlap(rows, lengths)) return VC_ERR_INVALID_ARG;
    for (const Words& in : {table_words(table, s_table, B, cols), Words{kv_len, B}, Words{parents, N}})
        if (overlap(in, rows) || overlap(in, lengths)) return VC_ERR_INVALID_ARG;
    // (lens may be new_len: len_i read in its place gives len_i again)
    if (overlap(Words{lens, N}, rows) || (overlap(Words{lens, N}, lengths) && lens != new_len)) return VC_ERR_INVALID_ARG;
    ForkArgs f;
    f.table_in = table;
    f.kv_in = kv_len;
    f.parents = parents;
    f.lens = lens;
    f.table_out = new_table;
    f.kv_out = new_len;
    f.s_in = s_table;
    f.s_out = s_new;
    f.B = B;
    f.cols_in = cols;
    f.cols_out = new_cols;
    f.pages = cache.pages;
    f.page_log2 = __builtin_ctz((unsigned)cache.page_size);
    f.dev_status = dev_status;
    return launch_pages_fork(f, p, N, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_pages_trim(vc_cache_shape cache, vc_pool pool, int32_t* table, int64_t s_table, int B, int cols,
                        int32_t* kv_len, const int32_t* lens, int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    Pool p;
    if ((st = check_pool(cache, pool, &p)) != VC_OK) return st;
    if ((st = check_table(cache, table, s_table, B, cols)) != VC_OK) return st;
    if (!kv_len || !lens || !aligned4(kv_len) || !aligned4(lens)) return VC_ERR_INVALID_ARG;
    const Words rows = table_words(table, s_table, B, cols), lengths{kv_len, B}, keep{lens, B};
    if (overlap(rows, lengths) || overlap(rows, keep) || (overlap(lengths, keep) && lens != kv_len)) return VC_ERR_INVALID_ARG;
    TrimArgs t;
    t.table = table;
    t.kv_len = kv_len;
    t.lens = lens;
    t.s_table = s_table;
    t.cols = cols;
    t.pages = cache.pages;
    t.page_log2 = __builtin_ctz((unsigned)cache.page_size);
    t.dev_status = dev_status;
    return launch_pages_trim(t, p, B, reinterpret_cast<cudaStream_t>(stream));
}

size_t vc_pages_compact_workspace(vc_cache_shape cache) {
    return check_cache_shape(cache) == VC_OK ? pages_compact_workspace(cache.pages) : 0;
}

vc_status vc_pages_compact(vc_cache_shape cache, uint8_t* K8, float* sk, uint8_t* V8, float* sv, vc_pool pool,
                           int32_t* table, int64_t s_table, int B, int cols, int32_t* used, void* workspace,
                           size_t workspace_bytes, int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    Pool p;
    if ((st = check_pool(cache, pool, &p)) != VC_OK || (st = check_page_bytes(cache)) != VC_OK) return st;
    if ((st = check_table(cache, table, s_table, B, cols)) != VC_OK) return st;
    if (!aligned4(used)) return VC_ERR_INVALID_ARG;
    const vc_batch batch{table, table, table, B, 0, cols, s_table};  // no tokens: cu and kv_len are not read
    CacheView v;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, &v)) != VC_OK) return st;
    if (!workspace_ok(workspace, workspace_bytes, pages_compact_workspace(cache.pages))) return VC_ERR_WORKSPACE;
    if (overlap(table_words(table, s_table, B, cols), Words{used, 1})) return VC_ERR_INVALID_ARG;
    return launch_pages_compact(v, cache.d, p, used, workspace, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_cache_copy(vc_cache_shape source, const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv,
                        vc_cache_shape target, uint8_t* K8_to, float* sk_to, uint8_t* V8_to, float* sv_to,
                        const int32_t* from, const int32_t* to, int N, int32_t* dev_status, vc_stream_t stream) {
    vc_status st = check_cache_shape(source);
    if (st != VC_OK || (st = check_cache_shape(target)) != VC_OK) return st;
    if (source.page_size != target.page_size || source.H != target.H || source.d != target.d || N < 0)
        return VC_ERR_INVALID_ARG;
    if ((st = check_page_bytes(source)) != VC_OK) return st;
    if (N == 0) return VC_OK;
    if (!from || !to || !aligned4(from) || !aligned4(to)) return VC_ERR_INVALID_ARG;
    const vc_batch none{from, from, from, 1, 0, 1, 1};  // no batch: not read
    CacheView s, t;
    if ((st = cache_view(source, K8, sk, V8, sv, none, dev_status, &s)) != VC_OK ||
        (st = cache_view(target, K8_to, sk_to, V8_to, sv_to, none, dev_status, &t)) != VC_OK)
        return st;
    return launch_cache_copy(s, t, source.d, from, to, N, reinterpret_cast<cudaStream_t>(stream));
}

static vc_status check_paged_heads(const vc_cache_shape& c, int Hq, int T, int max_q) {
    if (Hq < 1 || Hq % c.H || max_q < 0) return VC_ERR_INVALID_ARG;
    if ((int64_t)T * Hq >= (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
    return VC_OK;
}

size_t vc_attn_paged_workspace(vc_cache_shape cache, int Hq, int B, int T, int max_q) {
    if (check_cache_shape(cache) != VC_OK || B < 1 || T < 1 || check_paged_heads(cache, Hq, T, max_q) != VC_OK)
        return 0;
    return attn_paged_workspace(cache, Hq, B, T, max_q);
}

// Checks what the paged attention's calls share and fills the kernels' arguments; *nothing: no rows.
static vc_status paged_args(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, const vc_cache_shape& cache,
                            const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv,
                            const vc_batch& batch, float softmax_scale, int causal, int window, int max_q, void* O,
                            int64_t o_sn, int64_t o_sh, float* lse, int32_t* dev_status, PagedAttn* a, CacheView* v,
                            bool* nothing) {
    vc_status st = check_cache_shape(cache);
    if (st != VC_OK) return st;
    if ((st = check_batch_sizes(batch)) != VC_OK) return st;
    if ((st = check_paged_heads(cache, Hq, batch.T, max_q)) != VC_OK) return st;
    const double sc = softmax_scale > 0.f ? (double)softmax_scale : 1.0 / __builtin_sqrt((double)cache.d);
    const float scale_log2 = (float)(sc * 1.4426950408889634);
    if ((causal != 0 && causal != 1) || window < 0 || !__builtin_isfinite(softmax_scale) ||
        !__builtin_isfinite(scale_log2))
        return VC_ERR_INVALID_ARG;
    if (!row_strides_ok(q_sn, q_sh) || !row_strides_ok(o_sn, o_sh)) return VC_ERR_INVALID_ARG;
    *nothing = batch.T == 0;
    if (*nothing) return VC_OK;
    if (!Q || !O || !aligned16(Q) || !aligned16(O) || (reinterpret_cast<uintptr_t>(lse) & 3u))
        return VC_ERR_INVALID_ARG;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, v)) != VC_OK) return st;
    a->Q = static_cast<const uint16_t*>(Q);
    a->q_sn = q_sn;
    a->q_sh = q_sh;
    a->O = static_cast<uint16_t*>(O);
    a->o_sn = o_sn;
    a->o_sh = o_sh;
    a->lse = lse;
    a->G = Hq / cache.H;
    a->scale_log2 = scale_log2;
    a->causal = causal;
    a->window = window;
    a->max_q = max_q;
    return VC_OK;
}

static vc_status attn_paged_call(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, vc_cache_shape cache, const uint8_t* K8,
                                 const float* sk, const uint8_t* V8, const float* sv, vc_batch batch, float softmax_scale,
                                 int causal, int window, int max_q, void* O, int64_t o_sn, int64_t o_sh, float* lse,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status, vc_stream_t stream,
                                 int skip_unit) {
    PagedAttn a{};
    CacheView v;
    bool nothing = false;
    const vc_status st = paged_args(Q, q_sn, q_sh, Hq, cache, K8, sk, V8, sv, batch, softmax_scale, causal, window, max_q,
                                    O, o_sn, o_sh, lse, dev_status, &a, &v, &nothing);
    if (st != VC_OK || nothing) return st;
    const size_t need = attn_paged_workspace(cache, Hq, batch.B, batch.T, max_q);
    if (need && !workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_WORKSPACE;
    a.skip_unit = skip_unit;
    return launch_attn_paged(a, v, cache.d, workspace, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_attn_paged(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, vc_cache_shape cache, const uint8_t* K8,
                        const float* sk, const uint8_t* V8, const float* sv, vc_batch batch, float softmax_scale,
                        int causal, int window, int max_q, void* O, int64_t o_sn, int64_t o_sh, float* lse,
                        void* workspace, size_t workspace_bytes, int32_t* dev_status, vc_stream_t stream) {
    return attn_paged_call(Q, q_sn, q_sh, Hq, cache, K8, sk, V8, sv, batch, softmax_scale, causal, window, max_q, O,
                           o_sn, o_sh, lse, workspace, workspace_bytes, dev_status, stream, -1);
}

static vc_status check_groups(int N, int max_rows) { return N < 0 || max_rows < 0 ? VC_ERR_INVALID_ARG : VC_OK; }

size_t vc_attn_paged_shared_workspace(vc_cache_shape cache, int Hq, int B, int T, int N, int max_q, int max_rows) {
    if (check_cache_shape(cache) != VC_OK || B < 1 || T < 1 || check_paged_heads(cache, Hq, T, max_q) != VC_OK ||
        check_groups(N, max_rows) != VC_OK)
        return 0;
    return attn_shared_workspace(cache, Hq, B, T, N, max_q, max_rows);
}

static vc_status attn_shared_call(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, const vc_cache_shape& cache,
                                  const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv,
                                  const vc_batch& batch, const int32_t* groups, const int32_t* prefix, int N,
                                  float softmax_scale, int causal, int max_q, int max_rows, void* O, int64_t o_sn,
                                  int64_t o_sh, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                  vc_stream_t stream, int skip_pass, int skip_unit) {
    SharedAttn a{};
    CacheView v;
    bool nothing = false;
    if (check_groups(N, max_rows) != VC_OK) return VC_ERR_INVALID_ARG;
    vc_status st = paged_args(Q, q_sn, q_sh, Hq, cache, K8, sk, V8, sv, batch, softmax_scale, causal, 0, max_q, O, o_sn,
                              o_sh, lse, dev_status, &a, &v, &nothing);
    if (st != VC_OK || nothing) return st;
    if (N > 0 && (!groups || !prefix || !aligned4(groups) || !aligned4(prefix))) return VC_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, attn_shared_workspace(cache, Hq, v.B, v.T, N, max_q, max_rows)))
        return VC_ERR_WORKSPACE;
    a.groups = groups;
    a.prefix = prefix;
    a.N = N;
    a.skip_unit = skip_unit;
    return launch_attn_shared(a, cache, v, max_rows, skip_pass, workspace, reinterpret_cast<cudaStream_t>(stream));
}

vc_status vc_attn_paged_shared(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, vc_cache_shape cache,
                               const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv, vc_batch batch,
                               const int32_t* groups, const int32_t* prefix, int N, float softmax_scale, int causal,
                               int max_q, int max_rows, void* O, int64_t o_sn, int64_t o_sh, float* lse,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status, vc_stream_t stream) {
    return attn_shared_call(Q, q_sn, q_sh, Hq, cache, K8, sk, V8, sv, batch, groups, prefix, N, softmax_scale, causal,
                            max_q, max_rows, O, o_sn, o_sh, lse, workspace, workspace_bytes, dev_status, stream, 0, -1);
}

vc_status vc_debug_attn_paged_shared_timeout(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, vc_cache_shape cache,
                                             const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv,
                                             vc_batch batch, const int32_t* groups, const int32_t* prefix, int N,
                                             int max_q, int max_rows, void* O, int64_t o_sn, int64_t o_sh, float* lse,
                                             void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                             vc_stream_t stream, int skip_pass, int skip_unit) {
    if (!dev_status || skip_pass < 1 || skip_pass > 2 || skip_unit < 0) return VC_ERR_INVALID_ARG;
    return attn_shared_call(Q, q_sn, q_sh, Hq, cache, K8, sk, V8, sv, batch, groups, prefix, N, 0.f, 1, max_q, max_rows,
                            O, o_sn, o_sh, lse, workspace, workspace_bytes, dev_status, stream, skip_pass, skip_unit);
}

vc_status vc_debug_attn_paged_timeout(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, vc_cache_shape cache,
                                      const uint8_t* K8, const float* sk, const uint8_t* V8, const float* sv,
                                      vc_batch batch, int max_q, void* O, int64_t o_sn, int64_t o_sh, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status, vc_stream_t stream,
                                      int skip_unit) {
    if (!dev_status || skip_unit < 0) return VC_ERR_INVALID_ARG;
    return attn_paged_call(Q, q_sn, q_sh, Hq, cache, K8, sk, V8, sv, batch, 0.f, 1, 0, max_q, O, o_sn, o_sh, nullptr,
                           workspace, workspace_bytes, dev_status, stream, skip_unit);
}

vc_status vc_attn_fwd_debug(const uint8_t* Q8, const float* sq, const uint8_t* K8, const float* sk,
                            const uint8_t* V8T, const float* sv, const void* mu, vc_shape shape, float softmax_scale,
                            int expcast, int vsmooth, void* O, int32_t* dev_status, vc_stream_t stream, int dbg_bh,
                            int dbg_qtile, float* S_dump, uint8_t* P_dump, float exact_margin) {
    if (exact_margin != exact_margin) return VC_ERR_INVALID_ARG;
    vc_status st = attn_common(Q8, sq, K8, sk, V8T, sv, mu, shape, expcast, vsmooth, O);
    if (st != VC_OK) return st;
    if (!S_dump || !P_dump || dbg_bh < 0 || dbg_bh >= shape.B * shape.H || dbg_qtile < 0 ||
        dbg_qtile >= nblk_of(shape.N))
        return VC_ERR_INVALID_ARG;
    AttnDebug dbg;
    dbg.bh = dbg_bh;
    dbg.qtile = dbg_qtile;
    dbg.S = S_dump;
    dbg.P = P_dump;
    return launch_attn(Q8, sq, K8, sk, V8T, sv, static_cast<const uint16_t*>(mu), shape, softmax_scale, expcast,
                       exact_margin, vsmooth, static_cast<uint16_t*>(O), dev_status,
                       reinterpret_cast<cudaStream_t>(stream), &dbg);
}

vc_status vc_debug_attn_timeout(const uint8_t* Q8, const float* sq, const uint8_t* K8, const float* sk,
                                const uint8_t* V8T, const float* sv, const void* mu, vc_shape shape, int vsmooth,
                                void* O, int32_t* dev_status, vc_stream_t stream, int skip_k_tile,
                                uint32_t timeout_us) {
    vc_status st = attn_common(Q8, sq, K8, sk, V8T, sv, mu, shape, 1, vsmooth, O);
    if (st != VC_OK) return st;
    if (!dev_status || skip_k_tile < 0 || skip_k_tile >= nblk_of(shape.N) || timeout_us == 0 ||
        timeout_us > 10000000u)
        return VC_ERR_INVALID_ARG;
    AttnDebug dbg;
    dbg.skip_k_tile = skip_k_tile;
    dbg.timeout_ns = (uint64_t)timeout_us * 1000ull;
    return launch_attn(Q8, sq, K8, sk, V8T, sv, static_cast<const uint16_t*>(mu), shape, 0.f, 1, 0.f, vsmooth,
                       static_cast<uint16_t*>(O), dev_status, reinterpret_cast<cudaStream_t>(stream), &dbg);
}

}  // extern "C"

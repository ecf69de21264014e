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

static vc_status attn_paged_call(const void* Q, int64_t q_sn, int64_t q_sh, int Hq, vc_cache_shape cache, const uint8_t* K8,
                                 const float* sk, const uint8_t* V8, const float* sv, vc_batch batch, float softmax_scale,
                        int causal, int window, int max_q, void* O, int64_t o_sn, int64_t o_sh, float* lse,
                        void* workspace, size_t workspace_bytes, int32_t* dev_status, vc_stream_t stream,
                                 int skip_unit) {
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
    if (batch.T == 0) return VC_OK;
    if (!Q || !O || !aligned16(Q) || !aligned16(O) || (reinterpret_cast<uintptr_t>(lse) & 3u))
        return VC_ERR_INVALID_ARG;
    CacheView v;
    if ((st = cache_view(cache, K8, sk, V8, sv, batch, dev_status, &v)) != VC_OK) return st;
    const size_t need = attn_paged_workspace(cache, Hq, batch.B, batch.T, max_q);
    if (need && !workspace_ok(workspace, workspace_bytes, need)) return VC_ERR_WORKSPACE;
    PagedAttn a;
    a.Q = static_cast<const uint16_t*>(Q);
    a.q_sn = q_sn;
    a.q_sh = q_sh;
    a.O = static_cast<uint16_t*>(O);
    a.o_sn = o_sn;
    a.o_sh = o_sh;
    a.lse = lse;
    a.G = Hq / cache.H;
    a.scale_log2 = scale_log2;
    a.causal = causal;
    a.window = window;
    a.max_q = max_q;
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

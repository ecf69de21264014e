// vc_internal.h -- host-side declarations shared by the library's translation units.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "vc.h"
#include "vc_ctx_cache.h"

namespace vc {

constexpr int kBlock = 128;  // tokens per block (B_v) and per attention tile

inline int nblk_of(int N) { return (N + kBlock - 1) / kBlock; }
inline int64_t npad_of(int N) { return (int64_t)nblk_of(N) * kBlock; }

vc_status check_shape(const vc_shape& s);
vc_status cuda_status(cudaError_t e);

// The CUDA context current on this host thread and its device (CtxKey, in
// vc_ctx_cache.h): the key of every per-context cache below.
vc_status current_ctx(CtxKey* out);

// Raises the dynamic shared-memory limit of kernel `kern` to `bytes` once per
// context (cudaFuncSetAttribute acts on the current context only).  Thread
// safe: host threads may launch on one or several devices concurrently.
vc_status ensure_smem_attr(const void* kern, int bytes);

// Argument checks shared by the quantizer entry points (vc_quantize,
// vc_quantize_ex, vc_quantize_staged, vc_quantize_static).
vc_status quantize_args(const void* Q, const void* K, const void* V, const vc_shape& shape, int vsmooth,
                        const float* rope, int hadamard, const uint8_t* Q8, const float* sq, const uint8_t* K8,
                        const float* sk, const uint8_t* V8T, const float* sv, const void* mu);

// cuTensorMapEncodeTiled, looked up through the runtime so that the library
// does not link against the driver library directly; null if unavailable.
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled_fn();

// quantizer (vc_quantize.cu)
struct Preproc {
    const float* rope = nullptr;  // [N, d/2, 2] (cos, sin), or null: no rotary transform
    int hadamard = 0;             // 1: Walsh-Hadamard transform of Q and K rows, 1/d on the Q scale
    int v4 = 0;                   // 1: the V residual in the 4-bit form (E2M1, power-of-two scale per 32 tokens)
};
size_t quantize_workspace(const vc_shape& s);
size_t quantize_staged_workspace(const vc_shape& s);
vc_status launch_quantize(const uint16_t* Q, const uint16_t* K, const uint16_t* V, const vc_shape& s,
                          const int32_t* perm, int vsmooth, const Preproc& pp, uint8_t* Q8, float* sq, uint8_t* K8,
                          float* sk, uint8_t* V8T, float* sv, uint16_t* mu, void* ws, cudaStream_t st);
vc_status launch_quantize_staged(const uint16_t* Q, const uint16_t* K, const uint16_t* V, const vc_shape& s,
                                 const int32_t* perm, int vsmooth, const Preproc& pp, uint8_t* Q8, float* sq,
                                 uint8_t* K8, float* sk, uint8_t* V8T, float* sv, uint16_t* mu, void* ws,
                                 cudaStream_t st);

// grouping (vc_cluster.cu)
size_t cluster_workspace(const vc_shape& s, int k);
vc_status launch_cluster(const uint16_t* V, const vc_shape& s, int k, int iters, int warm, int fill, float* cent,
                         int32_t* labels, int32_t* perm, void* ws, int32_t* dev_status, cudaStream_t st);

// attention (vc_attn.cu)
struct AttnDebug {
    int bh = -1, qtile = -1;       // the query tile whose scores and bytes are dumped (with S, P)
    float* S = nullptr;
    uint8_t* P = nullptr;
    int skip_k_tile = -1;          // >= 0: the K loader never loads nor signals this key tile
    uint64_t timeout_ns = 0;       // bound of every device wait (0: the default, 4 s)
};
vc_status launch_attn(const uint8_t* Q8, const float* sq, const uint8_t* K8, const float* sk, const uint8_t* V8T,
                      const float* sv, const uint16_t* mu, const vc_shape& s, float softmax_scale, int expcast,
                      float exact_margin, int vsmooth, uint16_t* O, int32_t* dev_status, cudaStream_t st,
                      const AttnDebug* dbg);

// paged cache (vc_cache.cu) and the attention over it (vc_attn_paged.cu)
struct CacheView {                 // what a kernel needs of vc_cache_shape and vc_batch
    uint8_t* K8;
    float* sk;
    uint8_t* V8;
    float* sv;
    int64_t s_page, s_head, s_tok, t_page, t_head;
    const int32_t* cu;
    const int32_t* kv_len;
    const int32_t* table;
    int64_t s_table;
    int pages, page_log2, H, B, T, cols;
    int32_t* dev_status;
};
struct PagedAttn {
    const uint16_t* Q;
    int64_t q_sn, q_sh;
    uint16_t* O;
    int64_t o_sn, o_sh;
    float* lse;
    int G;             // query heads of a key/value head
    float scale_log2;  // softmax_scale * log2 e
    int causal, window, max_q;
    int skip_unit;     // test hook: each CTA's loaders of keys neither load nor signal this unit of theirs; -1 = off
};
struct SharedAttn : PagedAttn {  // attention over shared prefixes
    const int32_t* groups;  // [N + 1] runs of sequences
    const int32_t* prefix;  // [N]
    int run;                // keys of a run in one page: min(page_size, 128)
    // the pass of this launch; of pass 1 and 2 the rows of a tile, an item's own cost in units, the time of a unit in a
    // CTA, the CTAs on an SM
    int N, pass, rt[2], ic[2], unit[2], per_sm[2];
    // workspace: the CTAs' parts of both passes, their results, the rows' words, the planning kernel's sums
    struct PlanPart* plan;
    float *parts1, *parts2;
    uint32_t* words;
    int64_t* sums;
    int32_t* gave_up;  // not 0: a wait of a pass ran out
};
vc_status launch_cache_append(const uint16_t* K, const uint16_t* V, int64_t s_n, int64_t s_h, int d,
                              const CacheView& c, cudaStream_t st);
vc_status launch_cache_read(const CacheView& c, int d, uint16_t* K, uint16_t* V, int64_t s_n, int64_t s_h,
                            cudaStream_t st);
size_t attn_paged_workspace(const vc_cache_shape& c, int Hq, int B, int T, int max_q);
vc_status launch_attn_paged(const PagedAttn& a, const CacheView& c, int d, void* ws, cudaStream_t st);
// over shared prefixes, `a` without what the passes need
size_t attn_shared_workspace(const vc_cache_shape& c, int Hq, int B, int T, int N, int max_q, int max_rows);
// skip_pass: the pass that a.skip_unit (the test hook) is for, refused where the call takes one pass; 0: none
vc_status launch_attn_shared(const SharedAttn& a, const vc_cache_shape& shape, const CacheView& c, int max_rows, int skip_pass,
                             void* ws, cudaStream_t st);
// looks the batch and its groups over; plans the passes; joins their results (vc_attn_shared.cu)
vc_status launch_shared_check(const SharedAttn& a, const CacheView& c, cudaStream_t st);
vc_status launch_shared_plan(const SharedAttn& a, const CacheView& c, cudaStream_t st);
vc_status launch_shared_join(const SharedAttn& a, const CacheView& c, int d, cudaStream_t st);
// its kernel for many rows, in tiles of RT = 128 or 256 (vc_attn_chunk.cu)
vc_status launch_attn_many(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const CacheView& c,
                           int d, int RT, int ctas, void* ws, cudaStream_t st);
vc_status launch_attn_many(const CUtensorMap& mk, const CUtensorMap& mv, const SharedAttn& a, const CacheView& c,
                           int d, int RT, int ctas, cudaStream_t st);

// rotary positions (vc_rope.cu)
struct RopeRows {
    const uint16_t* Q;             // rows to turn (and the queries of an append)
    const uint16_t* K;
    const uint16_t* V;
    uint16_t* out;
    int64_t q_sn, q_sh, k_sn, k_sh, o_sn, o_sh;
    const int64_t* turns;          // [rot / 2] turns a position, as fractions of 2^64
    const int32_t* pos;            // [T], or null: the positions in the cache
    int Hq, rot, pairs;            // rows of a token in Q, turned channels, layout
    int tokens, steps;             // most tokens of a block; rows of a group of its lanes
    float magnitude, sign;         // what cos and sin are multiplied by
};
vc_status launch_rope(const RopeRows& a, const CacheView& c, int d, cudaStream_t st);
vc_status launch_append_rope(const RopeRows& a, const CacheView& c, int d, cudaStream_t st);

// pages of a cache (vc_pages.cu)
struct Pool {
    int32_t* refs;                 // [pages] table entries that name a page
    uint32_t* free;                // a bit for each page that none names
};
struct ForkArgs {
    const int32_t* table_in;
    const int32_t* kv_in;
    const int32_t* parents;
    const int32_t* lens;           // or null: the parents' lengths
    int32_t* table_out;
    int32_t* kv_out;
    int64_t s_in, s_out;
    int B, cols_in, cols_out, pages, page_log2;
    int32_t* dev_status;
};
struct TrimArgs {
    int32_t* table;
    int32_t* kv_len;
    const int32_t* lens;
    int64_t s_table;
    int cols, pages, page_log2;
    int32_t* dev_status;
};
struct ReserveWs {                 // entry w of the call: its page, what becomes of it, the w-th new page;
    int32_t *page, *cls, *fresh;   // sequence b: what is to be copied, its first entry
    int32_t *from, *to, *off;
};
struct CompactWs {
    int32_t *head, *number, *from, *to;  // pages in use and to move; a page's place in the lists; the lists
};
vc_status launch_pages_fork(const ForkArgs& f, const Pool& pool, int N, cudaStream_t st);
vc_status launch_pages_trim(const TrimArgs& t, const Pool& pool, int B, cudaStream_t st);
size_t pages_reserve_workspace(int B, int T, int page_log2);
vc_status launch_pages_reserve(const CacheView& c, int d, const Pool& pool, void* workspace, cudaStream_t st);
vc_status launch_cache_copy(const CacheView& s, const CacheView& t, int d, const int32_t* from, const int32_t* to,
                            int count, cudaStream_t st);
size_t pages_compact_workspace(int pages);
vc_status launch_pages_compact(const CacheView& c, int d, const Pool& pool, int32_t* count, void* workspace,
                               cudaStream_t st);

}  // namespace vc

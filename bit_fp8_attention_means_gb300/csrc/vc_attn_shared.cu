// vc_attn_shared.cu -- the end of attention over shared prefixes (vc_attn_paged_shared): joining
// what the two passes left for each row.
//
// A row has parts k, of the prefix and of its own keys, each with a maximum m_k (log2 units), a sum
// l_k and an accumulator A_k; with m their maximum and w_k = 2^(m_k - m),
//   O = sum_k w_k A_k / sum_k w_k l_k,   lse = ln 2 (m + log2 sum_k w_k l_k).
// A row's word in each pass says in which CTA its item begins and how many have parts of it, so
// that one launch joins everything, in key order.  A warp takes a row: the parts' maxima and sums a
// lane each, then their accumulators, D/32 channels a lane.
#include <cuda_bf16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) shared_join_kernel(const SharedAttn a, const CacheView c, void* ws1, void* ws2) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, Hq = c.H * a.G;
    const int64_t rows = (int64_t)c.T * Hq, row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= rows) {
        wait_for_primary();  // no block ends before the passes have
        return;
    }
    const int tok = (int)(row / Hq), hq = (int)(row - (int64_t)tok * Hq), h = hq / a.G, j = hq - h * a.G;
    const int b = find_seq<32>(c, tok, lane, 0xffffffffu), g = group_of(a, b);
    const SharedPartials part[2] = {shared_partials_at(ws1, a.rt[0], D, rows), shared_partials_at(ws2, a.rt[1], D, rows)};
    // pass 1: the row among its group's; pass 2: among its sequence's
    const SeqPass s = seq_of<true>(c, a, b, 2);
    if (tok < s.q0 || tok >= s.q0 + s.n) {
        wait_for_primary();
        return;
    }
    bool has[2];
    int in[2];  // row of its tile
    const int r2 = (tok - s.q0) * a.G + j;
    has[1] = item_range<true>(a, s, r2 / a.rt[1], a.rt[1], 2).units() > 0;
    in[1] = r2 % a.rt[1];
    has[0] = false;
    in[0] = 0;
    if (g >= 0) {
        const SeqPass p = group_info(c, a, g);
        if (tok >= p.q0 && tok < p.q0 + p.n && p.L > 0) {
            has[0] = true;
            in[0] = (int)((((int64_t)(tok - p.q0)) * a.G + j) % a.rt[0]);
        }
    }
    wait_for_primary();
    int cta[2], n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = has[i] ? __ldcg(part[i].word + row) : 0u;
        cta[i] = min((int)(w >> 8), kMaxCtas - 1);
        n[i] = min((int)(w & 255u), kMaxCtas - cta[i]);
    }
    // place of part k of pass i
    auto place = [&](int i, int k) -> int64_t {
        if (n[i] == 1) return own_slot(a.rt[i], row);
        return (int64_t)(k ? 2 * (cta[i] + k) : 2 * cta[i] + 1) * a.rt[i] + in[i];
    };
    auto place_of = [&](int k) -> int64_t { return k < n[0] ? place(0, k) : place(1, k - n[0]); };
    const int all = n[0] + n[1];
    float m = -INFINITY;
    for (int k = lane; k < all; k += 32) m = fmaxf(m, __ldcg((k < n[0] ? part[0].m : part[1].m) + place_of(k)));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < all; k0 += 32) {
        float w = 0.f, lw = 0.f;
        int64_t at = 0;
        if (k0 + lane < all) {
            const bool own = k0 + lane >= n[0];
            at = place_of(k0 + lane);
            w = part_weight(__ldcg((own ? part[1].m : part[0].m) + at), m);
            lw = w * __ldcg((own ? part[1].l : part[0].l) + at);
        }
        const int some = min(all - k0, 32);
#pragma unroll
        for (int o = 16; o; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
        l += lw;
#pragma unroll 4
        for (int k = 0; k < some; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float* o = (k0 + k < n[0] ? part[0].o : part[1].o) + __shfl_sync(0xffffffffu, at, k) * D + lane * E;
            if constexpr (E == 4) {
                const float4 u = __ldcg(reinterpret_cast<const float4*>(o));
                acc[0] = fmaf(wk, u.x, acc[0]);
                acc[1] = fmaf(wk, u.y, acc[1]);
                acc[2] = fmaf(wk, u.z, acc[2]);
                acc[3] = fmaf(wk, u.w, acc[3]);
            } else {
                const float2 u = __ldcg(reinterpret_cast<const float2*>(o));
                acc[0] = fmaf(wk, u.x, acc[0]);
                acc[1] = fmaf(wk, u.y, acc[1]);
            }
        }
    }
    store_row(a, tok, h, j, lane * E, acc, inverse_sum(l));
    if (lane == 0) store_lse(a, c, tok, h, j, m, l);
}

}  // namespace

vc_status launch_shared_join(const SharedAttn& a, const CacheView& c, int d, void* ws1, void* ws2, cudaStream_t st) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((int64_t)c.T * c.H * a.G + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cuda_status(d == 128 ? cudaLaunchKernelEx(&cfg, shared_join_kernel<128>, a, c, ws1, ws2)
                                : cudaLaunchKernelEx(&cfg, shared_join_kernel<64>, a, c, ws1, ws2));
}

}  // namespace vc

// vc_attn_paged.cu -- attention of a chunk of new tokens over the paged FP8
// cache (vc_attn_paged).
//
// One warp per (row, query head): each lane holds d/32 channels of q and of
// the accumulator, and walks the keys the row sees with the running maximum
// and sum of the softmax.  Reads the whole visible cache once per row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_rows_kernel(const PagedAttn a, const CacheView c) {
    constexpr int E = D / 32;  // channels of a lane
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < c.B; b += kWarps * 32)
            if (!seq_valid(c, b)) flag_invalid(c.dev_status);
    const int lane = threadIdx.x & 31;
    const int Hq = c.H * a.G;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)c.T * Hq) return;
    const int tok = (int)(row / Hq), hq = (int)(row % Hq), h = hq / a.G;
    int b = 0;
    while (b + 1 < c.B && __ldg(c.cu + b + 1) <= tok) ++b;
    const SeqInfo s = seq_info(c, b);
    if (tok < s.q0 || tok >= s.q0 + s.n) return;
    const int last = a.causal ? s.L - s.n + (tok - s.q0) : s.L - 1;
    const int first = a.window ? max(0, last - a.window + 1) : 0;
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_bits_to_f32(a.Q[(int64_t)tok * a.q_sn + (int64_t)hq * a.q_sh + lane * E + e]);
        acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int p = first; p <= last; ++p) {
        const int pg = page_of(c, b, p);
        if (pg < 0) {
            if (lane == 0) flag_invalid(c.dev_status);
            continue;
        }
        const int in = p & ((1 << c.page_log2) - 1);
        const int64_t at = (int64_t)pg * c.s_page + (int64_t)h * c.s_head + (int64_t)in * c.s_tok + lane * E;
        const int64_t st = (int64_t)pg * c.t_page + (int64_t)h * c.t_head + in;
        const float sk = c.sk[st], sv = c.sv[st];
        float dot = 0.f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const __half_raw kr = __nv_cvt_fp8_to_halfraw(c.K8[at + e], __NV_E4M3);
            const __half_raw vr = __nv_cvt_fp8_to_halfraw(c.V8[at + e], __NV_E4M3);
            dot = fmaf(q[e], __half2float(__half(kr)), dot);
            v[e] = __half2float(__half(vr)) * sv;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float x = dot * sk * a.scale_log2;
        const float m_new = fmaxf(m, x);
        const float alpha = exp2f(m - m_new), w = exp2f(x - m_new);
        m = m_new;
        l = fmaf(l, alpha, w);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], alpha, w * v[e]);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.O[(int64_t)tok * a.o_sn + (int64_t)hq * a.o_sh + lane * E + e] =
            __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * inv));
    if (a.lse && lane == 0)
        a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t attn_paged_workspace(const vc_cache_shape&, int, int, int, int) { return 0; }

vc_status launch_attn_paged(const PagedAttn& a, const CacheView& c, int d, void*, cudaStream_t st) {
    const unsigned grid = (unsigned)(((int64_t)c.T * c.H * a.G + kWarps - 1) / kWarps);
    if (d == 128) attn_rows_kernel<128><<<grid, kWarps * 32, 0, st>>>(a, c);
    else attn_rows_kernel<64><<<grid, kWarps * 32, 0, st>>>(a, c);
    return cuda_status(cudaGetLastError());
}

}  // namespace vc

// vc_rope.cu -- rotary positions: rows turned by the angles of their positions
// (vc_rope), and the same on the way into the paged cache (vc_cache_append_rope).
//
// Channels (x0, x1) of pair i of a row at position p become
//   y0 = x0 c - x1 s,  y1 = x0 s + x1 c,   c = m cos(2 pi p w_i),  s = m sin(2 pi p w_i),
// w_i being turns a position.  With w_i as a 64-bit fixed-point fraction the fraction of
// p w_i is the low half of an integer product, exact for every position, so that no table
// of angles is read and none limits how far a context goes; its upper 32 bits go to
// sincospi.  (In fp32 a position of 10^6 would lose 20 of 24 bits of the angle; fp64 would
// be right and slow here.)
//
// Memory bounds both calls: 4d bytes a row, in the cache 2d + d + 4.  A block takes
// consecutive rows, token by token (queries, keys, values), computes the angles of its
// tokens once for all their heads while the rows' loads are under way, and then turns, a
// group of d/8 lanes a row.  What is written to the cache is quantized straight from fp32,
// as in vc_cache.cu otherwise.
#include <cuda_bf16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;  // rows of a group of lanes

struct Place {
    int64_t code, scale;  // of head 0; scale < 0: not in the cache
    int pos;
    int found;            // the row belongs to a sequence
};

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <int D, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeRows a, const CacheView c) {
    constexpr int W = D / 8, GROUPS = kThreads / W, U = kRows, HALF = D / 2, TOKENS = GROUPS * U;
    __shared__ float2 turn[TOKENS * HALF];
    __shared__ Place place[TOKENS];
    const int tid = threadIdx.x, lane = tid & 31, sub = lane & (W - 1), group = tid / W;
    const unsigned mask = ((W == 16) ? 0xFFFFu : 0xFFu) << (lane & ~(W - 1));
    if (blockIdx.x == 0 && c.cu)
        for (int b = tid; b < c.B; b += kThreads)
            if (!seq_valid(c, b)) flag_invalid(c.dev_status);

    // this group's rows: token and number among the token's rows (queries, keys, values)
    const uint32_t per = APPEND ? a.Hq + 2 * c.H : a.Hq, rows = (uint32_t)c.T * per, first = blockIdx.x * (uint32_t)TOKENS;
    const int tok0 = (int)(first / per), tokens = (int)((min(first + TOKENS, rows) - 1) / per) - tok0 + 1;
    uint4 x[U];
    int tk[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t row = first + group * U + u;
        const int tok = (int)(row / per);
        tk[u] = row < rows ? tok - tok0 : -1;
        r[u] = (int)(row - (uint32_t)tok * per);
        if (tk[u] < 0) continue;
        const uint16_t* src;
        if (!APPEND || r[u] < a.Hq) src = a.Q + (int64_t)tok * a.q_sn + (int64_t)r[u] * a.q_sh;
        else if (r[u] < a.Hq + c.H) src = a.K + (int64_t)tok * a.k_sn + (int64_t)(r[u] - a.Hq) * a.k_sh;
        else src = a.V + (int64_t)tok * a.k_sn + (int64_t)(r[u] - a.Hq - c.H) * a.k_sh;
        x[u] = __ldcs(reinterpret_cast<const uint4*>(src) + sub);
    }
    // where the tokens are
    const int pair = tid & (HALF - 1);
    const uint64_t w = pair < a.rot / 2 ? (uint64_t)__ldg(a.turns + pair) : 0;
    for (int i = group; i < tokens; i += GROUPS) {
        const int tok = tok0 + i;
        Place p{0, -1, 0, 1};
        if (c.cu) {
            const int b = find_seq<W>(c, tok, sub, mask);
            const SeqInfo s = seq_info(c, b);
            p.found = tok >= s.q0 && tok < s.q0 + s.n;
            p.pos = s.L - s.n + (tok - s.q0);
            if (APPEND && p.found) {
                const int pg = p.pos >= 0 ? page_of(c, b, p.pos) : -1;
                if (pg >= 0) {
                    const int in = p.pos & ((1 << c.page_log2) - 1);
                    p.code = (int64_t)pg * c.s_page + (int64_t)in * c.s_tok;
                    p.scale = (int64_t)pg * c.t_page + in;
                } else if (sub == 0) {
                    flag_invalid(c.dev_status);
                }
            }
        }
        if (a.pos) p.pos = __ldg(a.pos + tok);
        if (sub == 0) place[i] = p;
    }
    __syncthreads();
    if (pair < a.rot / 2)
        for (int i = tid / HALF; i < tokens; i += kThreads / HALF) {
            const uint64_t t = w * (uint64_t)(int64_t)place[i].pos;
            float sn, cs;
            sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &sn, &cs);
            turn[i * HALF + pair] = make_float2(cs * a.magnitude, sn * a.sign);
        }
    __syncthreads();

    const int half = a.rot / 2, c0 = sub * 8;
    // halves: the lane that holds the other channels of this one's pairs
    const int apart = half / 8, other = a.pairs || c0 >= a.rot ? lane : c0 < half ? lane + apart : lane - apart;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool there = tk[u] >= 0 && place[max(tk[u], 0)].found;
        if (!__any_sync(0xffffffffu, there)) continue;
        const uint4 v = there ? x[u] : make_uint4(0, 0, 0, 0);
        const uint4 o = make_uint4(__shfl_sync(0xffffffffu, v.x, other), __shfl_sync(0xffffffffu, v.y, other),
                                   __shfl_sync(0xffffffffu, v.z, other), __shfl_sync(0xffffffffu, v.w, other));
        float y[8];
        unpack(v, y);
        const bool value = APPEND && r[u] >= a.Hq + c.H;
        const float2* t = turn + max(tk[u], 0) * HALF;
        if (there && c0 < a.rot && !value) {
            if (a.pairs) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = t[c0 / 2 + i];
                    const float y0 = y[2 * i], y1 = y[2 * i + 1];
                    y[2 * i] = y0 * e.x - y1 * e.y;
                    y[2 * i + 1] = y0 * e.y + y1 * e.x;
                }
            } else {
                float z[8];
                unpack(o, z);
                const bool second = c0 >= half;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 e = t[second ? c0 - half + i : c0 + i];
                    y[i] = second ? z[i] * e.y + y[i] * e.x : y[i] * e.x - z[i] * e.y;
                }
            }
        }
        if (!APPEND || r[u] < a.Hq) {
            if (there) {
                uint32_t q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                    q[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                uint16_t* dst = a.out + (int64_t)(tok0 + tk[u]) * a.o_sn + (int64_t)r[u] * a.o_sh;
                reinterpret_cast<uint4*>(dst)[sub] = make_uint4(q[0], q[1], q[2], q[3]);
            }
        } else if (there && place[tk[u]].scale >= 0) {
            float scale;
            const uint2 codes = quantize_row8<W>(y, mask, &scale);
            const int h = value ? r[u] - a.Hq - c.H : r[u] - a.Hq;
            const int64_t at = place[tk[u]].code + (int64_t)h * c.s_head;
            *reinterpret_cast<uint2*>((value ? c.V8 : c.K8) + at + sub * 8) = codes;
            if (sub == 0) (value ? c.sv : c.sk)[place[tk[u]].scale + (int64_t)h * c.t_head] = scale;
        }
    }
}

template <bool APPEND>
vc_status launch(const RopeRows& a, const CacheView& c, int d, cudaStream_t st) {
    const int per_block = kThreads / (d / 8) * kRows;
    const uint32_t rows = (uint32_t)c.T * (uint32_t)(APPEND ? a.Hq + 2 * c.H : a.Hq);
    const unsigned grid = (rows + per_block - 1) / per_block;
    if (d == 128) rope_kernel<128, APPEND><<<grid, kThreads, 0, st>>>(a, c);
    else rope_kernel<64, APPEND><<<grid, kThreads, 0, st>>>(a, c);
    return cuda_status(cudaGetLastError());
}

}  // namespace

vc_status launch_rope(const RopeRows& a, const CacheView& c, int d, cudaStream_t st) {
    return launch<false>(a, c, d, st);
}

vc_status launch_append_rope(const RopeRows& a, const CacheView& c, int d, cudaStream_t st) {
    return launch<true>(a, c, d, st);
}

}  // namespace vc

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
// Memory bounds both calls: 4d bytes a row, in the cache 2d + d + 4; and instructions, of which a row
// has as many as its bytes take time.  So a block takes consecutive rows, token by token (queries,
// keys, values), and computes the angles of its tokens once for all their heads; a group of
// d/16 lanes a row keeps them in registers from row to row; a lane holds both channels of its pairs, in
// either layout, so that nothing is exchanged; and the loads of the next two rows are under way while one
// is computed.  What is written to the cache is quantized straight from fp32, as in vc_cache.cu otherwise.
// Measured: 20,011 rows of 40 heads turned 68 us, 6.0 TB/s; 14,315 tokens of 40 + 8 heads turned and cached
// 74 us, 5.2 TB/s.
#include <cuda_bf16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

// Threads of a block, and rows of a group of its lanes at most.  Measured with 128 and 256 threads: 800,000 rows of
// one head turned 144 and 170 us, 20,011 rows of 40 heads 68 and 70 us; 14,000 rows of 56 (8 of them keys, 8 values)
// turned and appended 79 and 76 us.
constexpr int threads_of(bool append) { return append ? 256 : 128; }
constexpr int steps_of(bool append) { return append ? 8 : 16; }

struct Place {
    int64_t code, scale;  // of head 0; scale < 0: not in the cache
    int pos;
    int found;            // the row belongs to a sequence
};

// Eight bf16, two at a time.
__device__ __forceinline__ void unpack(const uint4& v, float2* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16_bits_to_f32(w[i] & 0xFFFFu), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack(const float2* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[i].x, x[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude; NaN where one is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// Sixteen fp32 values of a row that W lanes share -> as many codes and the row's scale, by the steps of
// vc_cache_append.
template <int W>
__device__ __forceinline__ void quantize(const float2 (&x)[8], unsigned mask, float* scale, uint2 (&codes)[2]) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_abs(amax, max_abs(x[i].x, x[i].y));
#pragma unroll
    for (int o = W / 2; o; o >>= 1) amax = max_abs(amax, __shfl_xor_sync(mask, amax, o));
    if (!(amax < INFINITY) || amax < 0x1p-100f) {
        *scale = amax < 1.f ? 0.f : __int_as_float(0x7FFFFFFF);
        codes[0] = codes[1] = make_uint2(0u, 0u);
        return;
    }
    *scale = __fdiv_rn(amax, 448.f);
    const float inv = __fdiv_rn(448.f, amax);
    const float2 inv2 = make_float2(inv, inv);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __fmul2_rn(x[2 * i], inv2), z = __fmul2_rn(x[2 * i + 1], inv2);
        q[i] = cvt_e4m3x2(y.x, y.y) | (cvt_e4m3x2(z.x, z.y) << 16);
    }
    codes[0] = make_uint2(q[0], q[1]);
    codes[1] = make_uint2(q[2], q[3]);
}

// PAIRS: the layout of neighbouring channels.  A lane's sixteen channels are two pieces of eight: of those that
// turn, channels 8 l .. of the first half and as many of the second in halves, neighbours otherwise.
template <int D, bool APPEND, bool PAIRS>
__global__ void __launch_bounds__(threads_of(APPEND)) rope_kernel(const RopeRows a, const CacheView c) {
    constexpr int kThreads = threads_of(APPEND);
    constexpr int W = D / 16, GROUPS = kThreads / W, HALF = D / 2;
    extern __shared__ float4 smem[];
    float4* turn = smem;                                                   // [tokens][4][HALF / 8]: two pairs' c, c, s, s
    Place* place = reinterpret_cast<Place*>(turn + a.tokens * (HALF / 2));  // [tokens]
    const int tid = threadIdx.x, lane = tid & 31, sub = lane & (W - 1), group = tid / W;
    const unsigned mask = ((1u << W) - 1u) << (lane & ~(W - 1));
    if (blockIdx.x == 0 && c.cu)
        for (int b = tid; b < c.B; b += kThreads)
            if (!seq_valid(c, b)) flag_invalid(c.dev_status);

    // rows first + group, + GROUPS and so on: token and number among the token's rows (queries, keys, values)
    const uint32_t per = APPEND ? a.Hq + 2 * c.H : a.Hq, rows = (uint32_t)c.T * per, block_rows = (uint32_t)(GROUPS * a.steps);
    const uint32_t first = blockIdx.x * block_rows, end = min(first + block_rows, rows);
    const int tok0 = (int)(first / per), tokens = (int)((end - 1) / per) - tok0 + 1;
    const int step_tok = (int)((uint32_t)GROUPS / per), step_r = (int)((uint32_t)GROUPS % per);
    const bool turns = sub * 16 < a.rot;
    const int p0 = PAIRS || !turns ? sub * 16 : sub * 8, p1 = PAIRS || !turns ? sub * 16 + 8 : a.rot / 2 + sub * 8;
    int tok = (int)((first + group) / per), r = (int)(first + group - (uint32_t)tok * per);
    auto advance = [&](int& t, int& n) {
        t += step_tok;
        n += step_r;
        if (n >= (int)per) {
            n -= (int)per;
            ++t;
        }
    };
    struct Row {
        uint4 lo, hi;
    };
    auto load = [&](int t, int n) -> Row {
        const uint16_t* src;
        if (!APPEND || n < a.Hq) src = a.Q + (int64_t)t * a.q_sn + (int64_t)n * a.q_sh;
        else if (n < a.Hq + c.H) src = a.K + (int64_t)t * a.k_sn + (int64_t)(n - a.Hq) * a.k_sh;
        else src = a.V + (int64_t)t * a.k_sn + (int64_t)(n - a.Hq - c.H) * a.k_sh;
        return Row{__ldcs(reinterpret_cast<const uint4*>(src + p0)), __ldcs(reinterpret_cast<const uint4*>(src + p1))};
    };
    uint32_t ahead = first + group;  // the next row to load
    int t_ahead = tok, r_ahead = r;
    auto next = [&]() -> Row {
        Row x{};
        if (ahead < end) x = load(t_ahead, r_ahead);
        ahead += GROUPS;
        advance(t_ahead, r_ahead);
        return x;
    };
    Row x0 = next(), x1 = next();

    // where the tokens are
    const int pair = tid & (HALF - 1);
    const uint64_t w = pair < a.rot / 2 ? (uint64_t)__ldg(a.turns + pair) : 0;
    for (int i = tid >> 5; i < tokens; i += kThreads / 32) {
        const int t = tok0 + i;
        Place p{0, -1, 0, 1};
        if (c.cu) {
            const int b = find_seq<32>(c, t, lane, 0xffffffffu);
            const SeqInfo s = seq_info(c, b);
            p.found = t >= s.q0 && t < s.q0 + s.n;
            p.pos = s.L - s.n + (t - s.q0);
            if (APPEND && p.found) {
                const int pg = p.pos >= 0 ? page_of(c, b, p.pos) : -1;
                if (pg >= 0) {
                    const int in = p.pos & ((1 << c.page_log2) - 1);
                    p.code = (int64_t)pg * c.s_page + (int64_t)in * c.s_tok;
                    p.scale = (int64_t)pg * c.t_page + in;
                } else if (lane == 0) {
                    flag_invalid(c.dev_status);
                }
            }
        }
        if (a.pos) p.pos = __ldg(a.pos + t);
        if (lane == 0) place[i] = p;
    }
    __syncthreads();
    if (pair < a.rot / 2)
        for (int i = tid / HALF; i < tokens; i += kThreads / HALF) {
            const uint64_t t = w * (uint64_t)(int64_t)place[i].pos;
            float sn, cs;
            sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &sn, &cs);
            // the j-th two pairs of each lane's eight side by side: no bank conflicts where a lane reads its own
            float* at = reinterpret_cast<float*>(turn + i * (HALF / 2) + (pair & 7) / 2 * (HALF / 8) + pair / 8) + (pair & 1);
            at[0] = cs * a.magnitude;
            at[2] = sn * a.sign;
        }
    __syncthreads();

    float4 e[4];      // this lane's angles
    int angles = -1;  // of this token
    auto turn_row = [&](const Row& v) {
        const int tk = tok - tok0, n = r;
        advance(tok, r);
        if (!place[tk].found) return;
        const bool value = APPEND && n >= a.Hq + c.H;
        float2 x[8];
        unpack(v.lo, x);
        unpack(v.hi, x + 4);
        if (turns && !value) {
            if (tk != angles) {
                angles = tk;
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] = turn[tk * (HALF / 2) + j * (HALF / 8) + sub];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (PAIRS) {
                    const float2 u = x[2 * j], w = x[2 * j + 1];
                    x[2 * j] = make_float2(u.x * e[j].x - u.y * e[j].z, u.x * e[j].z + u.y * e[j].x);
                    x[2 * j + 1] = make_float2(w.x * e[j].y - w.y * e[j].w, w.x * e[j].w + w.y * e[j].y);
                } else {
                    const float2 u = x[j], w = x[4 + j];
                    x[j] = make_float2(u.x * e[j].x - w.x * e[j].z, u.y * e[j].y - w.y * e[j].w);
                    x[4 + j] = __ffma2_rn(w, make_float2(e[j].x, e[j].y), __fmul2_rn(u, make_float2(e[j].z, e[j].w)));
                }
            }
        }
        if (!APPEND || n < a.Hq) {
            uint16_t* dst = a.out + (int64_t)(tok0 + tk) * a.o_sn + (int64_t)n * a.o_sh;
            *reinterpret_cast<uint4*>(dst + p0) = pack(x);
            *reinterpret_cast<uint4*>(dst + p1) = pack(x + 4);
        } else if (place[tk].scale >= 0) {
            float scale;
            uint2 codes[2];
            quantize<W>(x, mask, &scale, codes);
            const int h = value ? n - a.Hq - c.H : n - a.Hq;
            uint8_t* dst = (value ? c.V8 : c.K8) + place[tk].code + (int64_t)h * c.s_head;
            *reinterpret_cast<uint2*>(dst + p0) = codes[0];
            *reinterpret_cast<uint2*>(dst + p1) = codes[1];
            if (sub == 0) (value ? c.sv : c.sk)[place[tk].scale + (int64_t)h * c.t_head] = scale;
        }
    };
    // two rows in turn, so that nothing moves between registers
    for (uint32_t row = first + group; row < end; row += 2 * GROUPS) {
        turn_row(x0);
        x0 = next();
        if (row + GROUPS >= end) break;
        turn_row(x1);
        x1 = next();
    }
}

template <int D, bool APPEND, bool PAIRS>
vc_status launch_layout(RopeRows a, const CacheView& c, cudaStream_t st) {
    constexpr int THREADS = threads_of(APPEND), GROUPS = THREADS / (D / 16), MOST = steps_of(APPEND);
    constexpr int TOKEN = D / 2 * (int)sizeof(float2) + (int)sizeof(Place);
    const uint32_t per = APPEND ? a.Hq + 2 * c.H : a.Hq, rows = (uint32_t)c.T * per;
    // rows of a group: as many as leave 1,024 threads an SM
    const uint32_t some = rows / (GROUPS * kMaxCtas * (1024 / THREADS));
    a.steps = some < 1 ? 1 : some > MOST ? MOST : (int)some;
    if (per < 4 && a.steps > MOST / 4) a.steps = MOST / 4;  // many tokens a block: their angles fill the shared memory
    const uint32_t block_rows = GROUPS * a.steps;
    a.tokens = (int)(per == 1 ? block_rows : (block_rows + per - 2) / per + 1);  // that so many rows can belong to
    static_assert(GROUPS * MOST / 4 * TOKEN <= 48 * 1024 && (GROUPS * MOST / 4 + 1) * TOKEN <= 48 * 1024, "without asking for more");
    rope_kernel<D, APPEND, PAIRS><<<(rows + block_rows - 1) / block_rows, THREADS, a.tokens * TOKEN, st>>>(a, c);
    return cuda_status(cudaGetLastError());
}

template <bool APPEND>
vc_status launch(const RopeRows& a, const CacheView& c, int d, cudaStream_t st) {
    if (d == 128) return a.pairs ? launch_layout<128, APPEND, true>(a, c, st) : launch_layout<128, APPEND, false>(a, c, st);
    return a.pairs ? launch_layout<64, APPEND, true>(a, c, st) : launch_layout<64, APPEND, false>(a, c, st);
}

}  // namespace

vc_status launch_rope(const RopeRows& a, const CacheView& c, int d, cudaStream_t st) {
    return launch<false>(a, c, d, st);
}

vc_status launch_append_rope(const RopeRows& a, const CacheView& c, int d, cudaStream_t st) {
    return launch<true>(a, c, d, st);
}

}  // namespace vc

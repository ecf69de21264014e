// vc_cache.cu -- the paged FP8 key/value cache: quantizing new tokens as they
// are written (vc_cache_append) and reading tokens back (vc_cache_read).
//
// Per (token, head) and for K and V alike:
//   write: amax = max_c |x_c|, scale = amax / 448, code_c = E4M3(x_c * (448 / amax))
//   read:  x_c = bf16(code_c * scale)
// Both move 4d bytes of bf16 and 2d + 8 bytes of cache per (token, head) with
// a handful of operations per channel, so memory bounds them: a group of d/8
// lanes owns a row, each lane 8 channels (one 16-byte access of bf16 and one
// 8-byte access of codes), the maximum goes around the group by shuffles, and
// a row is touched once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kThreads = 256;

struct RowArgs {
    const uint16_t* K;  // append: source rows; read: written through Kout, Vout
    const uint16_t* V;
    uint16_t* Kout;
    uint16_t* Vout;
    int64_t s_n, s_h;
};

// The sequence of row `tok`: the last b with cu[b] <= tok.  W lanes (a group
// with mask `mask`) probe W places a round, so B <= W^2 takes two rounds.
template <int W>
__device__ __forceinline__ int find_seq(const CacheView& c, int tok, int sub, unsigned mask) {
    int lo = 0, hi = c.B;  // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + W - 1) / W;
        const int at = lo + sub * step;
        const bool le = at < hi && __ldg(c.cu + at) <= tok;
        const unsigned votes = (__ballot_sync(mask, le) & mask) >> (__ffs(mask) - 1);
        const int k = max(31 - __clz((int)(votes | 1u)), 0);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Where row (tok, h) of the call lies: the element offsets of its codes and
// its scale.  False where the row belongs to no sequence (*found = false too),
// has a negative position or a page that is not there.
template <int W>
__device__ __forceinline__ bool locate(const CacheView& c, int tok, int h, int sub, unsigned mask, int64_t* code_off,
                                       int64_t* scale_off, bool* found) {
    const int b = find_seq<W>(c, tok, sub, mask);
    const SeqInfo s = seq_info(c, b);
    *found = tok >= s.q0 && tok < s.q0 + s.n;
    if (!*found) return false;
    const int p = s.L - s.n + (tok - s.q0);
    const int pg = p >= 0 ? page_of(c, b, p) : -1;
    if (pg < 0) {
        if (sub == 0) flag_invalid(c.dev_status);
        return false;
    }
    const int in = p & ((1 << c.page_log2) - 1);
    *code_off = (int64_t)pg * c.s_page + (int64_t)h * c.s_head + (int64_t)in * c.s_tok;
    *scale_off = (int64_t)pg * c.t_page + (int64_t)h * c.t_head + in;
    return true;
}

// Eight bf16 of a row -> eight codes; the row's scale.  amax comes from the
// bit patterns with the sign off, which order like the magnitudes and put
// infinities and NaN above every number.
template <int W>
__device__ __forceinline__ uint2 quantize_row(const uint4& x, unsigned mask, float* scale) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = W / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
    const float amax = bf16_bits_to_f32(top);
    if (top >= 0x7F80u || amax < 0x1p-100f) {
        *scale = top >= 0x7F80u ? __int_as_float(0x7FFFFFFF) : 0.f;
        return make_uint2(0u, 0u);
    }
    *scale = __fdiv_rn(amax, 448.f);
    const float inv = __fdiv_rn(448.f, amax);
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a0 = __fmul_rn(bf16_bits_to_f32(w[2 * i] & 0xFFFFu), inv);
        const float a1 = __fmul_rn(__uint_as_float(w[2 * i] & 0xFFFF0000u), inv);
        const float a2 = __fmul_rn(bf16_bits_to_f32(w[2 * i + 1] & 0xFFFFu), inv);
        const float a3 = __fmul_rn(__uint_as_float(w[2 * i + 1] & 0xFFFF0000u), inv);
        o[i] = cvt_e4m3x2(a0, a1) | (cvt_e4m3x2(a2, a3) << 16);
    }
    return make_uint2(o[0], o[1]);
}

// Eight codes * scale -> eight bf16.
__device__ __forceinline__ uint4 dequantize_row(const uint2& codes, float scale) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = ((i & 2) ? codes.y : codes.x) >> (16 * (i & 1));
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)pair));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        const __nv_bfloat162 r = __floats2bfloat162_rn(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
        o[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The first block also looks the batch over: cu and kv_len of every sequence.
__device__ __forceinline__ void check_batch(const CacheView& c) {
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < c.B; b += kThreads)
            if (!seq_valid(c, b)) flag_invalid(c.dev_status);
}

// A group of lanes takes kRows consecutive rows (heads of one token, as a rule),
// whose loads are on their way while the place of the token is looked up, once.
// Measured, for 3,600 tokens of 40 heads written (112 MB) and 75,600 read back
// (2.35 GB): one row 26.0 and 391 us, two 23.3 us (4.8 TB/s) and 342 us (6.9 TB/s),
// four 25.1 and 347 us, eight 32.1 and 389 us; one token each of 96 sequences of 8
// heads takes 3.5 us with one or two.
constexpr int kRows = 2;

template <int D, bool READ>
__global__ void __launch_bounds__(kThreads) cache_rows_kernel(const RowArgs a, const CacheView c) {
    constexpr int W = D / 8, U = kRows;  // lanes of a row, rows of a group
    check_batch(c);
    const int lane = threadIdx.x & 31, sub = lane & (W - 1);
    const unsigned mask = ((W == 16) ? 0xFFFFu : 0xFFu) << (lane & ~(W - 1));
    const int64_t rows = (int64_t)c.T * c.H, row0 = ((int64_t)blockIdx.x * (kThreads / W) + threadIdx.x / W) * U;
    if (row0 >= rows) return;
    int tok = (int)(row0 / c.H), h = (int)(row0 - (int64_t)tok * c.H);
    // rows of the group: token and head, and where their bf16 lie
    int toks[U], hs[U];
    int64_t x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        toks[u] = tok;
        hs[u] = h;
        x[u] = (int64_t)tok * a.s_n + (int64_t)h * a.s_h + sub * 8;
        if (++h == c.H) {
            h = 0;
            ++tok;
        }
    }
    uint4 kx[U], vx[U];
    if (!READ) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row0 + u >= rows) break;
            kx[u] = __ldcs(reinterpret_cast<const uint4*>(a.K + x[u]));
            vx[u] = __ldcs(reinterpret_cast<const uint4*>(a.V + x[u]));
        }
    }
    int64_t at[U], st[U];
    bool found[U], there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        found[u] = there[u] = false;
        if (row0 + u >= rows) continue;
        if (u == 0 || toks[u] != toks[u - 1]) {
            there[u] = locate<W>(c, toks[u], hs[u], sub, mask, &at[u], &st[u], &found[u]);
        } else {
            found[u] = found[u - 1];
            there[u] = there[u - 1];
            at[u] = at[u - 1] + c.s_head;
            st[u] = st[u - 1] + c.t_head;
        }
    }
    if (!READ) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!there[u]) continue;
            float ks, vs;
            const uint2 kc = quantize_row<W>(kx[u], mask, &ks), vc = quantize_row<W>(vx[u], mask, &vs);
            *reinterpret_cast<uint2*>(c.K8 + at[u] + sub * 8) = kc;
            *reinterpret_cast<uint2*>(c.V8 + at[u] + sub * 8) = vc;
            if (sub == 0) {
                c.sk[st[u]] = ks;
                c.sv[st[u]] = vs;
            }
        }
    } else {
        uint2 kc[U], vc[U];
        float ks[U], vs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!there[u]) continue;
            kc[u] = __ldcs(reinterpret_cast<const uint2*>(c.K8 + at[u] + sub * 8));
            vc[u] = __ldcs(reinterpret_cast<const uint2*>(c.V8 + at[u] + sub * 8));
            ks[u] = __ldg(c.sk + st[u]);
            vs[u] = __ldg(c.sv + st[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!found[u]) continue;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            __stcs(reinterpret_cast<uint4*>(a.Kout + x[u]), there[u] ? dequantize_row(kc[u], ks[u]) : zero);
            __stcs(reinterpret_cast<uint4*>(a.Vout + x[u]), there[u] ? dequantize_row(vc[u], vs[u]) : zero);
        }
    }
}

template <bool READ>
vc_status launch_rows(const RowArgs& a, const CacheView& c, int d, cudaStream_t st) {
    const int rows_per_block = kThreads / (d / 8) * kRows;
    const unsigned grid = (unsigned)(((int64_t)c.T * c.H + rows_per_block - 1) / rows_per_block);
    if (d == 128) cache_rows_kernel<128, READ><<<grid, kThreads, 0, st>>>(a, c);
    else cache_rows_kernel<64, READ><<<grid, kThreads, 0, st>>>(a, c);
    return cuda_status(cudaGetLastError());
}

}  // namespace

vc_status launch_cache_append(const uint16_t* K, const uint16_t* V, int64_t s_n, int64_t s_h, int d,
                              const CacheView& c, cudaStream_t st) {
    RowArgs a{K, V, nullptr, nullptr, s_n, s_h};
    return launch_rows<false>(a, c, d, st);
}

vc_status launch_cache_read(const CacheView& c, int d, uint16_t* K, uint16_t* V, int64_t s_n, int64_t s_h,
                            cudaStream_t st) {
    RowArgs a{nullptr, nullptr, K, V, s_n, s_h};
    return launch_rows<true>(a, c, d, st);
}

}  // namespace vc

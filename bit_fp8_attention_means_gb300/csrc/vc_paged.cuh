// vc_paged.cuh -- device-side view of a batch over the paged cache: which rows
// and positions a sequence has, where a position lies, and how the attention
// kernels share the work.  Everything read from cu, kv_len and table is clamped
// or checked here, so that no value in them leads outside the caller's buffers.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>

#include "vc_device.cuh"
#include "vc_internal.h"

namespace vc {

struct SeqInfo {
    int q0, n;  // first row of the call and number of rows
    int L;      // tokens in the cache
};

__device__ __forceinline__ void flag_invalid(int32_t* dev_status) {
    if (dev_status) atomicMax(reinterpret_cast<int*>(dev_status), (int)VC_ERR_INVALID_ARG);
}

__device__ __forceinline__ SeqInfo seq_info(const CacheView& c, int b) {
    SeqInfo s;
    const int a = __ldg(c.cu + b), e = __ldg(c.cu + b + 1), len = __ldg(c.kv_len + b);
    s.q0 = min(max(a, 0), c.T);
    s.n = min(max(e, s.q0), c.T) - s.q0;
    s.L = min(max(len, 0), c.cols << c.page_log2);
    return s;
}

// Whether cu[b], cu[b+1] and kv_len[b] keep the batch's rules.
__device__ __forceinline__ bool seq_valid(const CacheView& c, int b) {
    const int a = __ldg(c.cu + b), e = __ldg(c.cu + b + 1), len = __ldg(c.kv_len + b);
    return a >= 0 && e >= a && e <= c.T && len >= 0 && len <= (c.cols << c.page_log2);
}

// Page of position p (0 <= p < cols * page_size), or -1 where it is not there.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int p) {
    const int pg = __ldg(c.table + (int64_t)b * c.s_table + (p >> c.page_log2));
    return (pg >= 0 && pg < c.pages) ? pg : -1;
}

// ------------------------------------------------------------ work of the attention kernels
//
// The rows of a sequence for one key/value head are its n * G (token, query
// head) pairs, token by token; an item is a tile of RT of them, and its work is
// the units of 128 keys that at least one of its rows sees.  All items of a
// call stand in one order (sequence, head, tile), each as long as its units and
// what beginning and ending an item costs, IC units more; CTA i of C takes
// the i-th of C equal parts of this line, so lengths that differ, few rows and
// long caches keep all SMs equally busy.  (Without the items' own cost, CTAs with
// many short items took three times as long as those with one long one.)  An
// item cut by the border of two CTAs leaves partial results (running maximum,
// sum, accumulator) in the workspace, which a second kernel joins in key order.

constexpr int kUnit = 128;       // keys of a unit
constexpr int kMaxCtas = 152;    // one CTA on each SM

struct ItemRange {
    int lo, hi;     // first and last key that some row sees (hi < lo: none)
    int lo_all, hi_all;  // first and last key that every row sees
    __device__ int first() const { return lo / kUnit; }
    __device__ int units() const { return hi < lo ? 0 : hi / kUnit - lo / kUnit + 1; }
};

__device__ __forceinline__ int row_last(const PagedAttn& a, const SeqInfo& s, int token) {
    return a.causal ? s.L - s.n + token : s.L - 1;
}
__device__ __forceinline__ int row_first(const PagedAttn& a, int last) {
    return a.window && last >= a.window ? last - a.window + 1 : 0;  // no overflow for any window
}

__device__ __forceinline__ ItemRange item_range(const PagedAttn& a, const SeqInfo& s, int tile, int RT) {
    const int r0 = tile * RT, r1 = min(r0 + RT, s.n * a.G) - 1;
    const int h0 = row_last(a, s, r0 / a.G), h1 = row_last(a, s, r1 / a.G);
    ItemRange r;
    r.lo = row_first(a, h0);
    r.hi = h1;
    r.lo_all = row_first(a, h1);
    r.hi_all = h0;
    return r;
}

// Tiles of a sequence: of 0 rows none; n * G < 2^31.
__device__ __forceinline__ int seq_tiles(const PagedAttn& a, const SeqInfo& s, int RT) {
    return (int)(((int64_t)s.n * a.G + RT - 1) / RT);
}

__device__ __forceinline__ int item_cost(const PagedAttn& a, const SeqInfo& s, int tile, int RT, int IC) {
    const int u = item_range(a, s, tile, RT).units();
    return u ? u + IC : 0;
}

// Cost of one head's tiles of a sequence: by one thread, or by a warp.
__device__ __forceinline__ int64_t seq_cost(const CacheView& c, const PagedAttn& a, int b, int RT, int IC) {
    const SeqInfo s = seq_info(c, b);
    const int nt = seq_tiles(a, s, RT);
    int64_t u = 0;
    for (int t = 0; t < nt; ++t) u += item_cost(a, s, t, RT, IC);
    return u;
}
__device__ __forceinline__ int64_t seq_cost_warp(const PagedAttn& a, const SeqInfo& s, int RT, int IC) {
    const int nt = seq_tiles(a, s, RT);
    int64_t u = 0;
    for (int t = threadIdx.x & 31; t < nt; t += 32) u += item_cost(a, s, t, RT, IC);
    for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
}

// a / b of numbers that are small as a rule: a 64-bit division is a long subroutine,
// and a CTA's first microsecond.
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The part of a CTA: [g0, g1) of the line, and where g0 lies.
struct Part {
    int64_t g0, g1;
    int b;        // sequence of g0
    int64_t off;  // g0's place in its sequence (all heads)
    int64_t total;  // length of the line, and number of parts
    int parts;
};

// Called by all NT threads of a block; the result is the same in all of them.
// Two passes over the sequences, NT at a time: the total, then the one that
// holds g0.  Sequences of many tiles are added up by a warp each.
template <int NT>
__device__ __forceinline__ Part plan_part(const CacheView& c, const PagedAttn& a, int RT, int IC, int part, int parts) {
    __shared__ int64_t warp_sum[NT / 32];
    __shared__ int64_t cost[NT];
    __shared__ Part found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool by_warp = (int64_t)c.T * a.G > (int64_t)c.B * RT * 4;
    // cost of sequence b0 + threadIdx.x
    auto costs = [&](int b0) -> int64_t {
        if (by_warp) {
            for (int i = warp; i < NT && b0 + i < c.B; i += NT / 32) {
                const int64_t u = seq_cost_warp(a, seq_info(c, b0 + i), RT, IC);
                if (lane == 0) cost[i] = u * c.H;
            }
            __syncthreads();
            return b0 + (int)threadIdx.x < c.B ? cost[threadIdx.x] : 0;
        }
        return b0 + (int)threadIdx.x < c.B ? seq_cost(c, a, b0 + threadIdx.x, RT, IC) * c.H : 0;
    };
    if (threadIdx.x == 0) found = Part{};
    const int64_t first_u = costs(0);
    int64_t mine = first_u;
    for (int b0 = NT; b0 < c.B; b0 += NT) {
        __syncthreads();
        mine += costs(b0);
    }
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) warp_sum[warp] = mine;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < NT / 32; ++w) total += warp_sum[w];
    Part p;
    if (total < parts) parts = (int)total;  // no empty part between two others
    p.b = 0;
    p.off = 0;
    p.total = total;
    p.parts = parts;
    if (part >= parts) {
        p.g0 = p.g1 = 0;
        return p;
    }
    p.g0 = div_small(total * part, parts);
    p.g1 = div_small(total * (part + 1), parts);
    int64_t before = 0;  // cost of the sequences of earlier rounds
    for (int b0 = 0; b0 < c.B; b0 += NT) {
        __syncthreads();
        const int64_t u = b0 ? costs(b0) : first_u;
        int64_t scan = u;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int64_t base = before, all = before;
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) base += warp_sum[w];
            all += warp_sum[w];
        }
        const int64_t end = base + scan, begin = end - u;
        if (begin <= p.g0 && p.g0 < end) {
            found.b = b0 + threadIdx.x;
            found.off = p.g0 - begin;
        }
        before = all;
        if (all > p.g0) break;  // the same in all threads
    }
    __syncthreads();
    p.b = found.b;
    p.off = found.off;
    return p;
}

// Walks the items of a CTA's part that have units in it, in order.  For whole
// warps; all members are uniform over the warp.
template <int IC>
struct ItemWalk {
    int64_t at, left;  // place in the line, and what is left of the part
    int b, h, tile;  // the item
    SeqInfo s;
    ItemRange r;
    int unit, end;   // units [unit, end) of 128 keys, of this item in this part
    int64_t item_end;  // the item's end in the line
    bool head;       // an earlier CTA has the item's first units
    bool tail;       // a later CTA has its last units

    // Parts from this one on that have units of the item.
    __device__ int parts_on(const Part& p, int part) const {
        return tail ? (int)div_small(item_end * p.parts - 1, p.total) - part + 1 : 1;
    }
    // To the first item; false where the part holds no unit at all.
    __device__ bool start(const CacheView& c, const PagedAttn& a, int RT, const Part& p) {
        at = p.g0;
        left = p.g1 - p.g0;
        b = p.b;
        s = seq_info(c, b);
        const int64_t per_head = seq_cost_warp(a, s, RT, IC);
        h = (int)div_small(p.off, per_head);
        int64_t off = p.off - h * per_head;
        const int nt = seq_tiles(a, s, RT), lane = threadIdx.x & 31;
        for (int t0 = 0;; t0 += 32) {
            int64_t scan = t0 + lane < nt ? item_cost(a, s, t0 + lane, RT, IC) : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
                if (lane >= o) scan += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, scan > off);
            if (past || t0 + 32 >= nt) {
                const int k = past ? __ffs(past) - 1 : 0;
                const int64_t before = __shfl_sync(0xffffffffu, scan, k ? k - 1 : 0);
                tile = t0 + k;
                if (k) off -= before;
                break;
            }
            off -= __shfl_sync(0xffffffffu, scan, 31);
        }
        r = item_range(a, s, tile, RT);
        return take((int)off) || next(c, a, RT);
    }
    // The item from place `off` of its length on; false where that holds none of its units.
    __device__ bool take(int off) {
        const int u = r.units(), all = u + IC;
        const int to = left < all - off ? off + (int)left : all;
        item_end = at + all - off;
        at += to - off;
        left -= to - off;
        const int u0 = max(off - IC, 0), u1 = to - IC;
        head = u0 > 0;
        tail = u1 < u;
        unit = r.first() + u0;
        end = r.first() + u1;
        return u1 > u0;
    }
    // To the next item with units in the part; false at its end.
    __device__ bool next(const CacheView& c, const PagedAttn& a, int RT) {
        while (left > 0) {
            if (++tile >= seq_tiles(a, s, RT)) {
                tile = 0;
                if (++h >= c.H) {
                    h = 0;
                    if (++b >= c.B) return false;
                    s = seq_info(c, b);
                }
                if (seq_tiles(a, s, RT) == 0) {  // a sequence without rows has no heads to walk
                    h = c.H;
                    continue;
                }
            }
            r = item_range(a, s, tile, RT);
            if (r.units() && take(0)) return true;
        }
        return false;
    }
};

// What a CTA leaves in the workspace for an item that it shares: a header and,
// for its rows, the running maximum (log2 units), the sum, the accumulator.
struct PartHeader {
    int parts;       // from this one on that have units of the item; 0: nothing here
    int q0, h, r0, rows;  // first row of the sequence, head, first (token, head) pair and number of pairs
};

// Slot 2i: the item whose first units an earlier CTA has; slot 2i + 1: the
// item that begins in CTA i's part and goes on in the next one.
struct Partials {
    PartHeader* head;  // [2 * kMaxCtas]
    float* m;          // [2 * kMaxCtas][RT]
    float* l;
    float* o;          // [2 * kMaxCtas][RT][D]
};

inline __host__ __device__ size_t partials_bytes(int RT, int D) {
    return 2 * (size_t)kMaxCtas * (32 + (size_t)RT * (D + 2) * sizeof(float));
}
static_assert(sizeof(PartHeader) <= 32, "header slots");

inline __host__ __device__ Partials partials_at(void* ws, int RT, int D) {
    Partials p;
    p.o = static_cast<float*>(ws);
    p.m = p.o + 2 * (size_t)kMaxCtas * RT * D;
    p.l = p.m + 2 * (size_t)kMaxCtas * RT;
    p.head = reinterpret_cast<PartHeader*>(p.l + 2 * (size_t)kMaxCtas * RT);
    return p;
}

// 1 / l for a row's sum: 0 for a row that saw nothing, NaN kept.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : __frcp_rn(l); }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}
// Weight of a part with maximum m_part in a whole with maximum m.
__device__ __forceinline__ float part_weight(float m_part, float m) {
    return m_part == -INFINITY ? 0.f : ex2_approx(m_part - m);
}

// ------------------------------------------------------------ shared by the attention kernels

constexpr float kStale = 8.f;          // how far the maximum may rise before M follows

// What a producer tells the other warps of a CTA about a unit.
struct StageInfo {
    int flags;  // bits below
    int key0;   // position of the stage's first key
    int q0, n, L, h, r0, rows;
    int box_ok;  // bit i: the stage's i-th run of min(128, page_size) keys has its page
    int pad[7];
};
static_assert(sizeof(StageInfo) == 64, "one line");
enum : int { kFirst = 1, kLast = 2, kMasked = 4, kEnd = 8, kHead = 16, kTail = 32, kHoles = 64 };

// Four E4M3 codes -> four fp16.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Power of two that brings a row whose largest magnitude has the bf16 bits
// `top` into [128, 256); 1 for rows of zeros and for rows that are not finite.
__device__ __forceinline__ float row_factor(uint32_t top) {
    if (top == 0u || top >= 0x7F80u) return 1.f;
    const int e = max((int)(top >> 7), 14) - 127;
    return __int_as_float((134 - e) << 23);
}

// Channels ch .. ch + N - 1 (N = 2 or 4) of row r (a (token, head) pair of its sequence), acc * inv as bf16.
template <int N>
__device__ __forceinline__ void store_row(const PagedAttn& a, int q0, int h, int r, int ch, const float (&acc)[N],
                                          float inv) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&v);
    }
    const int tok = r / a.G;
    uint16_t* dst = a.O + (int64_t)(q0 + tok) * a.o_sn + (int64_t)(h * a.G + r - tok * a.G) * a.o_sh + ch;
    if constexpr (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

__device__ __forceinline__ void store_lse(const PagedAttn& a, const CacheView& c, int q0, int h, int r, float m,
                                          float l) {
    if (a.lse) a.lse[(int64_t)(q0 + r / a.G) * (c.H * a.G) + h * a.G + r % a.G] = lse_of(m, l);
}

}  // namespace vc

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
// the units of 128 keys that at least one of its rows sees.  All units of a
// call stand in one order (sequence, head, tile, key) and CTA i of C takes the
// i-th of C equal parts (with fewer units than CTAs, one unit each), so lengths
// that differ, few rows and long caches keep all SMs equally busy.  An item cut by the border of two CTAs leaves partial
// results (running maximum, sum, accumulator) in the workspace, which a second
// kernel joins in key order.

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
    return a.window ? max(0, last - a.window + 1) : 0;
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

__device__ __forceinline__ int64_t seq_units(const CacheView& c, const PagedAttn& a, int b, int RT) {
    const SeqInfo s = seq_info(c, b);
    const int nt = seq_tiles(a, s, RT);
    int64_t u = 0;
    for (int t = 0; t < nt; ++t) u += item_range(a, s, t, RT).units();
    return u;
}

// The part of a CTA: global units [g0, g1), and where g0 lies.
struct Part {
    int64_t g0, g1;
    int b;        // sequence of unit g0
    int64_t off;  // unit g0's place in its sequence (all heads)
};

// Called by all NT threads of a block; the result is the same in all of them.
// Two passes over the sequences: the total, then the one that holds g0.
template <int NT>
__device__ __forceinline__ Part plan_part(const CacheView& c, const PagedAttn& a, int RT, int part, int parts) {
    __shared__ int64_t warp_sum[NT / 32 + 1];
    __shared__ Part found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t mine = 0, first_u = 0;
    for (int b = threadIdx.x; b < c.B; b += NT) {
        const int64_t u = seq_units(c, a, b, RT) * c.H;
        if (b == (int)threadIdx.x) first_u = u;
        mine += u;
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
    if (part >= parts) {
        p.g0 = p.g1 = 0;
        return p;
    }
    p.g0 = total * part / parts;
    p.g1 = total * (part + 1) / parts;
    int64_t before = 0;  // units of the sequences of earlier rounds
    for (int b0 = 0; b0 < c.B; b0 += NT) {
        const int b = b0 + threadIdx.x;
        const int64_t u = b >= c.B ? 0 : b0 ? seq_units(c, a, b, RT) * c.H : first_u;
        int64_t scan = u;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int64_t base = before, all = before;
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) base += warp_sum[w];
            all += warp_sum[w];
        }
        const int64_t end = base + scan, begin = end - u;
        if (begin <= p.g0 && p.g0 < end) {
            found.b = b;
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

// Walks the items of a CTA's part, in order.  All members are uniform over the
// threads that walk together.
struct ItemWalk {
    int64_t left;    // units still to take
    int b, h, tile;  // the item
    SeqInfo s;
    ItemRange r;
    int unit, end;   // units [unit, end) of 128 keys, of this item in this part
    bool head;       // an earlier CTA has the item's first units
    bool tail;       // a later CTA has its last units

    __device__ void start(const CacheView& c, const PagedAttn& a, int RT, const Part& p) {
        left = p.g1 - p.g0;
        b = p.b;
        s = seq_info(c, b);
        const int nt = seq_tiles(a, s, RT);
        int64_t per_head = 0;
        for (int t = 0; t < nt; ++t) per_head += item_range(a, s, t, RT).units();
        h = (int)(p.off / per_head);
        int64_t off = p.off % per_head;
        tile = 0;
        while (true) {
            r = item_range(a, s, tile, RT);
            if (off < r.units()) break;
            off -= r.units();
            ++tile;
        }
        head = off > 0;
        set((int)off);
    }
    __device__ void set(int off) {
        unit = r.first() + off;
        const int u = r.units() - off;
        tail = u > left;
        end = unit + (tail ? (int)left : u);
        left -= end - unit;
    }
    // To the next item; false at the part's end.
    __device__ bool next(const CacheView& c, const PagedAttn& a, int RT) {
        if (left == 0) return false;
        head = false;
        do {
            if (++tile >= seq_tiles(a, s, RT)) {
                tile = 0;
                if (++h == c.H) {
                    h = 0;
                    if (++b >= c.B) return false;
                    s = seq_info(c, b);
                }
                if (seq_tiles(a, s, RT) == 0) {  // a sequence without rows has no heads to walk
                    h = c.H - 1;
                    r.lo = 0;
                    r.hi = -1;
                    continue;
                }
            }
            r = item_range(a, s, tile, RT);
        } while (r.units() == 0);
        set(0);
        return true;
    }
};

// What a CTA leaves in the workspace for an item that it shares: a header and,
// for its rows, the running maximum (log2 units), the sum, the accumulator.
struct PartHeader {
    int valid;       // 0: nothing here
    int last;        // the item's last units are in this part
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
constexpr float kZeroLog2 = -60.f;     // log2 sv of a token whose values are all zero
constexpr uint64_t kTimeoutNs = 4000000000ull;  // bound of every wait

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

// Channels ch .. ch + 3 of row r (a (token, head) pair of its sequence), acc * inv as bf16.
__device__ __forceinline__ void store_row(const PagedAttn& a, int q0, int h, int r, int ch, const float (&acc)[4],
                                          float inv) {
    const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
    const __nv_bfloat162 v1 = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(a.O + (int64_t)(q0 + r / a.G) * a.o_sn + (int64_t)(h * a.G + r % a.G) * a.o_sh + ch) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
}

__device__ __forceinline__ void store_lse(const PagedAttn& a, const CacheView& c, int q0, int h, int r, float m,
                                          float l) {
    if (a.lse) a.lse[(int64_t)(q0 + r / a.G) * (c.H * a.G) + h * a.G + r % a.G] = lse_of(m, l);
}

}  // namespace vc

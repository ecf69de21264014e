// vc_attn_paged.cu -- attention of a chunk of new tokens over the paged FP8
// cache (vc_attn_paged): the kernel for few rows, the kernel that joins partial
// results, and the choice among kernels.
//
// Row (token, query head) sees keys t with scores s_t = scale q . k_t; with the
// cached codes k8, v8 and the tokens' scales sk, sv,
//   y_t = (q . k8_t) sk_t scale log2 e,   x_t = y_t + log2 sv_t,
//   A = sum_t 2^(x_t - M) v8_t,   l = sum_t 2^(y_t - N),
//   O = 2^(M - N) A / l,   lse = ln 2 (N + log2 l),
// M and N being the running maxima of x and of y.  Folding sv into the exponent lets
// P = 2^(x - M) enter the product with the value codes as fp16 whatever the scales are;
// E4M3 codes are fp16 numbers exactly.  (A single exponential, with l the sum of P / sv,
// would lose the weight of small values beside large ones and leave fp32's range for many
// small ones.)  M and N move only when their maximum has risen by more than 8 (P then stays
// below 2^8, far inside fp16), which saves most of the rescaling of A.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

// ------------------------------------------------------------ few rows
//
// attn_few_kernel: tiles of 8 RG rows.  What bounds it is reading the cache
// once (2d + 8 bytes per key and head), so everything else is arranged around a
// full memory pipe: one persistent CTA on each SM, four producer warps (two for
// keys, two for values) that keep NS stages of 128 keys in flight, and sixteen
// consumer warps that share nothing until an item ends.  A consumer warp owns 8
// rows and blocks of 16 keys, with its own M, l and A in registers.  Keys and
// channels are the wide side of the products (K q^T, V^T P^T as m16n8k16 fp16),
// so 8 rows fill them; a tcgen05 tile of 128 rows would be mostly padding here.
// Codes become fp16 on the way from shared memory to registers; the channels of
// q . k and the keys and channels of P V are permuted so that each thread reads
// 16 consecutive bytes, in an order without bank conflicts under the TMA
// swizzle.  One token of 96 sequences of 100 to 8,192 keys (747 MB, pages of 16):
// 153 us, 4.9 TB/s; rows as the wide side, 8 warps and one producer took 251 us.
// One token against 75,600 keys (160 MB): 40 us, of which 25 us at 6.4 TB/s lie
// between the first data (6 us) and the joining (6 us).

// What an item costs besides its units, in units: the queries, and adding up the warps' parts.
constexpr int kItemCost = 3;
constexpr int kConsumers = 16;
constexpr int kFewThreads = (kConsumers + 4) * 32;
// 640 threads start with 96 registers each; 4 x 128 x 104 + 128 x 56 = 60,416 fit into those 61,440
constexpr int kFewRegsUp = 104, kFewRegsDown = 56;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int D>
struct FewCfg {
    static constexpr int NS = D == 128 ? 4 : 8;
    static constexpr int TILE = kUnit * D;                       // codes of K or V in a stage
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + NS * TILE;
    static constexpr int OFF_SCR = OFF_V + NS * TILE;            // [warp][8][D] accumulators at an item's end
    static constexpr int OFF_SC = OFF_SCR + kConsumers * 8 * D * 4;  // [stage][sk | sv][128]
    static constexpr int OFF_ML = OFF_SC + NS * 2 * kUnit * 4;   // [m | l][warp][8]
    static constexpr int OFF_INFO = OFF_ML + 2 * kConsumers * 8 * 4;
    static constexpr int OFF_BAR = OFF_INFO + NS * 64;           // full[NS], empty[NS], written, read
    static constexpr int OFF_MISC = OFF_BAR + (2 * NS + 2) * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    // Key (of 8) that row n of a score tile stands for, so that the eight
    // lanes of a 16-byte shared-memory phase fall on different banks.
    __device__ static int key_of(int n) {
        if (D == 128) return (n >> 1) + 4 * (n & 1);
        const int i = n >> 1;
        return (n & 1) ? 2 * i + 1 - (i & 1) : 2 * i + (i & 1);
    }
    // Byte offset of 16-byte chunk ch of key row r under the TMA swizzle.
    __device__ static int chunk(int r, int ch) {
        return D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
    }
    // First of the D/8 consecutive channels that rows n and n + 8 of the output tiles stand for.
    __device__ static int channel_of(int n) { return D == 128 ? ((n >> 1) + 4 * (n & 1)) * 16 : n * 8; }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// SKIP: the test hook that leaves out the keys of unit a.skip_unit, in instances of its own.
template <int D, int RG, bool SKIP>
__global__ void __launch_bounds__(kFewThreads, 1)
    attn_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedAttn a, const CacheView c, void* ws) {
    using C = FewCfg<D>;
    constexpr int NS = C::NS, RT = 8 * RG;
    constexpr uint32_t ATTEMPTS = SKIP ? kHookAttempts : kWaitAttempts;
    // offsets from the array itself: through an integer the compiler would lose sight of
    // the address space, and generic loads take the slow road to shared memory
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full = sbase + C::OFF_BAR, empty = full + 8 * NS, written = empty + 8 * NS, read = written + 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const Partials part = partials_at(ws, RT, D);

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full + 8 * s, 4 + 64);  // the producers, and each lane of the two that load scales
            mbar_init(empty + 8 * s, kConsumers);
        }
        mbar_init(written, kConsumers);
        mbar_init(read, kConsumers);
        *abort_flag = 0;
        fence_barrier_init();
        part.head[2 * blockIdx.x].parts = 0;
        part.head[2 * blockIdx.x + 1].parts = 0;
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < c.B; b += kFewThreads)
            if (!seq_valid(c, b)) flag_invalid(c.dev_status);
    const Part p = plan_part<kFewThreads>(c, a, RT, kItemCost, blockIdx.x, gridDim.x);
    __syncthreads();
    launch_dependents();
    if (p.g0 == p.g1) return;

    const int box_log2 = min(c.page_log2, 7);  // runs of keys in one page
    if (warp >= kConsumers) {
        regs_down<kFewRegsDown>();
        // ------------------------------------------------------------ producers
        // Warps 0 and 1 of them load keys, 2 and 3 values, every other run of keys in one page
        // each (a run is a TMA load, and a thread's loads are issued one after the other: eight
        // runs of 16 keys in one warp took longer than the data); the odd ones load the scales.
        const int role = warp - kConsumers, odd = role & 1;
        const CUtensorMap* map = role < 2 ? &tmK : &tmV;
        if (lane == 0) prefetch_tensormap(map);
        const int boxes = kUnit >> box_log2;
        const bool mine = lane < boxes && (lane & 1) == odd;
        ItemWalk<kItemCost> w;
        bool more = w.start(c, a, RT, p), ok = true;
        int it = 0;
        while (more && ok) {
            const int r0 = w.tile * RT, rows = min(RT, w.s.n * a.G - r0), on = w.parts_on(p, blockIdx.x);
            // table entry of run `lane` of unit u, asked for one unit ahead; -1 where no row sees the run
            auto entry = [&](int u) -> int {
                const int k = u * kUnit + (lane << box_log2);
                if (lane >= boxes || u >= w.end || k > w.r.hi || k + (1 << box_log2) <= w.r.lo) return -1;
                const int pg = __ldg(c.table + (int64_t)w.b * c.s_table + (k >> c.page_log2));
                return pg < 0 ? -2 : pg;
            };
            int ahead = entry(w.unit);
            if (role == 0)
                // the item's queries on their way to L2 while the last item's units are under way
                for (int i = lane; i < rows; i += 32) {
                    const int tok = (r0 + i) / a.G;
                    const uint16_t* src =
                        a.Q + (int64_t)(w.s.q0 + tok) * a.q_sn + (int64_t)(w.h * a.G + r0 + i - tok * a.G) * a.q_sh;
                    prefetch_l2(src);
                    if (D == 128) prefetch_l2(src + 64);
                }
            for (int u = w.unit; u < w.end; ++u, ++it) {
                const int st = it % NS, key0 = u * kUnit;
                const bool skip = SKIP && it == a.skip_unit && role < 2;
                int pg = ahead;
                ahead = entry(u + 1);
                if (pg == -2 || pg >= c.pages) {
                    flag_invalid(c.dev_status);
                    pg = -1;
                }
                const int box_ok = (int)__ballot_sync(0xffffffffu, pg >= 0);
                if (it >= NS && !mbar_wait_counted<ATTEMPTS>(empty + 8 * st, (it / NS - 1) & 1, abort_flag, c.dev_status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (role == 0) {
                        StageInfo* f = reinterpret_cast<StageInfo*>(smem + C::OFF_INFO + st * 64);
                        const bool all_seen = key0 >= w.r.lo_all && key0 + kUnit - 1 <= w.r.hi_all &&
                                              box_ok == (1 << boxes) - 1;
                        f->flags = (u == w.unit ? kFirst : 0) | (u == w.end - 1 ? kLast : 0) |
                                   (all_seen ? 0 : kMasked) | (w.head ? kHead : 0) | (w.tail ? kTail : 0);
                        f->key0 = key0;
                        f->q0 = w.s.q0;
                        f->n = w.s.n;
                        f->L = w.s.L;
                        f->h = w.h;
                        f->r0 = r0;
                        f->rows = rows;
                        f->box_ok = box_ok;
                        f->pad[1] = on;
                    }
                    if (!skip) mbar_arrive_expect_tx(full + 8 * st, (uint32_t)((boxes + 1 - odd) >> 1 << box_log2) * D);
                }
                __syncwarp();
                if (mine && !skip) {
                    const uint32_t at = sbase + (role < 2 ? C::OFF_K : C::OFF_V) + st * C::TILE +
                                        (uint32_t)(lane << box_log2) * D;
                    const int in = (key0 + (lane << box_log2)) & ((1 << c.page_log2) - 1);
                    tma_load_4d(at, map, 0, in, w.h, pg, full + 8 * st);
                }
                if (odd && !skip) {
                    // four keys' scales a lane; 0 where the page is not there
                    const int spg = __shfl_sync(0xffffffffu, pg, (4 * lane) >> box_log2);
                    const int in = (key0 + 4 * lane) & ((1 << c.page_log2) - 1);
                    const int64_t off = spg < 0 ? 0 : (int64_t)spg * c.t_page + (int64_t)w.h * c.t_head + in;
                    cp_async16(sbase + C::OFF_SC + (2 * st + role / 2) * (kUnit * 4) + lane * 16,
                               (role < 2 ? c.sk : c.sv) + off, spg < 0 ? 0 : 16);
                    cp_async_arrive(full + 8 * st);
                }
            }
            if (ok) more = w.next(c, a, RT);
        }
        if (ok) {
            // the stage that ends the consumers' loop
            const int st = it % NS;
            if (it < NS || mbar_wait_counted<ATTEMPTS>(empty + 8 * st, (it / NS - 1) & 1, abort_flag, c.dev_status)) {
                if (lane == 0 && role == 0) reinterpret_cast<StageInfo*>(smem + C::OFF_INFO + st * 64)->flags = kEnd;
                if (lane == 0) mbar_arrive(full + 8 * st);
                if (odd) mbar_arrive(full + 8 * st);
                ++it;
            }
        }
        // this CTA's own copies land before it can exit
        uint32_t left = ATTEMPTS;
        for (int j = it > NS ? it - NS : 0; j < it; ++j)
            if (!SKIP || j != a.skip_unit) drain_wait_counted(full + 8 * (j % NS), (j / NS) & 1, left);
    } else {
        // ------------------------------------------------------------ consumers
        regs_up<kFewRegsUp>();
        constexpr int SLICES = RG <= 2 ? 8 : kConsumers / RG, SLICE = kUnit / SLICES;  // of a stage's keys
        constexpr int SETS = kConsumers / (RG * SLICES);  // sets of warps that take turns at the stages
        constexpr int KSTEPS = D / 16, MT = D / 16;
        const int g = lane >> 2, tig = lane & 3;
        const int rg = warp % RG, slice = warp / RG % SLICES, set = warp / (RG * SLICES);
        float* scr = reinterpret_cast<float*>(smem + C::OFF_SCR);
        float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
        const int kr0 = C::key_of(2 * tig), kr1 = C::key_of(2 * tig + 1), krg = C::key_of(g);
        uint32_t q[KSTEPS][2];
        float o[MT][4], M[2], N[2], l[2], qs[2];  // rows 2 tig and 2 tig + 1 of the warp's 8
        int last[2], first[2];
        int it = 0, items = 0;
        while (true) {
            const int st = it % NS;
            if (!mbar_wait_counted<ATTEMPTS>(full + 8 * st, (it / NS) & 1, abort_flag, c.dev_status)) break;
            const StageInfo* info = reinterpret_cast<const StageInfo*>(smem + C::OFF_INFO + st * 64);
            const int flags = info->flags;
            if (flags & kEnd) break;
            if (flags & kFirst) {
                const int q0 = info->q0, h = info->h, r0 = info->r0, rows = info->rows;
                // this thread's channels of row g, as the narrow operand: step s of 16
                // channels holds, per thread, 4 consecutive ones
                const int row = rg * 8 + g;
                const int r = r0 + (row < rows ? row : 0), tok = r / a.G, j = r - tok * a.G;
                const uint16_t* src = a.Q + (int64_t)(q0 + tok) * a.q_sn + (int64_t)(h * a.G + j) * a.q_sh + tig * 16;
                uint32_t wd[D / 32][4], top = 0;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 x = row < rows ? __ldg(reinterpret_cast<const uint4*>(src + (i / 2) * 64) + (i & 1))
                                               : make_uint4(0, 0, 0, 0);
                    wd[i][0] = x.x;
                    wd[i][1] = x.y;
                    wd[i][2] = x.z;
                    wd[i][3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) top = max(top, max(wd[i][k] & 0x7FFFu, (wd[i][k] >> 16) & 0x7FFFu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // a query that is not finite gives NaN, also where all its scores are -inf
                const float f = row_factor(top), qg = top < 0x7F80u ? a.scale_log2 / f : __int_as_float(0x7FFFFFFF);
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        q[2 * i + k / 2][k & 1] = pack_f16(bf16_bits_to_f32(wd[i][k] & 0xFFFFu) * f,
                                                           __uint_as_float(wd[i][k] & 0xFFFF0000u) * f);
                const SeqInfo s{q0, info->n, info->L};
                const int lg = row_last(a, s, tok);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qs[e] = __shfl_sync(0xffffffffu, qg, (2 * tig + e) * 4);
                    last[e] = __shfl_sync(0xffffffffu, lg, (2 * tig + e) * 4);
                    first[e] = row_first(a, last[e]);
                    M[e] = N[e] = -INFINITY;
                    l[e] = 0.f;
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[m][i] = 0.f;
            }
            const uint8_t* ks = smem + C::OFF_K + st * C::TILE;
            const uint8_t* vs = smem + C::OFF_V + st * C::TILE;
            const float* sks = reinterpret_cast<const float*>(smem + C::OFF_SC + st * (2 * kUnit * 4));
            const float* svs = sks + kUnit;
            if (SETS == 1 || it % SETS == set)
#pragma unroll 1
                for (int blk = 0; blk < SLICE / 16; ++blk) {
                    const int kb = slice * SLICE + blk * 16;  // 16 keys
                    float x[4] = {0.f, 0.f, 0.f, 0.f};  // keys g (x[0], x[1]) and g + 8, rows 2 tig and 2 tig + 1
                    float z[4] = {0.f, 0.f, 0.f, 0.f};  // the same of the other half of the channels' steps
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        const uint4 u0 = *reinterpret_cast<const uint4*>(ks + C::chunk(kb + krg, hf * 4 + tig));
                        const uint4 u1 = *reinterpret_cast<const uint4*>(ks + C::chunk(kb + 8 + krg, hf * 4 + tig));
                        const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t ka[4];
                            e4m3x4_to_f16(w0[k], ka[0], ka[2]);
                            e4m3x4_to_f16(w1[k], ka[1], ka[3]);
                            mma_f16((k & 1) ? z : x, ka, q[hf * 4 + k][0], q[hf * 4 + k][1]);
                        }
                    }
                    // y = (q . k8) sk scale log2 e, x = y + log2 sv: -inf where a token's values are all
                    // zero, NaN both where they are no numbers
                    float y[4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int k = kb + 8 * t + krg;
                        const float sv = svs[k], lv = lg2_approx(sv);
                        const float sk = sv < INFINITY ? sks[k] : __int_as_float(0x7FFFFFFF);
                        y[2 * t] = (x[2 * t] + z[2 * t]) * sk * qs[0];
                        y[2 * t + 1] = (x[2 * t + 1] + z[2 * t + 1]) * sk * qs[1];
                        x[2 * t] = y[2 * t] + lv;
                        x[2 * t + 1] = y[2 * t + 1] + lv;
                    }
                    if (flags & kMasked) {
                        const int key0 = info->key0, L = info->L, box_ok = info->box_ok;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int k = kb + 8 * t + krg, pos = key0 + k;
                            const bool there = pos < L && ((box_ok >> (k >> box_log2)) & 1);
                            if (!there || pos > last[0] || pos < first[0]) x[2 * t] = y[2 * t] = -INFINITY;
                            if (!there || pos > last[1] || pos < first[1]) x[2 * t + 1] = y[2 * t + 1] = -INFINITY;
                        }
                    }
                    float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
                    float my0 = fmaxf(y[0], y[2]), my1 = fmaxf(y[1], y[3]);
                    if (__any_sync(0xffffffffu, mx0 > M[0] + kStale || mx1 > M[1] + kStale || my0 > N[0] + kStale ||
                                                    my1 > N[1] + kStale)) {
#pragma unroll
                        for (int i = 4; i < 32; i <<= 1) {
                            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, i));
                            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, i));
                            my0 = fmaxf(my0, __shfl_xor_sync(0xffffffffu, my0, i));
                            my1 = fmaxf(my1, __shfl_xor_sync(0xffffffffu, my1, i));
                        }
                        const float n0 = fmaxf(M[0], mx0), n1 = fmaxf(M[1], mx1);
                        const float a0 = part_weight(M[0], n0), a1 = part_weight(M[1], n1);
                        M[0] = n0;
                        M[1] = n1;
                        my0 = fmaxf(N[0], my0);
                        my1 = fmaxf(N[1], my1);
                        l[0] *= part_weight(N[0], my0);
                        l[1] *= part_weight(N[1], my1);
                        N[0] = my0;
                        N[1] = my1;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            o[m][0] *= a0;
                            o[m][1] *= a1;
                            o[m][2] *= a0;
                            o[m][3] *= a1;
                        }
                    }
                    const float m0 = M[0] == -INFINITY ? 0.f : M[0], m1 = M[1] == -INFINITY ? 0.f : M[1];
                    const float n0 = N[0] == -INFINITY ? 0.f : N[0], n1 = N[1] == -INFINITY ? 0.f : N[1];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        x[2 * t] = ex2_approx(x[2 * t] - m0);
                        x[2 * t + 1] = ex2_approx(x[2 * t + 1] - m1);
                        l[0] += ex2_approx(y[2 * t] - n0);
                        l[1] += ex2_approx(y[2 * t + 1] - n1);
                    }
                    // P^T: keys as the products' inner index, this thread's row g
                    const uint32_t p0 = transpose8(pack_f16(x[0], x[1])), p1 = transpose8(pack_f16(x[2], x[3]));
                    // V^T P^T: the four keys of this thread, D/8 channels of each
                    uint32_t v[4][D / 32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = kb + 8 * (k >> 1) + ((k & 1) ? kr1 : kr0);
                        if (D == 128) {
                            const uint4 t4 = *reinterpret_cast<const uint4*>(vs + C::chunk(r, (g >> 1) + 4 * (g & 1)));
                            v[k][0] = t4.x;
                            v[k][1] = t4.y;
                            v[k][2 % (D / 32)] = t4.z;
                            v[k][3 % (D / 32)] = t4.w;
                        } else {
                            const uint2 t2 = *reinterpret_cast<const uint2*>(vs + C::chunk(r, g >> 1) + (g & 1) * 8);
                            v[k][0] = t2.x;
                            v[k][1] = t2.y;
                        }
                    }
                    if (flags & kMasked) {
                        // what lies behind the last token may be any bits: not a factor
                        const int key0 = info->key0, L = info->L, box_ok = info->box_ok;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = kb + 8 * (k >> 1) + ((k & 1) ? kr1 : kr0);
                            const bool there = key0 + r < L && ((box_ok >> (r >> box_log2)) & 1);
#pragma unroll
                            for (int i = 0; i < D / 32; ++i) v[k][i] = there ? v[k][i] : 0u;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        // channels 4 i .. 4 i + 3 of this thread: rows g and g + 8 of two tiles
                        uint32_t va[4], vb[4];
                        e4m3x4_to_f16(prmt(v[0][i], v[1][i], 0x5140u), va[0], va[1]);
                        e4m3x4_to_f16(prmt(v[2][i], v[3][i], 0x5140u), va[2], va[3]);
                        e4m3x4_to_f16(prmt(v[0][i], v[1][i], 0x7362u), vb[0], vb[1]);
                        e4m3x4_to_f16(prmt(v[2][i], v[3][i], 0x7362u), vb[2], vb[3]);
                        mma_f16(o[2 * i], va, p0, p1);
                        mma_f16(o[2 * i + 1], vb, p0, p1);
                    }
                }
            const int key_end = flags & kLast;
            const int q0 = info->q0, h = info->h, r0 = info->r0, rows = info->rows, on = info->pad[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * st);
            ++it;
            if (!key_end) continue;

            // ------------------------------------------------------------ the item's end
            // the accumulators are free to overwrite once the last item's were read
            if (items > 0 && !mbar_wait_counted<ATTEMPTS>(read, (items - 1) & 1, abort_flag, c.dev_status)) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], i);
                // one maximum for both from here on
                const float m = fmaxf(M[e], N[e]), wo = part_weight(M[e], m);
                l[e] *= part_weight(N[e], m);
                float* dst = scr + ((size_t)warp * 8 + 2 * tig + e) * D + C::channel_of(g);
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    *reinterpret_cast<float4*>(dst + 4 * i) =
                        make_float4(o[2 * i][e] * wo, o[2 * i][2 + e] * wo, o[2 * i + 1][e] * wo, o[2 * i + 1][2 + e] * wo);
                if (g == 0) {
                    ml[warp * 8 + 2 * tig + e] = m;
                    ml[kConsumers * 8 + warp * 8 + 2 * tig + e] = l[e];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(written);
            if (!mbar_wait_counted<ATTEMPTS>(written, items & 1, abort_flag, c.dev_status)) break;
            const bool split = flags & (kHead | kTail);
            const int slot = 2 * blockIdx.x + ((flags & kHead) ? 0 : 1);
            for (int i = threadIdx.x; i < rows * (D / 4); i += kConsumers * 32) {
                const int row = i / (D / 4), ch = (i % (D / 4)) * 4;
                const int at0 = (row / 8) * 8 + row % 8;  // warp rg of the first slice
                float m = -INFINITY, lsum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kConsumers / RG; ++s) m = fmaxf(m, ml[at0 + s * RG * 8]);
#pragma unroll
                for (int s = 0; s < kConsumers / RG; ++s) {
                    const int at = at0 + s * RG * 8;
                    const float w = part_weight(ml[at], m);
                    lsum = fmaf(w, ml[kConsumers * 8 + at], lsum);
                    const float4 u = *reinterpret_cast<const float4*>(scr + (size_t)at * D + ch);
                    acc[0] = fmaf(w, u.x, acc[0]);
                    acc[1] = fmaf(w, u.y, acc[1]);
                    acc[2] = fmaf(w, u.z, acc[2]);
                    acc[3] = fmaf(w, u.w, acc[3]);
                }
                if (split) {
                    *reinterpret_cast<float4*>(part.o + ((size_t)slot * RT + row) * D + ch) =
                        make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (ch == 0) {
                        part.m[(size_t)slot * RT + row] = m;
                        part.l[(size_t)slot * RT + row] = lsum;
                    }
                } else {
                    store_row(a, q0, h, r0 + row, ch, acc, inverse_sum(lsum));
                    if (ch == 0) store_lse(a, c, q0, h, r0 + row, m, lsum);
                }
            }
            if (split && threadIdx.x == 0)
                part.head[slot] = PartHeader{on, q0, h, r0, rows};
            __syncwarp();
            if (lane == 0) mbar_arrive(read);
            ++items;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------ joining
//
// join_kernel: blocks (i, .) take the item that begins in CTA i's part and goes
// on in the next ones, and add its rows' parts in key order; the blocks also
// share out the rows whose tiles see no key at all, which no CTA had.  A launch
// and two L2 round trips: the header, then the parts' maxima and sums (a lane
// each) with the first accumulators.  A block has WR warps a row, which take every
// WR-th part: 4 for tiles of few rows, of which a long cache makes many parts, 1
// for those of many.  (4 to 20 bytes of spill loads in each instance.)
constexpr int kJoinThreads = 128;

template <int D, int WR>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const PagedAttn a, const CacheView c, void* ws, int RT, int parts) {
    constexpr int E = D / 32, NW = kJoinThreads / 32;  // channels of a lane; warps
    __shared__ float sums[WR > 1 ? NW : 1][D];
    const Partials part = partials_at(ws, RT, D);
    const int i0 = 2 * blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    wait_for_primary();
    const PartHeader hd = part.head[i0];
    const int n = min(hd.parts, parts - (int)blockIdx.x);
    auto slot = [&](int k) { return (size_t)(k ? 2 * ((int)blockIdx.x + k) : i0) * RT; };
    if (n > 0)
        for (int row = blockIdx.y * (NW / WR) + warp / WR; row < hd.rows; row += gridDim.y * (NW / WR)) {
            float m = -INFINITY, l = 0.f, acc[E];
            for (int k = lane; k < n; k += 32) m = fmaxf(m, part.m[slot(k) + row]);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
            for (int k0 = 0; k0 < n; k0 += 32) {
                float w = 0.f, lw = 0.f;
                if (k0 + lane < n) {
                    w = part_weight(part.m[slot(k0 + lane) + row], m);
                    lw = w * part.l[slot(k0 + lane) + row];
                }
                const int some = min(n - k0, 32);
#pragma unroll
                for (int o = 16; o; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
                l += lw;
#pragma unroll 8
                for (int k = warp % WR; k < some; k += WR) {
                    const float wk = __shfl_sync(0xffffffffu, w, k);
                    const float* o = part.o + (slot(k0 + k) + row) * D + lane * E;
                    if constexpr (E == 4) {
                        const float4 u = *reinterpret_cast<const float4*>(o);
                        acc[0] = fmaf(wk, u.x, acc[0]);
                        acc[1] = fmaf(wk, u.y, acc[1]);
                        acc[2] = fmaf(wk, u.z, acc[2]);
                        acc[3] = fmaf(wk, u.w, acc[3]);
                    } else {
                        const float2 u = *reinterpret_cast<const float2*>(o);
                        acc[0] = fmaf(wk, u.x, acc[0]);
                        acc[1] = fmaf(wk, u.y, acc[1]);
                    }
                }
            }
            if (WR > 1) {
                // one row a block at a time: all four warps are here
#pragma unroll
                for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    acc[e] = 0.f;
                    for (int k = 0; k < WR; ++k) acc[e] += sums[k][lane * E + e];
                }
                __syncthreads();
                if (warp) continue;
            }
            store_row(a, hd.q0, hd.h, hd.r0 + row, lane * E, acc, inverse_sum(l));
            if (lane == 0) store_lse(a, c, hd.q0, hd.h, hd.r0 + row, m, l);
        }
    float none[E];
#pragma unroll
    for (int e = 0; e < E; ++e) none[e] = 0.f;
    for (int b = blockIdx.y * gridDim.x + blockIdx.x; b < c.B; b += gridDim.x * gridDim.y) {
        const SeqInfo s = seq_info(c, b);
        const int nt = seq_tiles(a, s, RT);
        for (int t = 0; t < nt; ++t) {
            if (item_range(a, s, t, RT).units()) continue;
            const int r0 = t * RT, rows = min(RT, s.n * a.G - r0);
            for (int i = threadIdx.x / 32; i < c.H * rows; i += kJoinThreads / 32) {
                store_row(a, s.q0, i / rows, r0 + i % rows, lane * E, none, 0.f);
                if (lane == 0) store_lse(a, c, s.q0, i / rows, r0 + i % rows, 0.f, 0.f);
            }
        }
    }
}

// ------------------------------------------------------------ host side

// K8 or V8 as a tensor [page][head][token][channel] of bytes, in boxes of up to 128 tokens.
bool make_cache_map(CUtensorMap* map, const uint8_t* base, int d, const CacheView& c) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_tiled_fn();
    if (!enc) return false;
    const int page = 1 << c.page_log2;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)c.H, (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.s_tok, (cuuint64_t)c.s_head, (cuuint64_t)c.s_page};
    const cuuint32_t box[4] = {(cuuint32_t)d, (cuuint32_t)(page < kUnit ? page : kUnit), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a tile, by the rows of the longest chunk as far as the caller told: up to
// 32 go to the kernel for few rows, more to the one for many.  Measured on 24
// sequences of 500 to 6,000 keys, d = 128, few rows against many: 16 rows 36.0
// against 51.0 us, 32 rows 47.0 against 51.3 (d = 64: 34.8 against 45.3), 64 rows 75.5
// in tiles of 32 against 52.5.  128 rows take 56.0 us in tiles of 128 and 60.9 in
// tiles of 256.  One choice for the whole call: a chunk of 2,000 tokens beside 60 single
// ones (8 x 4 heads) takes 250 us, in two calls 200.
int tile_rows(int G, int B, int T, int max_q) {
    const int64_t q = max_q > 0 ? max_q : ((int64_t)T + B - 1) / B;
    const int64_t rows = q * G;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
}

template <int D>
vc_status launch_join(const PagedAttn& a, const CacheView& c, void* ws, int RT, int parts, cudaStream_t st) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    // few rows: a row a block; many: 32 blocks an item
    cfg.gridDim = dim3(parts, RT <= 32 ? RT : 32);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cuda_status(RT <= 32 ? cudaLaunchKernelEx(&cfg, join_kernel<D, 4>, a, c, ws, RT, parts)
                                : cudaLaunchKernelEx(&cfg, join_kernel<D, 1>, a, c, ws, RT, parts));
}

template <int D, int RG, bool SKIP = false>
vc_status launch_few(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const CacheView& c, void* ws,
                     int ctas, cudaStream_t st) {
    auto kern = attn_few_kernel<D, RG, SKIP>;
    vc_status s = ensure_smem_attr(reinterpret_cast<const void*>(kern), FewCfg<D>::SMEM);
    if (s != VC_OK) return s;
    kern<<<ctas, kFewThreads, FewCfg<D>::SMEM, st>>>(mk, mv, a, c, ws);
    return cuda_status(cudaGetLastError());
}

// CTAs of a call: one on each SM, fewer where there cannot be that much work.
int part_count(const PagedAttn& a, const CacheView& c, int RT) {
    const int64_t tiles = (int64_t)c.T * a.G / RT + c.B;
    const int64_t units = (((int64_t)c.cols << c.page_log2) + kUnit - 1) / kUnit + 1;
    if (tiles * c.H >= kMaxCtas || units >= kMaxCtas) return kMaxCtas;
    return (int)(tiles * c.H * units < kMaxCtas ? tiles * c.H * units : kMaxCtas);
}

template <int D>
vc_status launch_d(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const CacheView& c, void* ws,
                   cudaStream_t st) {
    int RT = tile_rows(a.G, c.B, c.T, a.max_q);
    const bool skip = a.skip_unit >= 0 && RT <= 32;
    if (skip) RT = 8;  // of the kernel for few rows, one instance with the hook
    const int ctas = part_count(a, c, RT);
    vc_status s;
    switch (RT) {
        case 8:
            s = skip ? launch_few<D, 1, true>(mk, mv, a, c, ws, ctas, st) : launch_few<D, 1>(mk, mv, a, c, ws, ctas, st);
            break;
        case 16: s = launch_few<D, 2>(mk, mv, a, c, ws, ctas, st); break;
        case 32: s = launch_few<D, 4>(mk, mv, a, c, ws, ctas, st); break;
        default: s = launch_attn_many(mk, mv, a, c, D, RT, ctas, ws, st);
    }
    return s == VC_OK ? launch_join<D>(a, c, ws, RT, ctas, st) : s;
}

}  // namespace

size_t attn_paged_workspace(const vc_cache_shape& c, int Hq, int B, int T, int max_q) {
    return partials_bytes(tile_rows(Hq / c.H, B, T, max_q), c.d);
}

vc_status launch_attn_paged(const PagedAttn& a, const CacheView& c, int d, void* ws, cudaStream_t st) {
    CUtensorMap mk, mv;
    if (!make_cache_map(&mk, c.K8, d, c) || !make_cache_map(&mv, c.V8, d, c)) return VC_ERR_CUDA;
    return d == 128 ? launch_d<128>(mk, mv, a, c, ws, st) : launch_d<64>(mk, mv, a, c, ws, st);
}

}  // namespace vc

// vc_attn_chunk.cu -- vc_attn_paged for chunks of many rows, on tcgen05.
//
// Per row, over its keys t, with the cached codes k8, v8 and scales sk, sv:
//   s_t = (q . k8_t) sk_t scale log2 e,   P_t = 2^(s_t - M),   l = sum_t P_t,
//   A = sum_t (P_t sv_t) v8_t,            O = A / l,
// M being the running maximum of s_t + log2 sv_t, rounded down to a whole number:
// P sv, which goes to the product as fp16, is then below 2 whatever the scales
// are.  M follows only where the sum of P over the 16 to 64 keys at hand times their
// unit's largest sv passes 2^15, so that P sv stays finite in fp16 (whose precision is
// the same up to there) without a maximum being taken; then a pass of its own over
// these keys finds the new M, and what was summed before is scaled by a power of two.
// l may then have terms of up to 2^111 (1 / sv of the smallest values), or sums of 2^118
// before M follows: where it passes 2^100 it is kept as l lf with lf = 2^-64, and at an
// item's end M, l and O are brought to l < 2, so that parts of any maxima can be added up.
//
// One persistent CTA on each SM takes tiles of 256 rows as two pipelines A and B
// of 128 rows, which share the keys and values and the tensor core, so that the
// softmax of one overlaps the products of the other; a tile of up to 128 rows is
// given to both, which then take its units of 128 keys in turn and are added up at
// its end.
//
// Per unit and pipeline, 128 rows x 128 keys:
//   S = q K8^T in kind::f8f6f4, straight from the cached codes: the query row,
//       scaled by a power of two, is the sum of two E4M3 numbers (4 + 4 bits of
//       the 8 that bf16 has: exact down to 2^-9 of its largest channel, within
//       2^-17 of it below), so two FP8 products of depth d give the score.
//       They cost what one bf16 product would and need no conversion of keys.
//   P V8 in kind::f16: P as fp16 in tensor memory, in the place of S; V8 as fp16,
//       which a warpgroup converts once a unit for both pipelines.  (P as two
//       E4M3 numbers would spare that, but lose everything below 2^-17 of the
//       row's largest: a few thousand keys there are a visible part of a sum.)
// The floor is the tensor core's 4 x 512 clocks a unit of both pipelines (d = 128).
// Measured: 3,770 clocks; 3,600 tokens of 40 heads over 75,600 keys take 4.53 ms call after
// call, 1,229 TFLOP/s at the 1,940 MHz of the power cap, and 4.30 ms for ten calls.  Without
// softmax arithmetic a unit still took 3,150 clocks.  Shared memory's data path is the
// busiest part (products 37 %, loads and stores 56 %, TMA besides), and code
// that runs beside other code costs instruction fetches: two threads a row (5.9 ms), loads
// that need fewer scales (16x256b, 4.6 ms) and warps of their own for the scales (4.8 ms)
// all lost.  With d = 64 the chain from scores to P bounds it as well (tensor core 25 %
// busy).
//
// 16 warps:
//   0-3, 4-7  softmax of A and B: a thread owns a row (its TMEM lane).
//   8-11      converter: a thread owns a key for the scales and 16-byte pieces of
//             the values.
//   12        MMA issuer (and owner of the tensor memory).
//   13        loader: K8, V8 and scales by TMA and bulk copies, and what the
//             others need to know of a unit.  14 and 15 are idle.
// Tensor memory of pipeline X at X (d + 128): O [0, d), S [d, d + 128), P in the
// first 64 columns of S.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kThreads = 512;
constexpr int kConvWarp = 8, kMmaWarp = 12, kLoadWarp = 13;
// 512 x 128 registers at launch: 2 x 128 x 152 + 2 x 128 x 104 = 65,536
constexpr int kRegsSoftmax = 152, kRegsConv = 104, kRegsOther = 104;

// What an item costs besides its units, in units: its queries (5 us), the first scores and the
// last rows, with both pipelines empty, against 2 us a unit.
constexpr int kItemCost = 7;
// The value scale, as -log2, up to which M follows s + log2 sv: below those of the cache that are not 0
// (2^-109), and so that the P of 64 keys whose values are all zero sum up to less than 2^118.
constexpr float kLeastLog2 = 110.f;
// A unit's scales: sk[128], sv[128] (0 where there is no token), the largest sv of each 32.
constexpr int kScaleBytes = (2 * kUnit + 4) * 4;

template <int D>
struct ManyCfg {
    static constexpr int NK = 3, NV = 2, NW = 2, NC = 3, NI = 4;  // stages: K8, V8, fp16 V, scales, infos
    static constexpr int QB = 128 * D;                    // one E4M3 part of a pipeline's queries
    static constexpr int TILE = kUnit * D;                // codes of K or V in a unit
    static constexpr int WB = kUnit * D * 2;              // fp16 values of a unit
    static constexpr int OFF_Q = 0;                       // [X][hi, lo]
    static constexpr int OFF_K = OFF_Q + 4 * QB;
    static constexpr int OFF_V = OFF_K + NK * TILE;
    static constexpr int OFF_W = OFF_V + NV * TILE;
    static constexpr int OFF_RAW = OFF_W + NW * WB;       // [NV][sk | sv][128]
    static constexpr int OFF_SC = OFF_RAW + NV * 2 * kUnit * 4;  // [NC]
    static constexpr int OFF_ML = OFF_SC + NC * kScaleBytes;   // [m | l | factor of O][128] of B, for A
    static constexpr int OFF_INFO = OFF_ML + 3 * 128 * 4;
    static constexpr int OFF_BAR = OFF_INFO + NI * 64;
    static constexpr int OFF_MISC = OFF_BAR + 48 * 8;
    static constexpr int USED = OFF_MISC + 32;
    // at least 116 KB, so that one CTA (and one owner of the tensor memory) sits on an SM
    static constexpr int SMEM = (USED > 118784 ? USED : 118784) + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(QB % 1024 == 0 && TILE % 1024 == 0 && WB % 1024 == 0, "swizzle alignment");
    // barriers
    static constexpr int IF = 0, IE = IF + NI, KF = IE + NI, KE = KF + NK, VF = KE + NK, VE = VF + NV, WF = VE + NV,
                         WE = WF + NW, CF = WE + NW, CE = CF + NC, QF = CE + NC, SF = QF + 2, PF = SF + 2,
                         OD = PF + 2, OE = OD + 2, MB = OE + 2, TD = MB + 1, NBAR = TD + 1;
    static_assert(NBAR <= 48, "barrier area");
    static constexpr uint32_t SWZ = D == 128 ? kSwizzle128B : kSwizzle64B;
    __host__ __device__ static constexpr uint32_t base(int X) { return (uint32_t)X * (D + 128); }
    // Byte offset of 16-byte piece ch of code row r under the swizzle.
    __device__ static int chunk(int r, int ch) {
        return D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
    }
};

// Instruction descriptor, kind::f16: A and B fp16, D fp32, B with its N index contiguous.
__host__ __device__ constexpr uint32_t idesc_f16_bn(uint32_t M, uint32_t N) {
    return (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// 2^e for a whole e <= 127, exactly; 0 below 2^-149.
__device__ __forceinline__ float pow2_whole(int e) {
    return __int_as_float(e >= -126 ? (e + 127) << 23 : e >= -149 ? 1 << (e + 149) : 0);
}
__device__ __forceinline__ int exponent_of(float x) { return (__float_as_int(x) >> 23) - 127; }  // x >= 2^-126

// The same value, as far as the compiler may know another one each time.
__device__ __forceinline__ int no_hoist(int x) {
    asm volatile("" : "+r"(x));
    return x;
}

// SKIP: the test hook that leaves out the keys of unit a.skip_unit, in instances of its own (in the others
// these few instructions of the loader cost 4 % of the time of windowed chunks).
// SHARED: a pass of the attention over shared prefixes.
template <int D, int kChunk, bool SKIP, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const AttnOf<SHARED> a, const CacheView c, int RT, void* ws) {
    using C = ManyCfg<D>;
    constexpr uint32_t ATTEMPTS = SKIP ? kHookAttempts : kWaitAttempts;
    // Keys that the softmax takes between two decisions about M: kChunk, and in units with a mask,
    // whose code is longer, kMaskedChunk.  The less code, the better the instruction caches hold it
    // beside the other pipeline's; the longer a chunk, the more overlaps within it.
    //   d = 128, tiles of 256 rows, 3,600 rows over 75,600 keys: 64 keys 4.51 ms, 32 4.95, 16 5.22,
    //     all 128 5.10; masked 16 against 32: ragged chunks 115 against 124 us.
    //   d = 128, tiles of 128 rows, a few tokens of 24 sequences: 16 keys 53.1 us, 32 54.8, 64 58.4.
    //   d = 64, windowed chunks: 32 keys 0.750 ms, 64 0.918, 16 0.797; masked 16 0.759.
    // (The instance of 16 keys has 8 bytes of spill stores and 136 of spill loads, the others none.)
    constexpr int kMaskedChunk = D == 128 ? 16 : 32;
    // offsets from the array itself: through an integer the compiler would lose sight of
    // the address space, and generic loads take the slow road to shared memory
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    auto wait = [&](int i, int phase) -> bool {
        return mbar_wait_counted<ATTEMPTS>(bar(i), phase & 1, abort_flag, c.dev_status);
    };

    if (threadIdx.x == 0) {
        auto init = [&](int first, int n, int count) {
            for (int i = 0; i < n; ++i) mbar_init(bar(first + i), count);
        };
        init(C::IF, C::NI, 1);
        init(C::IE, C::NI, 8 + 4 + 1);  // softmax and converter warps, MMA issuer
        init(C::KF, C::NK, 1);
        init(C::KE, C::NK, 1);
        init(C::VF, C::NV, 1);
        init(C::VE, C::NV, 4);
        init(C::WF, C::NW, 4);
        init(C::WE, C::NW, 1);
        init(C::CF, C::NC, 4);
        init(C::CE, C::NC, 8);
        init(C::QF, 2, 4);
        init(C::SF, 2, 1);
        init(C::PF, 2, 4);
        init(C::OD, 2, 1);
        init(C::OE, 2, 4);
        init(C::MB, 1, 4);
        init(C::TD, 1, 1);
        *abort_flag = 0;
        fence_barrier_init();
        if constexpr (!SHARED) {
            const Partials part = partials_at(ws, RT, D);
            part.head[2 * blockIdx.x].parts = 0;
            part.head[2 * blockIdx.x + 1].parts = 0;
        }
    }
    auto plan = [&] {
        if constexpr (SHARED) {
            if (a.pass == 1) wait_for_primary();  // the plan; the second pass starts when all of the first have it
            return load_part(a.plan + (a.pass == 1 ? 0 : kMaxCtas * a.per_sm[0]) + blockIdx.x);
        } else {
            if (blockIdx.x == 0)
                for (int b = threadIdx.x; b < c.B; b += kThreads)
                    if (!seq_valid(c, b)) flag_invalid(c.dev_status);
            return plan_part<kThreads>(c, a, RT, kItemCost, blockIdx.x, gridDim.x);
        }
    };
    const auto p = plan();
    __syncthreads();
    launch_dependents();
    if (p.g0 == p.g1) {
        if (SHARED) wait_for_primary();
        return;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int box_log2 = min(c.page_log2, 7);  // runs of keys in one page
    auto info_at = [&](int it) -> const StageInfo* {
        return reinterpret_cast<const StageInfo*>(smem + C::OFF_INFO + (it % C::NI) * 64);
    };

    if (warp >= kMmaWarp) {
        regs_down<kRegsOther>();
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ loader
            if (lane == 0) {
                prefetch_tensormap(&tmK);
                prefetch_tensormap(&tmV);
            }
            const int boxes = kUnit >> box_log2;
            ItemWalk<kItemCost, SHARED> w;
            bool more = w.start(c, a, RT, p), ok = true;
            int it = 0, loaded_k = 0, loaded_v = 0;
            while (more && ok) {
                const int r0 = w.tile * RT, rows = min(RT, w.s.n * a.G - r0), on = w.parts_on(p, blockIdx.x);
                // table entry of run `lane` of unit u, asked for one unit ahead; -1 where no row sees the run
                auto entry = [&](int u) -> int {
                    const int k = u * kUnit + (lane << box_log2);
                    if (lane >= boxes || u >= w.end || k > w.r.hi || k + (1 << box_log2) <= w.r.lo) return -1;
                    const int pg = __ldg(c.table + (int64_t)w.table_row() * c.s_table + (k >> c.page_log2));
                    return pg < 0 ? -2 : pg;
                };
                int ahead = -1;
                Runs runs;
                if constexpr (SHARED) runs.start(c, w, box_log2);
                else ahead = entry(w.unit);
                // the item's queries on their way to L2 while the last item's units are under way
                for (int i = lane; i < rows; i += 32) {
                    const int r = r0 + i, tok = r / a.G;
                    const uint16_t* src =
                        a.Q + (int64_t)(w.s.q0 + tok) * a.q_sn + (int64_t)(w.h * a.G + r - tok * a.G) * a.q_sh;
                    prefetch_l2(src);
                    if (D == 128) prefetch_l2(src + 64);
                }
                for (int u = w.unit; u < w.end; ++u, ++it) {
                    const int key0 = w.key0(u);
                    int pg = ahead;
                    if constexpr (SHARED) pg = runs.at(c, w, u, box_log2);
                    else ahead = entry(u + 1);
                    const bool missing = pg == -2 || pg >= c.pages;
                    if (missing) {
                        flag_invalid(c.dev_status);
                        pg = -1;
                    }
                    const bool holes = __any_sync(0xffffffffu, missing);
                    const int box_ok = (int)__ballot_sync(0xffffffffu, pg >= 0);
                    ok = it < C::NI || wait(C::IE + it % C::NI, it / C::NI - 1);
                    if (!ok) break;
                    if (lane == 0) {
                        StageInfo* f = const_cast<StageInfo*>(info_at(it));
                        const bool all_seen = key0 >= w.r.lo_all && key0 + kUnit - 1 <= w.r.hi_all;
                        f->flags = (u == w.unit ? kFirst : 0) | (u == w.end - 1 ? kLast : 0) |
                                   (all_seen && !holes ? 0 : kMasked) | (holes ? kHoles : 0) | (w.head ? kHead : 0) |
                                   (w.tail ? kTail : 0);
                        f->key0 = key0;
                        f->q0 = w.s.q0;
                        f->n = w.s.n;
                        f->L = w.s.L;
                        f->h = w.h;
                        f->r0 = r0;
                        f->rows = rows;
                        f->box_ok = box_ok;
                        f->pad[0] = u - w.unit;
                        f->pad[1] = on;
                        if (SHARED) f->pad[2] = first_of<SHARED>(w.s);
                        mbar_arrive(bar(C::IF + it % C::NI));
                    }
                    __syncwarp();
                    const int in = (key0 + (lane << box_log2)) & ((1 << c.page_log2) - 1);
                    const uint32_t at = (uint32_t)(lane << box_log2) * D;
                    const int sk = it % C::NK, sv = it % C::NV;
                    ok = it < C::NK || wait(C::KE + sk, it / C::NK - 1);
                    if (!ok) break;
                    const bool skip = SKIP && it == a.skip_unit;
                    if (lane == 0 && !skip) mbar_arrive_expect_tx(bar(C::KF + sk), C::TILE);
                    __syncwarp();
                    if (lane < boxes && !skip)
                        tma_load_4d(sbase + C::OFF_K + sk * C::TILE + at, &tmK, 0, in, w.h, pg, bar(C::KF + sk));
                    loaded_k = it + 1;
                    ok = it < C::NV || wait(C::VE + sv, it / C::NV - 1);
                    if (!ok) break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar(C::VF + sv),
                                              C::TILE + ((uint32_t)__popc(box_ok) << (box_log2 + 3)));
                    __syncwarp();
                    if (lane < boxes)
                        tma_load_4d(sbase + C::OFF_V + sv * C::TILE + at, &tmV, 0, in, w.h, pg, bar(C::VF + sv));
                    if (pg >= 0) {
                        const int64_t off = (int64_t)pg * c.t_page + (int64_t)w.h * c.t_head + in;
                        const uint32_t dst = sbase + C::OFF_RAW + sv * (2 * kUnit * 4) + (lane << (box_log2 + 2));
                        bulk_load(dst, c.sk + off, 4u << box_log2, bar(C::VF + sv));
                        bulk_load(dst + kUnit * 4, c.sv + off, 4u << box_log2, bar(C::VF + sv));
                    }
                    loaded_v = it + 1;
                }
                if (ok) more = w.next(c, a, RT);
            }
            if (ok && (it < C::NI || wait(C::IE + it % C::NI, it / C::NI - 1))) {
                if (lane == 0) {
                    const_cast<StageInfo*>(info_at(it))->flags = kEnd;
                    mbar_arrive(bar(C::IF + it % C::NI));
                }
                __syncwarp();
            }
            // this CTA's own copies land before it can exit
            uint32_t left = ATTEMPTS;
            for (int j = max(loaded_k - C::NK, 0); j < loaded_k; ++j)
                if (!SKIP || j != a.skip_unit) drain_wait_counted(bar(C::KF + j % C::NK), (j / C::NK) & 1, left);
            for (int j = max(loaded_v - C::NV, 0); j < loaded_v; ++j)
                drain_wait_counted(bar(C::VF + j % C::NV), (j / C::NV) & 1, left);
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------ MMA issuer
            // One warp issues for both pipelines, in turn: the product P V of a pipeline's last
            // unit, then its next scores, then the same for the other.  So the two stay half a
            // step apart, one in its softmax while the tensor core works for the other.  (Two
            // issuers side by side fell into step, each waiting for both pipelines' products.)
            constexpr uint32_t IDESC_QK = idesc_f8_e4m3(128, 128), IDESC_PV = idesc_f16_bn(128, D);
            int items = 0;                           // items ended
            int own[2] = {0, 0};                     // units whose P V has been issued
            int pend[2] = {-1, -1};                  // unit whose P V is to be issued
            bool pend_both = false, fresh[2] = {true, true}, ended = false, ok = true;
            for (int it = 0; ok; ++it) {
                if (!(ok = wait(C::IF + it % C::NI, it / C::NI))) break;
                const StageInfo* f = info_at(it);
                const int flags = f->flags, place = f->pad[0];
                const bool both = f->rows > 128;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::IE + it % C::NI));
                const int sk = it % C::NK;
                // P V of pipeline X's pending unit
                auto issue_pv = [&](int X) -> bool {
                    const uint32_t tb = tmem + C::base(X);
                    const int u = pend[X], sw = u % C::NW;
                    // a new item's first product waits until the last item's rows have been read
                    if (fresh[X] && items > 0 && !wait(C::OE + X, items - 1)) return false;
                    if (!wait(C::WF + sw, u / C::NW) || !wait(C::PF + X, own[X])) return false;
                    tc_fence_after();
                    const uint64_t wd = smem_desc_lbo(sbase + C::OFF_W + sw * C::WB, 128 * 128, 1024, kSwizzle128B);
#pragma unroll
                    for (int i = 0; i < kUnit / 16; ++i)
                        mma_bf16_ts_w(tb, tb + D + i * 8, wd + i * 128, IDESC_PV, (fresh[X] && i == 0) ? 0u : 1u);
                    if (!pend_both || X == 1) mma_commit_w(bar(C::WE + sw));
                    fresh[X] = false;
                    ++own[X];
                    pend[X] = -1;
                    return true;
                };
                if (ended) {
                    // both pipelines' ends before the new item: its queries wait for them
#pragma unroll
                    for (int X = 0; X < 2; ++X) {
                        if (pend[X] >= 0 && !(ok = issue_pv(X))) break;
                        mma_commit_w(bar(C::OD + X));
                        fresh[X] = true;
                    }
                    if (!ok) break;
                    ++items;
                }
                if (flags & kEnd) break;
#pragma unroll
                for (int X = 0; X < 2; ++X) {
                    if ((flags & kFirst) && !(ok = wait(C::QF + X, items))) break;
                    if (!both && (place & 1) != X) continue;
                    if (pend[X] >= 0 && !(ok = issue_pv(X))) break;
                    if (!(ok = wait(C::KF + sk, it / C::NK))) break;
                    // S is free: the product that reads the last P from its place was issued before
                    tc_fence_after();
                    // steps of 32 bytes (2 in a descriptor's units)
                    const uint64_t kd = smem_desc(sbase + C::OFF_K + sk * C::TILE, 8 * D, C::SWZ);
                    const uint64_t qd = smem_desc(sbase + C::OFF_Q + 2 * X * C::QB, 8 * D, C::SWZ);
#pragma unroll
                    for (int i = 0; i < 2 * (D / 32); ++i)
                        mma_f8_ss_w(tmem + C::base(X) + D, qd + (i / (D / 32)) * (C::QB / 16) + (i % (D / 32)) * 2,
                                    kd + (i % (D / 32)) * 2, IDESC_QK, i > 0 ? 1u : 0u);
                    mma_commit_w(bar(C::SF + X));
                    if (!both || X == 1) mma_commit_w(bar(C::KE + sk));
                    pend[X] = it;
                }
                pend_both = both;
                ended = flags & kLast;
            }
            // every MMA this warp issued has completed once this phase flips
            mma_commit_w(bar(C::TD));
            uint32_t left = ATTEMPTS;
            drain_wait_counted(bar(C::TD), 0, left);
            __syncwarp();
        }
    } else if (warp >= kConvWarp) {
        // ------------------------------------------------------------ converter
        regs_down<kRegsConv>();
        const int t = threadIdx.x - kConvWarp * 32;
        // Pieces of 16 codes: this thread's are piece ch of tokens row0 + i ROWS, whose swizzle is the
        // same for all i.  As fp16 a piece is two of 16 bytes: 64 channels a half, 128 bytes a token,
        // 128-byte swizzle; the halves' threads write theirs in opposite order, which keeps them on
        // different banks.
        constexpr int PIECES = D / 16, ROWS = 128 / PIECES;
        static_assert(ROWS % 8 == 0, "one swizzle");
        const int row0 = t / PIECES, ch = t % PIECES;
        const bool swap = ch >= 4;
        const int from = C::chunk(row0, ch);
        const int lo = (((ch & 3) * 2) ^ (row0 & 7)) << 4, hi = (((ch & 3) * 2 + 1) ^ (row0 & 7)) << 4;
        const int to = (ch / 4) * (kUnit * 128) + row0 * 128 + (swap ? hi : lo), other = swap ? lo - hi : hi - lo;
        for (int it = 0;; ++it) {
            if (!wait(C::IF + it % C::NI, it / C::NI)) break;
            const StageInfo* f = info_at(it);
            const int flags = f->flags, key0 = f->key0, L = f->L, box_ok = f->box_ok;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::IE + it % C::NI));
            const int sv = it % C::NV, sw = it % C::NW, sc = it % C::NC;
            if (flags & kEnd) break;
            if (!wait(C::VF + sv, it / C::NV)) break;
            if (it >= C::NC && !wait(C::CE + sc, it / C::NC - 1)) break;
            {
                const float* raw = reinterpret_cast<const float*>(smem + C::OFF_RAW + sv * (2 * kUnit * 4));
                float* out = reinterpret_cast<float*>(smem + C::OFF_SC + sc * kScaleBytes);
                const bool there = key0 + t < L && ((box_ok >> (t >> box_log2)) & 1);
                const float k = raw[t], v = raw[kUnit + t];
                const bool number = v < INFINITY;
                // a token whose values are not numbers gets a score that is none: it spoils the
                // rows that see it and no other, for which 0 * 0 stays 0
                out[t] = !there ? 0.f : number ? k : __int_as_float(0x7FFFFFFF);
                out[kUnit + t] = there && number ? v : 0.f;
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(there && number ? v : 0.f));
                if (lane == 0) out[2 * kUnit + (t >> 5)] = __uint_as_float(top);  // the largest of these 32
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::CF + sc));
            }
            if (it >= C::NW && !wait(C::WE + sw, it / C::NW - 1)) break;
            const uint8_t* src = smem + C::OFF_V + sv * C::TILE + from;
            uint8_t* dst = smem + C::OFF_W + sw * C::WB + to;
#pragma unroll 1
            for (int i = 0; i < PIECES; ++i) {
                uint4 x = *reinterpret_cast<const uint4*>(src + i * ROWS * D);
                if ((flags & kMasked) && key0 + row0 + i * ROWS >= L) x = make_uint4(0, 0, 0, 0);  // any bits behind the last token
                uint4 y0, y1;
                e4m3x4_to_f16(swap ? x.z : x.x, y0.x, y0.y);
                e4m3x4_to_f16(swap ? x.w : x.y, y0.z, y0.w);
                e4m3x4_to_f16(swap ? x.x : x.z, y1.x, y1.y);
                e4m3x4_to_f16(swap ? x.y : x.w, y1.z, y1.w);
                *reinterpret_cast<uint4*>(dst + i * ROWS * 128) = y0;
                *reinterpret_cast<uint4*>(dst + i * ROWS * 128 + other) = y1;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::WF + sw));
                mbar_arrive(bar(C::VE + sv));
            }
        }
    } else {
        // ------------------------------------------------------------ softmax of pipeline X
        regs_up<kRegsSoftmax>();
        const int X = warp >> 2, q = warp & 3, row = q * 32 + lane;
        const uint32_t la = tmem + ((uint32_t)(q * 32) << 16) + C::base(X);
        float M = -INFINITY, l = 0.f, lf = 1.f, qs = 0.f;
        int last = -1, first = 0, items = 0, own = 0, shared = 0;
        bool fresh = true, begin = true;
        for (int it = 0;; ++it) {
            const int sc = it % C::NC;
            // inside an item the scales' arrival says that the info, which the converter reads
            // before, is there too
            if (begin ? !wait(C::IF + it % C::NI, it / C::NI) : !wait(C::CF + sc, it / C::NC)) break;
            const StageInfo* f = info_at(it);
            const int flags = f->flags, key0 = f->key0, place = f->pad[0];
            if (flags & kEnd) break;
            const bool both = f->rows > 128, mine = both || (place & 1) == X;
            const int tr = both ? X * 128 + row : row;  // this thread's row of the tile
            if (flags & kFirst) {
                // The warp's 32 rows as two E4M3 parts each; the products that read the last item's
                // have completed.  LR lanes of 16 bytes take a row, so that a load is whole lines,
                // four loads ahead of their use.  A scaled channel's parts are its first 4
                // significant bits and the rest: x & ~15 on the bf16 bits, and the difference.
                constexpr int LR = D / 8, NR = 32 / LR, BATCH = 4;
                const int q0 = f->q0, r0 = f->r0, rows = f->rows;
                const int sub = lane % LR, my = (both ? X * 128 : 0) + q * 32 + lane;  // tile row `lane` of the warp
                const int mr = r0 + (my < rows ? my : 0), mtok = mr / a.G;
                const int64_t my_off = (int64_t)(q0 + mtok) * a.q_sn + (int64_t)(f->h * a.G + mr - mtok * a.G) * a.q_sh;
                const unsigned there = __ballot_sync(0xffffffffu, my < rows);
                uint8_t* qh = smem + C::OFF_Q + 2 * X * C::QB;
                auto load = [&](int i) -> uint4 {
                    const int rr = i * NR + lane / LR;
                    const int64_t off = __shfl_sync(0xffffffffu, my_off, rr & 31);
                    return rr < 32 && (there >> rr & 1u) ? __ldg(reinterpret_cast<const uint4*>(a.Q + off) + sub)
                                                         : make_uint4(0, 0, 0, 0);
                };
                uint4 nx[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) nx[i] = load(i);
#pragma unroll 1
                for (int i0 = 0; i0 < LR; i0 += BATCH) {
                    uint4 x[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        x[i] = nx[i];
                        nx[i] = load(i0 + BATCH + i);
                    }
                    // step by step over the batch: four chains of shuffles side by side
                    uint32_t top[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        top[i] = __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                          __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
                        top[i] = max(top[i] & 0xFFFFu, top[i] >> 16);
                    }
#pragma unroll
                    for (int o = LR / 2; o; o >>= 1)
#pragma unroll
                        for (int i = 0; i < BATCH; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
                    float fac[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        fac[i] = row_factor(top[i]);
                        // to the row's own thread
                        const float g = __shfl_sync(0xffffffffu, fac[i], (lane % NR) * LR);
                        if (lane / NR == i0 + i) qs = a.scale_log2 / g;
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const uint32_t w4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        const __nv_bfloat162 f2 = __float2bfloat162_rn(fac[i]);  // a power of two
                        uint32_t hw[2], lw[2];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w4[k]), f2);
                            const uint32_t hb = *reinterpret_cast<const uint32_t*>(&y) & 0xFFF0FFF0u;
                            const __nv_bfloat162 ly = __hsub2(y, *reinterpret_cast<const __nv_bfloat162*>(&hb));
                            const uint32_t lb = *reinterpret_cast<const uint32_t*>(&ly);
                            const uint32_t hc = cvt_e4m3x2(bf16_bits_to_f32(hb & 0xFFFFu), __uint_as_float(hb & 0xFFFF0000u));
                            const uint32_t lc = cvt_e4m3x2(bf16_bits_to_f32(lb & 0xFFFFu), __uint_as_float(lb & 0xFFFF0000u));
                            hw[k / 2] = (k & 1) ? hw[k / 2] | (hc << 16) : hc;
                            lw[k / 2] = (k & 1) ? lw[k / 2] | (lc << 16) : lc;
                        }
                        const int rr = (i0 + i) * NR + lane / LR;
                        const int at = C::chunk(q * 32 + rr, sub / 2) + (sub & 1) * 8;
                        *reinterpret_cast<uint2*>(qh + at) = make_uint2(hw[0], hw[1]);
                        *reinterpret_cast<uint2*>(qh + C::QB + at) = make_uint2(lw[0], lw[1]);
                    }
                }
                const int r = r0 + (tr < rows ? tr : 0), tok = r / a.G;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::QF + X));
                const SeqInfo s{f->q0, f->n, f->L};
                last = row_last(a, s, tok, pass_of(a));
                first = SHARED ? f->pad[2] : row_first(a, last);
                M = -INFINITY;
                l = 0.f;
                lf = 1.f;
                fresh = true;
            }
            if (begin && !wait(C::CF + sc, it / C::NC)) break;
            begin = flags & kLast;
            if (mine) {
                if (!wait(C::SF + X, own)) break;
                ++own;
                tc_fence_after();
                const uint32_t scl = sbase + C::OFF_SC + sc * kScaleBytes;
                const float2 qs2 = make_float2(qs, qs);
                const float4 tops = ld_shared4(scl + 2 * kUnit * 4);
                const float sv_top = fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w));
                float alpha = 1.f;
                const uint32_t scores = la + D;
                // -inf for those of the unit's keys 16 g .. 16 g + 15 that the row does not see.  Most groups
                // of a masked unit are seen by all of the warp's rows or by none.  Returns whether the row
                // sees one.
                auto hide = [&](float2(&y)[8], int g) -> bool {
                    // computed here: comparisons taken out of a loop would be made for every unit
                    const int at = key0 + g * 16, lo = no_hoist(first - at), hi = no_hoist(last - at);
                    // a run has 16 keys or more
                    const bool hole = (flags & kHoles) && !((f->box_ok >> ((g * 16) >> box_log2)) & 1);
                    if (__all_sync(0xffffffffu, lo <= 0 && hi >= 15) && !hole) return true;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (hole || 2 * i < lo || 2 * i > hi) y[i].x = -INFINITY;
                        if (hole || 2 * i + 1 < lo || 2 * i + 1 > hi) y[i].y = -INFINITY;
                    }
                    return !hole && lo <= 15 && hi >= 0;
                };
                // kChunk keys at a time in a loop, 16 of them side by side with the next scores and key scales on
                // their way.  P of a chunk takes the place of scores that have been read.
                auto softmax = [&](auto masked_tag) {
                    constexpr bool MASKED = decltype(masked_tag)::value;
                    constexpr int NG = (MASKED ? kMaskedChunk : kChunk) / 16;
                    uint32_t x[2][16];
                    float4 sk[4], sv[4];
                    bool raised = false;
                    tmem_ld16(scores, x[0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sk[i] = ld_shared4(scl + i * 16);
                    tmem_wait_ld();
#pragma unroll 1
                    for (int g = 0; g < kUnit / 16;) {
                        uint32_t pw[8 * NG];
                        float2 l2 = make_float2(0.f, 0.f), l3 = l2;
                        bool seen = !MASKED;
                        const float m = M == -INFINITY ? 0.f : M;
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            const int next = j + 1 < NG || g + NG < kUnit / 16 ? g + j + 1 : g + j;
                            if (NG > 1) tmem_ld16(scores + next * 16, x[(j + 1) & 1]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) sv[i] = ld_shared4(scl + kUnit * 4 + (g + j) * 64 + i * 16);
                            float2 y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                y[i] = __fmul2_rn(make_float2(__uint_as_float(x[j & 1][2 * i]), __uint_as_float(x[j & 1][2 * i + 1])),
                                                  (i & 1) ? make_float2(sk[i / 2].z, sk[i / 2].w)
                                                          : make_float2(sk[i / 2].x, sk[i / 2].y));
                            if (NG == 1) tmem_ld16(scores + next * 16, x[0]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) sk[i] = ld_shared4(scl + next * 64 + i * 16);
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = __ffma2_rn(y[i], qs2, make_float2(-m, -m));
                            if (MASKED) seen |= hide(y, g + j);
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = make_float2(ex2_approx(y[i].x), ex2_approx(y[i].y));
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                l2 = __fadd2_rn(l2, y[i]);
                                l3 = __fadd2_rn(l3, y[i + 1]);
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                y[i] = __fmul2_rn(y[i], (i & 1) ? make_float2(sv[i / 2].z, sv[i / 2].w)
                                                                : make_float2(sv[i / 2].x, sv[i / 2].y));
                                pw[j * 8 + i] = pack_f16(y[i].x, y[i].y);
                            }
                            tmem_wait_ld();
                        }
                        const float sum = (l2.x + l2.y) + (l3.x + l3.y);
                        // (a sum of over 2^118: tokens whose values are all zero far above M)
                        const bool raise = (M == -INFINITY && seen) || sum * sv_top > 32768.f || sum > 0x1p118f;
                        if (!raised && __any_sync(0xffffffffu, raise)) {
                            raised = true;
                            // M: the maximum of s + log2 sv, log2 0 counting as -kLeastLog2; then these keys again
                            float mj = -INFINITY;
#pragma unroll 1
                            for (int j = NG - 1; j >= 0; --j) {
                                float2 y[8];
                                tmem_ld16(scores + (g + j) * 16, x[0]);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    sk[i] = ld_shared4(scl + (g + j) * 64 + i * 16);
                                    y[2 * i] = make_float2(__uint_as_float(x[0][4 * i]) * sk[i].x,
                                                           __uint_as_float(x[0][4 * i + 1]) * sk[i].y);
                                    y[2 * i + 1] = make_float2(__uint_as_float(x[0][4 * i + 2]) * sk[i].z,
                                                               __uint_as_float(x[0][4 * i + 3]) * sk[i].w);
                                }
                                if (MASKED) hide(y, g + j);
#pragma unroll
                                for (int i = 0; i < 8; i += 2) {
                                    const float4 v = ld_shared4(scl + kUnit * 4 + (g + j) * 64 + i * 8);
                                    auto lg = [](float x) -> float { return fmaxf(lg2_approx(x), -kLeastLog2); };
                                    mj = max3(mj, fmaf(y[i].x, qs, lg(v.x)), fmaf(y[i].y, qs, lg(v.y)));
                                    mj = max3(mj, fmaf(y[i + 1].x, qs, lg(v.z)), fmaf(y[i + 1].y, qs, lg(v.w)));
                                }
                            }
                            const float mu = floorf(mj);
                            float w = 1.f;
                            if (raise && mu > M) {
                                // M may rise by 228 (values of 2^-100, then of 2^127): l, which is as far below 1
                                // for large values as above it for small ones, in two steps, lf = 1 first if that fits
                                float dn = fmaxf(M - mu, -250.f);
                                w = ex2_approx(dn);
                                if (lf < 1.f && (dn < -32.f || l < 1.f)) {
                                    dn += 64.f;
                                    lf = 1.f;
                                }
                                const float d1 = fmaxf(dn, -120.f);
                                l = l * ex2_approx(d1) * ex2_approx(dn - d1);
                                M = mu;
                            }
                            alpha *= w;
                            // the unit's P sv so far (and, at 16 keys a chunk, of scores that have been read), in
                            // fp32: they may be 2^15 and w 2^-29 with 2^-14 of the new largest left of them
                            tmem_wait_st();
#pragma unroll 1
                            for (int c0 = 0; c0 < g * 8; c0 += 16) {
                                uint32_t z[16];
                                tmem_ld16(scores + c0, z);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&z[i]));
                                    z[i] = pack_f16(v.x * w, v.y * w);
                                }
                                tmem_st16(scores + c0, z);
                            }
                            tmem_wait_st();
                            continue;
                        }
                        raised = false;
                        l = fmaf(sum, lf, l);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            uint32_t z[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) z[i] = pw[j * 8 + i];
                            tmem_st8(scores + (g + j) * 8, z);
                        }
                        g += NG;
                    }
                };
                if (flags & kMasked)
                    softmax(std::true_type{});
                else
                    softmax(std::false_type{});
                if (l > 0x1p100f) {
                    l *= 0x1p-64f;
                    lf *= 0x1p-64f;
                }
                if (!fresh && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O holds every product up to the pipeline's last unit: the scores' completion
                    // covers what was issued before them
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(la + c0, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                                        make_float2(alpha, alpha));
                            o[i] = __float_as_uint(v.x);
                            o[i + 1] = __float_as_uint(v.y);
                        }
                        tmem_st32(la + c0, o);
                    }
                }
                fresh = false;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::PF + X));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::CE + sc));
            const int q0 = f->q0, h = f->h, r0 = f->r0, rows = f->rows, on = f->pad[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::IE + it % C::NI));
            if (!(flags & kLast)) continue;

            // ------------------------------------------------------------ the item's end
            float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
            if (!wait(C::OD + X, items)) break;
            // l below 2, M by as much higher; wa is what O is multiplied by
            const int le = l >= 2.f ? exponent_of(l) : 0, oe = le - exponent_of(lf);
            l *= pow2_whole(-le);
            M += (float)oe;
            float wa = pow2_whole(-oe), wb = 0.f;
            if (!both && X == 1) {
                // A adds the two halves of the keys up; it reads this row's O in tensor memory
                // itself and gets M and l here, once it has read the last ones
                if (items > 0 && !wait(C::OE + 1, items - 1)) break;
                ml[row] = M;
                ml[128 + row] = l;
                ml[256 + row] = wa;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::MB));
                ++items;
                continue;
            }
            const bool add = !both && place > 0;  // B had units of this item
            if (!both) {
                if (!wait(C::OD + 1, items) || !wait(C::MB, shared)) break;
                ++shared;
                if (add) {
                    const float mb = ml[row], lb = ml[128 + row], m = fmaxf(M, mb);
                    const float fa = part_weight(M, m), fb = part_weight(mb, m);
                    l = fa * l + fb * lb;
                    wa *= fa;
                    wb = fb * ml[256 + row];
                    M = m;
                }
            }
            tc_fence_after();
            const bool split = SHARED || flags & (kHead | kTail), there = tr < rows;
            const int slot = 2 * blockIdx.x + ((flags & kHead) ? 0 : 1);
            const int r = r0 + (there ? tr : 0), tok = r / a.G, j = r - tok * a.G;
            const float inv = split ? 1.f : inverse_sum(l);
            const auto part = partials_of<SHARED>(c, a, ws, RT, D);
            // place of this thread's row in the workspace
            auto at_row = [&]() -> int64_t {
                if constexpr (!SHARED) return (int64_t)slot * RT + tr;
                else if (flags & (kHead | kTail)) return (int64_t)slot * RT + tr;
                else
                    return own_slot(a, (int64_t)(q0 + tok) * (c.H * a.G) + h * a.G + j);
            };
            const int64_t o_off = split ? at_row() * D
                                        : (int64_t)(q0 + tok) * a.o_sn + (int64_t)(h * a.G + j) * a.o_sh;
            // Rows go through shared memory (the warp's own rows of the queries, which no product reads
            // any more and no other warp writes for the next item), so that what leaves are whole
            // lines: 32 channels at a time, each row's 16-byte pieces turned by the row.
            uint8_t* stage = smem + C::OFF_Q + 2 * X * C::QB + q * 32 * D;
            auto staged = [&](int r, int piece) -> float4& {  // d = 64: 16 rows fit in each of the two parts
                return *reinterpret_cast<float4*>(stage + r * 128 + (D == 64 && r >= 16 ? C::QB - 2048 : 0) +
                                                  ((piece ^ (r & 7)) << 4));
            };
            const int piece = lane & 7;
            int64_t off[8];  // of the rows that this lane stores a piece of
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rr = 4 * i + lane / 8;  // of the warp's rows
                const int64_t o = __shfl_sync(0xffffffffu, o_off, rr);
                off[i] = tr - lane + rr < rows ? o + 4 * piece : -1;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t oa[32];
                float v[32];
                tmem_ld32(la + c0, oa);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(oa[i]) * wa;
                if (add) {
                    tmem_ld32(la + C::base(1) + c0, oa);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(oa[i]), wb, v[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    staged(lane, i) = make_float4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = 4 * i + lane / 8;
                    const float4 x = staged(rr, piece);
                    if (off[i] < 0) continue;
                    if (split) {
                        *reinterpret_cast<float4*>(part.o + off[i] + c0) = x;
                    } else {
                        const __nv_bfloat162 b0 = __floats2bfloat162_rn(x.x, x.y), b1 = __floats2bfloat162_rn(x.z, x.w);
                        *reinterpret_cast<uint2*>(a.O + off[i] + c0) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::OE + X));
                if (!both) mbar_arrive(bar(C::OE + 1));
            }
            if (there && split) {
                part.m[at_row()] = M;
                part.l[at_row()] = l;
                if constexpr (SHARED)
                    if (!(flags & kHead)) part.word[(int64_t)(q0 + tok) * (c.H * a.G) + h * a.G + j] = row_word(tr, blockIdx.x, on);
            } else if (there) {
                store_lse(a, c, q0, h, r, M, l);
            }
            if constexpr (!SHARED)
                if (split && threadIdx.x == 0)
                    part.head[slot] = PartHeader{on, q0, h, r0, rows};
            ++items;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if constexpr (SHARED) {
        if (threadIdx.x == 0 && *abort_flag) *a.gave_up = 1;
        wait_for_primary();  // the second pass's end is the first one's too
    }
}

template <int D, int kChunk, bool SKIP>
vc_status launch_many_as(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const CacheView& c, int RT,
                         int ctas, void* ws, cudaStream_t st) {
    auto kern = attn_many_kernel<D, kChunk, SKIP, false>;
    vc_status s = ensure_smem_attr(reinterpret_cast<const void*>(kern), ManyCfg<D>::SMEM);
    if (s != VC_OK) return s;
    kern<<<ctas, kThreads, ManyCfg<D>::SMEM, st>>>(mk, mv, a, c, RT, ws);
    return cuda_status(cudaGetLastError());
}

template <int D, int kChunk>
vc_status launch_many(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const CacheView& c, int RT,
                      int ctas, void* ws, cudaStream_t st) {
    return a.skip_unit < 0 ? launch_many_as<D, kChunk, false>(mk, mv, a, c, RT, ctas, ws, st)
                           : launch_many_as<D, kChunk, true>(mk, mv, a, c, RT, ctas, ws, st);
}

template <int D, int kChunk, bool SKIP>
vc_status launch_many_pass_as(const CUtensorMap& mk, const CUtensorMap& mv, const SharedAttn& a, const CacheView& c, int RT,
                              int ctas, cudaStream_t st) {
    auto kern = attn_many_kernel<D, kChunk, SKIP, true>;
    vc_status s = ensure_smem_attr(reinterpret_cast<const void*>(kern), ManyCfg<D>::SMEM);
    if (s != VC_OK) return s;
    return launch_after(kern, dim3(ctas), kThreads, ManyCfg<D>::SMEM, st, mk, mv, a, c, RT, (void*)nullptr);
}

template <int D, int kChunk>
vc_status launch_many_pass(const CUtensorMap& mk, const CUtensorMap& mv, const SharedAttn& a, const CacheView& c, int RT,
                           int ctas, cudaStream_t st) {
    return a.skip_unit < 0 ? launch_many_pass_as<D, kChunk, false>(mk, mv, a, c, RT, ctas, st)
                           : launch_many_pass_as<D, kChunk, true>(mk, mv, a, c, RT, ctas, st);
}

}  // namespace

vc_status launch_attn_many(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const CacheView& c,
                           int d, int RT, int ctas, void* ws, cudaStream_t st) {
    if (d == 64) return launch_many<64, 32>(mk, mv, a, c, RT, ctas, ws, st);
    return RT == 256 ? launch_many<128, 64>(mk, mv, a, c, RT, ctas, ws, st)
                     : launch_many<128, 16>(mk, mv, a, c, RT, ctas, ws, st);
}

vc_status launch_attn_many(const CUtensorMap& mk, const CUtensorMap& mv, const SharedAttn& a, const CacheView& c,
                           int d, int RT, int ctas, cudaStream_t st) {
    if (d == 64) return launch_many_pass<64, 32>(mk, mv, a, c, RT, ctas, st);
    return RT > 128 ? launch_many_pass<128, 64>(mk, mv, a, c, RT, ctas, st)
                     : launch_many_pass<128, 16>(mk, mv, a, c, RT, ctas, st);
}

}  // namespace vc

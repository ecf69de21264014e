// vc_attn_shared.cu -- what attention over shared prefixes (vc_attn_paged_shared) has around its two
// passes: their plan, and the joining of what they leave for each row.
#include <cuda_bf16.h>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kPlan = 1024;
constexpr int kThreads = 128;

// Inclusive sums over the block of two numbers a thread; the totals for all of them.
__device__ __forceinline__ void block_sums(int64_t (&v)[2], int64_t (&total)[2]) {
    __shared__ int64_t sums[2][kPlan / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += u;
        }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) sums[0][warp] = v[0], sums[1][warp] = v[1];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int64_t s = sums[i][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        total[i] = __shfl_sync(0xffffffffu, s, 31);
        const int64_t before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
        v[i] += warp ? before : 0;
    }
}

// shared_plan_kernel: the first block gives every CTA of both passes its part of the pass's line
// (vc_paged.cuh), with the item that it begins in; all blocks clear the rows' words.  The passes
// share the SMs so that both end together.  (Planned by every CTA for itself, those without a part held the
// joining up by 4 us at the end.)
__global__ void __launch_bounds__(kPlan) shared_plan_kernel(const SharedAttn a, const CacheView c) {
    __shared__ int64_t cost[kPlan];
    __shared__ unsigned long long found[3];  // items of the passes, the best share
    const int tid = threadIdx.x, lane = tid & 31;
    launch_dependents();
    const int64_t words = 2 * (int64_t)c.T * c.H * a.G;
    for (int64_t i = (int64_t)blockIdx.x * kPlan + tid; i < words; i += (int64_t)gridDim.x * kPlan) a.words[i] = 0u;
    if (blockIdx.x) return;
    if (tid == 0) *a.gave_up = 0;
    if (tid < 3) found[tid] = tid == 2 ? ~0ull : 0ull;
    int64_t total[2] = {0, 0};
    unsigned long long tiles[2] = {0, 0};
    for (int b0 = 0; b0 < max(a.N, c.B); b0 += kPlan) {
        int64_t u[2], all[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pass = i + 1, seqs = seq_count<true>(c, a, pass), RT = a.rt[i], IC = a.ic[i], b = b0 + tid;
            u[i] = 0;
            if (b0 >= seqs) continue;
            if ((int64_t)c.T * a.G > (int64_t)seqs * RT * 4) {  // many tiles: a warp a sequence
                __syncthreads();
                for (int k = tid >> 5; k < kPlan && b0 + k < seqs; k += kPlan / 32) {
                    const int64_t x = seq_cost_warp<true>(a, seq_of<true>(c, a, b0 + k, pass), RT, IC, pass);
                    if (lane == 0) cost[k] = x * c.H;
                }
                __syncthreads();
                if (b < seqs) u[i] = cost[tid];
            } else if (b < seqs) {
                u[i] = seq_cost<true>(c, a, b, RT, IC, pass) * c.H;
            }
            if (u[i]) tiles[i] += (unsigned long long)seq_tiles(a, seq_of<true>(c, a, b, pass), RT) * c.H;
        }
        block_sums(u, all);
        if (b0 + tid < a.N) a.sums[b0 + tid] = total[0] + u[0];
        if (b0 + tid < c.B) a.sums[a.N + b0 + tid] = total[1] + u[1];
        total[0] += all[0];
        total[1] += all[1];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 16; o; o >>= 1) tiles[i] += __shfl_xor_sync(0xffffffffu, tiles[i], o);
        if (lane == 0 && tiles[i]) atomicAdd(&found[i], tiles[i]);
    }
    __syncthreads();
    // pass 1's share of the SMs: the one with which the later of the two ends first.  A part's time is that of its
    // units and of beginning and ending its items, of which it has one at least.
    int sms = total[1] ? 0 : kMaxCtas;
    if (total[0] && total[1]) {
        if (tid < 160) {  // five warps
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float parts = (float)((i ? kMaxCtas - 1 - tid : tid + 1) * a.per_sm[i]), n = (float)found[i];
                const float units = (float)(total[i] - (int64_t)found[i] * a.ic[i]);
                t = fmaxf(t, (float)a.unit[i] * (units / parts + (float)a.ic[i] * fmaxf(n / parts, 1.f)));
            }
            unsigned long long x = tid < kMaxCtas - 1 ? (unsigned long long)__float_as_uint(t) << 32 | (unsigned)(tid + 1) : ~0ull;
#pragma unroll
            for (int o = 16; o; o >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (lane == 0) atomicMin(&found[2], x);
        }
        __syncthreads();
        sms = (int)(found[2] & 0xFFFFFFFFu);
    }
#pragma unroll
    for (int pass = 1; pass <= 2; ++pass) {
        const int seqs = seq_count<true>(c, a, pass), RT = a.rt[pass - 1], IC = a.ic[pass - 1], per_sm = a.per_sm[pass - 1];
        const int64_t* sums = a.sums + (pass == 1 ? 0 : a.N);
        const int64_t all = total[pass - 1];
        int parts = (pass == 1 ? sms : kMaxCtas - sms) * per_sm;
        if (all < parts) parts = (int)all;  // no empty part between two others
        PlanPart* out = a.plan + (pass == 1 ? 0 : kMaxCtas * a.per_sm[0]);
        for (int i = tid; i < kMaxCtas * per_sm; i += kPlan) {
            PlanPart p{};
            if (i < parts) {
                p.g0 = div_small(all * i, parts);
                p.g1 = div_small(all * (i + 1), parts);
                p.total = all;
                p.parts = parts;
                int lo = 0, hi = seqs - 1;  // the first sequence that ends behind g0
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (sums[mid] > p.g0) hi = mid;
                    else lo = mid + 1;
                }
                const int64_t begin = lo ? sums[lo - 1] : 0, per_head = div_small(sums[lo] - begin, c.H);
                p.b = lo;
                p.s = seq_of<true>(c, a, lo, pass);
                int64_t off = p.g0 - begin;
                p.h = (int)div_small(off, per_head);
                off -= p.h * per_head;
                for (int t = 0;; ++t) {
                    const int x = item_cost<true>(a, p.s, t, RT, IC, pass);
                    if (off < x || t + 1 >= seq_tiles(a, p.s, RT)) {
                        p.tile = t;
                        p.off = (int)off;
                        break;
                    }
                    off -= x;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) reinterpret_cast<int4*>(out + i)[k] = reinterpret_cast<const int4*>(&p)[k];
        }
    }
}

// Reports what breaks the rules of the batch and of its groups.
__device__ __forceinline__ void look_over(const SharedAttn& a, const CacheView& c) {
    for (int b = threadIdx.x; b < c.B; b += kThreads)
        if (!seq_valid_in<true>(c, a, b)) flag_invalid(c.dev_status);
    for (int g = threadIdx.x; g < a.N; g += kThreads)
        if (!group_valid(c, a, g)) flag_invalid(c.dev_status);
}
__global__ void __launch_bounds__(kThreads) shared_check_kernel(const SharedAttn a, const CacheView c) { look_over(a, c); }

// Joining.  A row has parts k, of the prefix and of its own keys, each with a maximum m_k (log2 units),
// a sum l_k and an accumulator A_k; with m their maximum and w_k = 2^(m_k - m),
//   O = sum_k w_k A_k / sum_k w_k l_k,   lse = ln 2 (m + log2 sum_k w_k l_k).
// A row's word in each pass says in which CTA its item begins and how many have parts of it, so
// that one launch joins everything, in key order.  A warp takes a row: the parts' maxima and sums a
// lane each, then their accumulators, D/32 channels a lane.  Where a pass gave up waiting, rows have no
// word, or slots of an earlier call: all of the call's become NaN.
template <int D>
__global__ void __launch_bounds__(kThreads) shared_join_kernel(const SharedAttn a, const CacheView c) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, Hq = c.H * a.G;
    const int64_t rows = (int64_t)c.T * Hq, row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (blockIdx.x == 0) look_over(a, c);  // while the passes run
    wait_for_primary();
    if (row >= rows) return;
    const int tok = (int)(row / Hq), hq = (int)(row - (int64_t)tok * Hq), h = hq / a.G, j = hq - h * a.G;
    const SharedPartials p1 = shared_partials(c, a, 1, D), p2 = shared_partials(c, a, 2, D);
    const uint32_t w1 = __ldcg(p1.word + row), w2 = __ldcg(p2.word + row);
    const bool lost = __ldcg(a.gave_up) != 0;
    if (!(w1 | w2)) {
        // no keys, or no sequence
        const SeqInfo s = seq_info(c, find_seq<32>(c, tok, lane, 0xffffffffu));
        if (tok < s.q0 || tok >= s.q0 + s.n) return;
    }
    const int cta1 = (w1 >> 10) & 1023, cta2 = (w2 >> 10) & 1023, n1 = w1 & 1023, n = n1 + (w2 & 1023);
    // place of part k
    auto place = [&](int k) -> int64_t {
        const bool own = k >= n1;
        const int parts = own ? n - n1 : n1, i = own ? k - n1 : k, cta = own ? cta2 : cta1;
        if (parts == 1) return (own ? slot_rows(a.rt[1], a.per_sm[1]) : slot_rows(a.rt[0], a.per_sm[0])) + row;
        return (int64_t)(i ? 2 * (cta + i) : 2 * cta + 1) * (own ? a.rt[1] : a.rt[0]) + ((own ? w2 : w1) >> 20);
    };
    // 32 parts at a time, a lane each; m is the maximum so far, as a rule of all
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
        float mk = -INFINITY, lk = 0.f;
        int64_t at = 0;
        if (k0 + lane < n) {
            const bool own = k0 + lane >= n1;
            at = place(k0 + lane);
            mk = __ldcg((own ? p2.m : p1.m) + at);
            lk = __ldcg((own ? p2.l : p1.l) + at);
        }
        float top = mk;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(m, top);
        const float before = part_weight(m, top), w = part_weight(mk, top);
        m = top;
        lk *= w;
#pragma unroll
        for (int o = 16; o; o >>= 1) lk += __shfl_xor_sync(0xffffffffu, lk, o);
        l = l * before + lk;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= before;
        const int some = min(n - k0, 32);
#pragma unroll 4
        for (int k = 0; k < some; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float* o = (k0 + k < n1 ? p1.o : p2.o) + __shfl_sync(0xffffffffu, at, k) * D + lane * E;
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
    if (lost) l = __int_as_float(0x7FFFFFFF);
    store_row(a, tok, h, j, lane * E, acc, inverse_sum(l));
    if (lane == 0) store_lse(a, c, tok, h, j, m, l);
}

}  // namespace

vc_status launch_shared_check(const SharedAttn& a, const CacheView& c, cudaStream_t st) {
    shared_check_kernel<<<1, kThreads, 0, st>>>(a, c);
    return cuda_status(cudaGetLastError());
}

vc_status launch_shared_plan(const SharedAttn& a, const CacheView& c, cudaStream_t st) {
    const int64_t words = 2 * (int64_t)c.T * c.H * a.G, blocks = (words + 16 * kPlan - 1) / (16 * kPlan);
    shared_plan_kernel<<<(unsigned)(blocks < kMaxCtas ? blocks : kMaxCtas), kPlan, 0, st>>>(a, c);
    return cuda_status(cudaGetLastError());
}

vc_status launch_shared_join(const SharedAttn& a, const CacheView& c, int d, cudaStream_t st) {
    const dim3 grid((unsigned)(((int64_t)c.T * c.H * a.G + kThreads / 32 - 1) / (kThreads / 32)));
    return d == 128 ? launch_after(shared_join_kernel<128>, grid, kThreads, 0, st, a, c)
                    : launch_after(shared_join_kernel<64>, grid, kThreads, 0, st, a, c);
}

}  // namespace vc
